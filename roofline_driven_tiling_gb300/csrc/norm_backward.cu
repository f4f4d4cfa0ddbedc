// norm_backward.cu -- the gradients of r = scale x + gate drop(post(h)), y = norm(r).
//
// With xh = (r - mean) rho, g = dy weight, and the same for h (hh, sigma) and its gradient:
//   d = dr + rho (g - [mean g] - xh mean(g xh)),  [mean g] for layer norms only;  dx = scale d
//   dn = drop'(d gate),  q = dn post_weight,  dh = sigma (q - [mean q] - hh mean(q hh))
//   dweight = sum dy xh, dbias = sum dy, dgate = sum d drop(n), dpost_weight = sum dn hh, dpost_bias = sum dn
// A CTA takes consecutive rows and adds its rows' share of the five sums in FP32; a second launch adds the
// CTAs' shares in their order.
//
// Rows are read once (N <= 8192). No single limit: instructions (every value of a warp's word costs about 20, 73 % of the issue
// slots), the sums' reads and writes of shared memory for every row, and the second launch of 4 us. With a gate: 8192 x 2048 and
// dropout 52 us (3.9 TB/s), 8192 x 4096 87 (4.6). Layer norms before and after with all five sums: 8192 x 2048 and
// dropout 91, 8192 x 4096 182 (one block of 512 threads to an SM, by the sums' shared memory). Off 16-byte boundaries 4096 x
// 4095 97 (50 on them), 1300 x 1003 26 (nine rows to a block). A gate for each of 4096 rows of 2048 51 us, and one for all 27:
// a block takes its gates one after another. Rows beyond 8192 take passes over memory of two bytes a load: 4096 x 12288 767 us
// (0.8 TB/s). Two words a thread with half the threads were no faster (8192 x 4096 98).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "matrix_args.h"
#include "norm_device.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kWideThreads = 1024;
constexpr int kVectors = 5;
enum Vector : int { kWeight = 0, kBias = 1, kGate = 2, kPostWeight = 3, kPostBias = 4 };

// How the rows lie on the CTAs. Few gates: `pieces` CTAs to each gate's rows. Otherwise a CTA takes whole
// gates (and one gate's sum is complete when its rows are).
struct Split {
  int ctas, pieces;  // pieces 0: whole gates
};
constexpr int kSms = 152, kMostCtas = 2 * kSms;
Split split_of(int64_t M, int64_t gates, int ctas) {
  const int64_t rows = M / gates;
  if (2 * gates > ctas) return {static_cast<int>(gates < ctas ? gates : ctas), 0};
  int64_t pieces = ctas / gates;
  if (pieces > rows) pieces = rows;
  return {static_cast<int>(gates * pieces), static_cast<int>(pieces)};
}

// From one of a CTA's sums to the next: rows of 16-byte words.
__host__ __device__ inline int64_t share_pitch(int64_t N) { return (N + 3) & ~static_cast<int64_t>(3); }

struct BackwardParams {
  BackwardTask t;
  Split split;
  int slot[kVectors];  // of a CTA's partial sums; -1: not wanted
  int slots;
};

// The rows of CTA c, and those of one gate after another among them.
struct Rows {
  int64_t first, last, per_gate;
};
__device__ __forceinline__ Rows rows_of(const BackwardParams& p, int64_t c) {
  const int64_t per_gate = p.t.M / p.t.gates;
  if (p.split.pieces > 0) {
    const int64_t g = c / p.split.pieces, j = c % p.split.pieces;
    return {g * per_gate + per_gate * j / p.split.pieces, g * per_gate + per_gate * (j + 1) / p.split.pieces, per_gate};
  }
  return {p.t.gates * c / p.split.ctas * per_gate, p.t.gates * (c + 1) / p.split.ctas * per_gate, per_gate};
}

// Rows of any length: passes over memory, the partial sums in memory too (each value belongs to one thread).
template <int KIND>
__global__ void __launch_bounds__(kWideThreads) wide_backward_kernel(const __grid_constant__ BackwardParams p) {
  __shared__ float room[96];
  ff::wait_for_earlier_kernels();
  const BackwardTask& t = p.t;
  const int64_t groups = (t.N + 3) / 4;
  const float inv_n = 1.0f / static_cast<float>(t.N);
  const uint64_t key = t.drop.dropped != 0 ? drop_key(t.drop) : 0;
  const Rows rows = rows_of(p, blockIdx.x);
  float* const partials = t.partials + static_cast<int64_t>(blockIdx.x) * p.slots * share_pitch(t.N);
  const bool has_h = t.H.p != nullptr;
  for (int64_t m = rows.first; m < rows.last; ++m) {
    const bool first = m == rows.first, gate_first = p.split.pieces > 0 ? first : m % rows.per_gate == 0;
    const bool gate_last = p.split.pieces == 0 && (m + 1) % rows.per_gate == 0;
    const uint16_t* r = t.R.p + m * t.R.ld;
    const uint16_t* dy = t.dY.p + m * t.dY.ld;
    const uint16_t* dr = t.dR.p == nullptr ? nullptr : t.dR.p + m * t.dR.ld;
    const uint16_t* h = t.H.p + m * t.H.ld;
    const uint16_t* gate = t.gate.p == nullptr ? nullptr : t.gate.p + m / rows.per_gate * t.gate.ld;
    float mean = 0.0f, rho = 1.0f, mean_g = 0.0f, mean_gx = 0.0f;
    if (t.norm == T2S_NORM_LAYER) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(r[n]);
      block_sums(s, room);
      mean = s[0] * inv_n;
    }
    if (t.norm != T2S_NORM_NONE) {
      float s[3] = {};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
        const float c = ff::to_f32<KIND>(r[n]) - mean, g = ff::to_f32<KIND>(dy[n]) * at<KIND>(t.weight, n, 1.0f);
        s[0] = fmaf(c, c, s[0]);
        s[1] += g;
        s[2] = fmaf(g, c, s[2]);
      }
      block_sums(s, room);
      rho = rsqrtf(s[0] * inv_n + t.eps);
      mean_g = t.norm == T2S_NORM_LAYER ? s[1] * inv_n : 0.0f;
      mean_gx = s[2] * inv_n * rho;
    }
    float h_mean = 0.0f, sigma = 1.0f;
    if (has_h && t.post == T2S_NORM_LAYER) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) s[0] += ff::to_f32<KIND>(h[n]);
      block_sums(s, room);
      h_mean = s[0] * inv_n;
    }
    if (has_h && t.post != T2S_NORM_NONE) {
      float s[1] = {0.0f};
      for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
        const float c = ff::to_f32<KIND>(h[n]) - h_mean;
        s[0] = fmaf(c, c, s[0]);
      }
      block_sums(s, room);
      sigma = rsqrtf(s[0] * inv_n + t.eps);
    }
    // d at a column, from memory each time.
    auto gradient = [&](int64_t n) {
      float d = at<KIND>(dr, n, 0.0f);
      if (t.norm != T2S_NORM_NONE) {
        const float xh = (ff::to_f32<KIND>(r[n]) - mean) * rho, g = ff::to_f32<KIND>(dy[n]) * at<KIND>(t.weight, n, 1.0f);
        d += rho * (g - mean_g - xh * mean_gx);
      }
      return d;
    };
    auto add = [&](int vector, int64_t n, float v, bool start) {
      if (p.slot[vector] < 0) return;
      float* to = partials + p.slot[vector] * share_pitch(t.N) + n;
      *to = start ? v : *to + v;
    };
    float s[2] = {};
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
      const float d = gradient(n);
      if (t.norm != T2S_NORM_NONE) {
        const float y = ff::to_f32<KIND>(dy[n]);
        add(kWeight, n, y * ((ff::to_f32<KIND>(r[n]) - mean) * rho), first);
        add(kBias, n, y, first);
      }
      if (t.dX.p != nullptr) t.dX.p[m * t.dX.ld + n] = ff::from_f32<KIND>(t.scale * d);
      if (!has_h) continue;
      const float hh = (ff::to_f32<KIND>(h[n]) - h_mean) * sigma, pw = at<KIND>(t.post_weight, n, 1.0f);
      float v = t.post == T2S_NORM_NONE ? hh : fmaf(hh, pw, at<KIND>(t.post_bias, n, 0.0f));
      float dn = d * at<KIND>(gate, n, 1.0f);
      if (t.drop.dropped != 0) {
        const uint64_t bits = drop_bits(key, static_cast<uint64_t>(m * groups + n / 4));
        v = drop(v, bits, n & 3, t.drop.dropped, t.drop.factor);
        dn = drop(dn, bits, n & 3, t.drop.dropped, t.drop.factor);
      }
      add(kGate, n, d * v, gate_first);
      if (gate_last && p.slot[kGate] >= 0)
        t.dgate.p[m / rows.per_gate * t.dgate.ld + n] = ff::from_f32<KIND>(partials[p.slot[kGate] * share_pitch(t.N) + n]);
      if (t.post == T2S_NORM_NONE) {
        if (t.dH.p != nullptr) t.dH.p[m * t.dH.ld + n] = ff::from_f32<KIND>(dn);
        continue;
      }
      add(kPostWeight, n, dn * hh, first);
      add(kPostBias, n, dn, first);
      s[0] += dn * pw;
      s[1] = fmaf(dn * pw, hh, s[1]);
    }
    if (!has_h || t.post == T2S_NORM_NONE || t.dH.p == nullptr) continue;
    block_sums(s, room);
    const float mean_q = t.post == T2S_NORM_LAYER ? s[0] * inv_n : 0.0f, mean_qh = s[1] * inv_n;
    for (int64_t n = threadIdx.x; n < t.N; n += kWideThreads) {
      float dn = gradient(n) * at<KIND>(gate, n, 1.0f);
      if (t.drop.dropped != 0)
        dn = drop(dn, drop_bits(key, static_cast<uint64_t>(m * groups + n / 4)), n & 3, t.drop.dropped, t.drop.factor);
      const float hh = (ff::to_f32<KIND>(h[n]) - h_mean) * sigma;
      t.dH.p[m * t.dH.ld + n] =
          ff::from_f32<KIND>(sigma * (dn * at<KIND>(t.post_weight, n, 1.0f) - mean_q - hh * mean_qh));
    }
  }
}

// Rows of up to 8192 values: a group of threads takes a row, a word of eight values a thread; a block holds several
// groups. The row's r, dy, dr and h come to shared memory, r and h of the next row as soon as this row's are in
// registers, and the parameters' words stay there. The sums over rows are added in shared memory too, each group's in its
// own place. All of these places belong to one thread each. At the end of a block's rows (of a gate's for dgate) the
// groups' sums are added in their order.
enum Place : int { kR = 0, kDy = 1, kDr = 2, kH = 3, kW = 4, kG = 5, kPw = 6, kPb = 7, kPlaces = 8 };
struct RowParams {
  row::View in[kPlaces], dx, dh;
  int at[kPlaces], sum_at[kVectors];  // of their words in shared memory, in bytes; -1: absent, or no room
  int sum_slots, sum_first;
  int rows_per_gate, share, longer;  // a block's rows of a gate, or its gates: one more in the first `longer` blocks
  int inner_end;  // of the rows whose aligned words lie within r, dy, dr and h
  Split split;
  int N, threads;  // threads of a row
  int norm, post;
  float scale, eps;
  Dropout drop;
  Matrix dgate;
  float* partials;
};

template <int KIND, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_backward_kernel(const __grid_constant__ RowParams p) {
  extern __shared__ uint4 words[];
  __shared__ float rooms[row::Group::kRoomFloats];
  constexpr uint32_t kSumPitch = THREADS * 16;  // in shared memory, from one of a sum's two places of a thread to the other
  row::Group group(p.threads, rooms);
  const int n = p.N, rows_at_once = static_cast<int>(blockDim.x) / p.threads;
  const int first_column = group.rank * row::kWord, left = n - first_column;
  const uint32_t first_byte = 2u * static_cast<uint32_t>(first_column);
  const uint32_t mine = smem_u32(words) + row::place_of_thread<WIDE>(), my_sums = smem_u32(words) + threadIdx.x * 16u;
  // A sum's eight values are two places of 16 bytes.
  for (int i = 0; i < 2 * p.sum_slots; ++i) st_shared_v4(my_sums + p.sum_first + i * kSumPitch, 0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int i = 0; i < kPlaces; ++i)
    if (p.at[i] >= 0) row::clear_place<WIDE>(mine + p.at[i], left);
  ff::wait_for_earlier_kernels();
  auto fetch = [&](int place, const uint16_t* from, bool inside) {
    if (p.at[place] >= 0) row::fetch_word<WIDE>(mine + p.at[place], p.in[place], from, left, inside);
  };
  auto settle = [&](int place, const uint16_t* from) {
    if (!WIDE && p.at[place] >= 0) row::settle<WIDE>(mine + p.at[place], from, left);
  };
  auto get = [&](int place, uint64_t(&f)[4]) { row::unpack<KIND>(row::arrived<WIDE>(mine + p.at[place], left), f); };
  // A parameter's words, in shared memory, or read again for each row where that is full.
  int gate_row = 0;
  auto parameter = [&](int place, uint64_t(&f)[4]) {
    if (p.at[place] >= 0) {
      get(place, f);
    } else {
      const uint16_t* from = p.in[place].row(place == kG ? gate_row : 0, first_byte);
      row::unpack<KIND>(row::load_word<WIDE>(p.in[place], from, left), f);
    }
  };
  fetch(kW, p.in[kW].row(0, first_byte), false);
  fetch(kPw, p.in[kPw].row(0, first_byte), false);
  fetch(kPb, p.in[kPb].row(0, first_byte), false);
  int fresh = kW;  // which parameters' words are new: all, the gate's (kG), none (kPlaces)
  const uint32_t groups = (static_cast<uint32_t>(n) + 3u) / 4u;
  const float inv_n = 1.0f / static_cast<float>(n);
  const uint64_t key = p.drop.dropped != 0 ? drop_key(p.drop) : 0;
  const bool has_h = p.in[kH].p != nullptr, has_norm = p.norm != T2S_NORM_NONE, has_post = has_h && p.post != T2S_NORM_NONE;
  const bool layer = p.norm == T2S_NORM_LAYER, post_layer = has_post && p.post == T2S_NORM_LAYER;

  auto add = [&](int vector, const uint64_t(&f)[4]) {
    if (p.sum_at[vector] < 0) return;
    const uint32_t to = my_sums + p.sum_at[vector];
    uint64_t a, b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lds128_pairs(to + i * kSumPitch, a, b);
      a = row::add2(a, f[2 * i]), b = row::add2(b, f[2 * i + 1]);
      asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(to + i * kSumPitch), "l"(a), "l"(b) : "memory");
    }
  };
  // Four columns of a sum from place `q` (two places a sum) over the groups, in their order; cleared if `clear`.
  auto total = [&](int q, bool clear) {
    float4* from = reinterpret_cast<float4*>(words + p.sum_first / 16) + q * THREADS + group.rank;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int g = 0; g < rows_at_once; ++g, from += p.threads) {
      const float4 v = *from;
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      if (clear) *from = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    return s;
  };

  int first, last;
  if (p.split.pieces > 0) {
    const int g = static_cast<int>(blockIdx.x) / p.split.pieces, j = static_cast<int>(blockIdx.x) - g * p.split.pieces;
    first = g * p.rows_per_gate + j * p.share + min(j, p.longer);
    last = first + p.share + (j < p.longer ? 1 : 0);
  } else {
    const int j = static_cast<int>(blockIdx.x);
    first = (j * p.share + min(j, p.longer)) * p.rows_per_gate;
    last = first + (p.share + (j < p.longer ? 1 : 0)) * p.rows_per_gate;
  }
  // One gate's rows after another (one stretch of rows where a gate has several blocks).
  const int stretch = p.split.pieces > 0 ? last - first : p.rows_per_gate;
  for (int m0 = first; m0 < last; m0 += stretch) {
    const int end = m0 + stretch;
    gate_row = m0 / p.rows_per_gate;
    fetch(kG, p.in[kG].row(gate_row, first_byte), false);
    if (fresh == kPlaces) fresh = kG;
    int m = m0 + group.index;
    if (m < end)
#pragma unroll 1
      for (int i = kR; i <= kH; ++i) fetch(i, p.in[i].row(m, first_byte), false);
    for (; m < end; m += rows_at_once) {
      auto fetch_next = [&](int i) {
        const int r = m + rows_at_once;
        if (r < end) fetch(i, p.in[i].row(r, first_byte), r < p.inner_end);
      };
      row::wait_copies();
      if (!WIDE) {
        // The row's words, and the parameters' when they are new.
#pragma unroll 1
        for (int i = kR; i < (fresh < kPlaces ? kPlaces : kW); ++i)
          if (i <= kH || i == kG || fresh == kW) settle(i, p.in[i].row(i <= kH ? m : i == kG ? gate_row : 0, first_byte));
        fresh = kPlaces;
      }
      uint64_t xh[4], hh[4], d[4];
      if (has_norm) get(kR, xh);
      if (has_h) get(kH, hh);
      fetch_next(kR);
      fetch_next(kH);
      if (layer || post_layer) {
        float means[2] = {0.0f, 0.0f};
        if (layer) means[0] = row::sum(xh);
        if (post_layer) means[1] = row::sum(hh);
        group.sums(means);
        if (layer) {
#pragma unroll
          for (int i = 0; i < 4; ++i) xh[i] = row::add2(xh[i], row::both(-means[0] * inv_n));
          row::clear_from<WIDE>(xh, left);
        }
        if (post_layer) {
#pragma unroll
          for (int i = 0; i < 4; ++i) hh[i] = row::add2(hh[i], row::both(-means[1] * inv_n));
          row::clear_from<WIDE>(hh, left);
        }
      }
      float rho = 1.0f, sigma = 1.0f, mean_g = 0.0f, mean_gx = 0.0f;
      // dy weight stays in registers, but for rows off boundaries, whose code has none to spare: there it is formed again
      // (4096 x 4095 97 us, and 103 with what the compiler then kept in memory; 8192 x 2048 with dropout 55 us and 53).
      constexpr bool kKeepG = WIDE;
      uint64_t g[4];
      if (has_norm || has_post) {
        float s[4] = {};
        if (has_norm) {
          uint64_t w[4];
          get(kDy, g);
          if (p.in[kW].p != nullptr) {
            parameter(kW, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = row::mul2(g[i], w[i]);
          }
          s[0] = row::dot(xh, xh);
          s[1] = row::dot(g, xh);
          if (layer) s[2] = row::sum(g);
        }
        if (has_post) s[3] = row::dot(hh, hh);
        if (layer || has_post) {
          group.sums(s);
        } else {
          float two[2] = {s[0], s[1]};
          group.sums(two);
          s[0] = two[0], s[1] = two[1];
        }
        if (has_norm) {
          rho = rsqrtf(s[0] * inv_n + p.eps);
          mean_gx = s[1] * inv_n * rho;
          mean_g = s[2] * inv_n;
        }
        if (has_post) sigma = rsqrtf(s[3] * inv_n + p.eps);
      }
      float q[2] = {0.0f, 0.0f};
      uint64_t f[4], w[4];
      if (p.at[kDr] >= 0) {
        get(kDr, d);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = 0;
      }
      if (has_norm) {
        get(kDy, f);
        add(kBias, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xh[i] = row::mul2(xh[i], row::both(rho));
          w[i] = row::mul2(f[i], xh[i]);
        }
        add(kWeight, w);
        if (!kKeepG) {
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = f[i];
          if (p.in[kW].p != nullptr) {
            parameter(kW, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = row::mul2(g[i], w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = row::fma2(xh[i], row::both(-mean_gx), g[i]);
          if (layer) f[i] = row::add2(f[i], row::both(-mean_g));
          d[i] = row::fma2(f[i], row::both(rho), d[i]);
        }
        if (layer) row::clear_from<WIDE>(d, left);  // the mean is not for the values beyond the row's end
      }
      if (p.dx.p != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = row::mul2(d[i], row::both(p.scale));
        row::store_word<WIDE>(p.dx, p.dx.row(m, first_byte), left, row::pack<KIND>(f));
      }
      if (has_h) {
        row::Keep keep;
        if (p.drop.dropped != 0) {
          keep.draw(key, static_cast<uint64_t>(static_cast<uint32_t>(m)) * groups + static_cast<uint32_t>(first_column) / 4u, p.drop.dropped);
          // The kept values' factor, for everything that follows.
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = row::mul2(d[i], row::both(p.drop.factor));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) hh[i] = row::mul2(hh[i], row::both(sigma));
        if (p.sum_at[kGate] >= 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = hh[i];
          if (p.in[kPw].p != nullptr) {
            parameter(kPw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = row::mul2(f[i], w[i]);
          }
          if (p.in[kPb].p != nullptr) {
            parameter(kPb, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = row::add2(f[i], w[i]);
          }
          if (p.drop.dropped != 0) keep.apply(f);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = row::mul2(f[i], d[i]);
          add(kGate, f);
        }
        if (p.in[kG].p != nullptr) {
          parameter(kG, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = row::mul2(d[i], w[i]);
        }
        if (p.drop.dropped != 0) keep.apply(d);
        if (has_post) {
          add(kPostBias, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = row::mul2(d[i], hh[i]);
          add(kPostWeight, f);
          if (p.in[kPw].p != nullptr) {
            parameter(kPw, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = row::mul2(d[i], w[i]);
          }
          if (post_layer) q[0] = row::sum(d);
          q[1] = row::dot(d, hh);
        }
      }
      fetch_next(kDy);
      fetch_next(kDr);
      if (p.dh.p == nullptr) continue;
      if (has_post) {
        group.sums(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[i] = row::fma2(hh[i], row::both(-q[1] * inv_n), d[i]);
          if (post_layer) d[i] = row::add2(d[i], row::both(-q[0] * inv_n));
          d[i] = row::mul2(d[i], row::both(sigma));
        }
      }
      row::store_word<WIDE>(p.dh, p.dh.row(m, first_byte), left, row::pack<KIND>(d));
    }
    if (p.split.pieces == 0 && p.sum_at[kGate] >= 0) {
      __syncthreads();
      for (int half = group.index; half < 2; half += rows_at_once) {
        const int i = first_column + 4 * half;
        if (i >= n) continue;
        const float4 v = total((p.sum_at[kGate] - p.sum_first) / static_cast<int>(kSumPitch) + half, true);
        uint16_t* to = p.dgate.p + static_cast<int64_t>(gate_row) * p.dgate.ld + i;
        const uint2 w = make_uint2(ff::pack_f32<KIND>(v.x, v.y), ff::pack_f32<KIND>(v.z, v.w));
        if (i + 4 <= n && (reinterpret_cast<uintptr_t>(to) & 7u) == 0) {
          *reinterpret_cast<uint2*>(to) = w;
        } else {
          row::store_values(to, 0, min(4, n - i), make_uint4(w.x, w.y, 0u, 0u));
        }
      }
      __syncthreads();
    }
  }
  row::wait_copies();  // a group without a row has waited for none: its parameters' copies land before the CTA's memory goes
  __syncthreads();
  // The groups share out the places.
  float* const out = p.partials + static_cast<int64_t>(blockIdx.x) * p.sum_slots * share_pitch(n);
  for (int q = group.index; q < 2 * p.sum_slots; q += rows_at_once) {
    const int i = first_column + 4 * (q & 1);
    if (i < n) *reinterpret_cast<float4*>(out + (q >> 1) * share_pitch(n) + i) = total(q, false);
  }
}

// Adds the CTAs' shares: a block takes 32 columns of one vector (or of one row of dgate), its warps every
// kSumWarps-th share each.
constexpr int kSumWarps = 16;
struct SumParams {
  const float* partials;
  int64_t N, ldgate;
  uint16_t* out[kVectors];
  int slot[kVectors];
  int slots, ctas, pieces, vectors, gate_rows;
};

template <int KIND>
__global__ void __launch_bounds__(32 * kSumWarps) share_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ float room[kSumWarps][33];
  ff::wait_for_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Vectors other than the gate first, then the gate's rows.
  int v = static_cast<int>(blockIdx.y), first = 0, last = p.ctas;
  int64_t row = 0;
  if (v >= p.vectors) {
    row = v - p.vectors;
    v = kGate;
    first = static_cast<int>(row) * p.pieces, last = first + p.pieces;
  }
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  // The slot's vector: the v-th wanted one that is not the gate.
  int which = v;
  if (static_cast<int>(blockIdx.y) < p.vectors) {
    which = 0;
    for (int left = v; which < kVectors; ++which) {
      if (which == kGate || p.slot[which] < 0) continue;
      if (left-- == 0) break;
    }
  }
  float sum = 0.0f;
  if (n < p.N)
#pragma unroll 10
    for (int c = first + warp; c < last; c += kSumWarps)
      sum += p.partials[(static_cast<int64_t>(c) * p.slots + p.slot[which]) * share_pitch(p.N) + n];
  room[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || n >= p.N) return;
  for (int i = 1; i < kSumWarps; ++i) sum += room[i][lane];
  p.out[which][row * p.ldgate + n] = ff::from_f32<KIND>(sum);
}

// How the row kernel takes a row: threads of a row, of a block.
struct RowPlan {
  int threads, block;  // threads 0: too long
  int pitch() const { return block <= 512 ? 512 : 1024; }  // the kernel's THREADS
};
RowPlan row_plan(int64_t N) {
  const int64_t words = (N + row::kWord - 1) / row::kWord;
  if (words > 1024) return {0, 0};
  const int threads = static_cast<int>((words + 31) / 32 * 32);
  return {threads, threads <= 512 ? 512 / threads * threads : threads};
}

// Of a block, beside the 1 KB of rooms: what rows of more than 4096 values off boundaries take with all four inputs and all five
// sums, to the byte (2048 x 4097 so 120 us and 2048 x 8191 157, and 226 and 453 in passes over memory).
constexpr int kMostSmem = 226 * 1024;

// Places in shared memory: inputs, parameters (those only while there is room for them all), sums. False: the inputs
// and sums alone do not fit.
template <bool WIDE>
bool lay_out(RowParams* p, const RowPlan& plan, const int* slot, int* bytes) {
  const int word = plan.pitch() * 16, in_word = plan.pitch() / 32 * static_cast<int>(row::kWarpBytes<WIDE>);
  int ins = 0, all = 0;
  for (int i = 0; i < kPlaces; ++i) {
    const bool present = p->in[i].p != nullptr;
    ins += present && i <= kH;
    all += present;
  }
  const int sums = 2 * p->sum_slots * word;
  const bool parameters = all * in_word + sums <= kMostSmem;
  if (ins * in_word + sums > kMostSmem) return false;
  int used = 0;
  for (int i = 0; i < kPlaces; ++i) {
    const bool here = p->in[i].p != nullptr && (i <= kH || parameters);
    p->at[i] = here ? used : -1;
    if (here) used += in_word;
  }
  p->sum_first = used;
  for (int i = 0; i < kVectors; ++i) p->sum_at[i] = slot[i] >= 0 ? used + 2 * slot[i] * word : -1;
  *bytes = used + sums;
  return true;
}

template <int KIND, bool WIDE, int THREADS>
cudaError_t launch_rows(const RowParams& p, const RowPlan& plan, int smem, cudaStream_t stream) {
  cudaError_t e = prepare_smem<row_backward_kernel<KIND, WIDE, THREADS>>(kMostSmem);
  return e != cudaSuccess ? e
                          : ff::launch_early(stream, {dim3(static_cast<unsigned>(p.split.ctas)), plan.block, 1, smem},
                                             row_backward_kernel<KIND, WIDE, THREADS>, p);
}

template <int KIND, bool WIDE>
cudaError_t run_rows(const RowParams& p, const RowPlan& plan, int smem, cudaStream_t stream) {
  return plan.block <= 512 ? launch_rows<KIND, WIDE, 512>(p, plan, smem, stream)
                           : launch_rows<KIND, WIDE, 1024>(p, plan, smem, stream);
}

template <int KIND>
cudaError_t run(const BackwardTask& t, cudaStream_t stream) {
  uint16_t* const outs[kVectors] = {t.dweight, t.dbias, t.dgate.p, t.dpost_weight, t.dpost_bias};
  int slot[kVectors], slots = 0;
  SumParams s;
  memset(&s, 0, sizeof(s));
  for (int i = 0; i < kVectors; ++i) {
    slot[i] = s.slot[i] = outs[i] != nullptr ? slots++ : -1;
    s.out[i] = outs[i];
    if (i != kGate && outs[i] != nullptr) ++s.vectors;
  }
  if (slots == 0 && t.dX.p == nullptr && t.dH.p == nullptr) return cudaSuccess;
  RowPlan plan = row_plan(t.N);
  cudaError_t e;
  Split split;
  RowParams p;
  memset(&p, 0, sizeof(p));
  bool wide = false;
  int smem = 0;
  if (plan.threads > 0) {
    const Input in[kPlaces] = {t.norm != T2S_NORM_NONE ? t.R : Input{}, t.dY, t.dR, t.H, {t.weight, 0}, t.gate,
                               {t.post_weight, 0}, {t.post_bias, 0}};
    p.dx = row::view_of(t.dX.p, t.dX.ld, t.M, t.N), p.dh = row::view_of(t.dH.p, t.dH.ld, t.M, t.N);
    wide = row::whole_words(p.dx, t.N) && row::whole_words(p.dh, t.N);
    for (int i = 0; i < kPlaces; ++i) {
      p.in[i] = row::view_of(in[i].p, in[i].ld, i <= kH ? t.M : i == kG ? t.gates : 1, t.N);
      wide = wide && row::whole_words(p.in[i], t.N);
    }
    p.inner_end = static_cast<int>(t.M);
    for (int i = kR; i <= kH; ++i) {
      const int end = static_cast<int>(row::inner_end(p.in[i], t.M));
      if (end < p.inner_end) p.inner_end = end;
    }
    p.sum_slots = slots;
    p.rows_per_gate = static_cast<int>(t.M / t.gates), p.N = static_cast<int>(t.N), p.threads = plan.threads;
    p.norm = t.norm, p.post = t.post, p.scale = t.scale, p.eps = t.eps, p.drop = t.drop;
    p.dgate = t.dgate, p.partials = t.partials;
    if (!(wide ? lay_out<true>(&p, plan, slot, &smem) : lay_out<false>(&p, plan, slot, &smem))) plan.threads = 0;
  }
  if (plan.threads > 0) {
    p.split = split = split_of(t.M, t.gates, plan.block <= 512 && smem <= 112 * 1024 ? kMostCtas : kSms);
    const int parts = split.pieces > 0 ? split.pieces : split.ctas;
    const int whole = split.pieces > 0 ? p.rows_per_gate : static_cast<int>(t.gates);
    p.share = whole / parts, p.longer = whole % parts;
    e = wide ? run_rows<KIND, true>(p, plan, smem, stream) : run_rows<KIND, false>(p, plan, smem, stream);
  } else {
    BackwardParams b;
    b.t = t;
    b.split = split = split_of(t.M, t.gates, kMostCtas);
    for (int i = 0; i < kVectors; ++i) b.slot[i] = slot[i];
    b.slots = slots;
    e = ff::launch_early(stream, {dim3(static_cast<unsigned>(split.ctas)), kWideThreads, 1, 0}, wide_backward_kernel<KIND>, b);
  }
  if (e != cudaSuccess) return e;
  s.gate_rows = t.dgate.p != nullptr && split.pieces > 0 ? static_cast<int>(t.gates) : 0;
  if (s.vectors + s.gate_rows == 0) return cudaSuccess;
  s.partials = t.partials;
  s.N = t.N;
  s.ldgate = t.dgate.ld;
  s.slots = slots;
  s.ctas = split.ctas;
  s.pieces = split.pieces;
  const dim3 grid(static_cast<unsigned>((t.N + 31) / 32), static_cast<unsigned>(s.vectors + s.gate_rows));
  return ff::launch_early(stream, {grid, 32 * kSumWarps, 1, 0}, share_sum_kernel<KIND>, s);
}

}  // namespace

size_t backward_workspace_bytes(int64_t M, int64_t N, int64_t gates, int vectors) {
  if (M == 0 || N == 0 || vectors == 0) return 0;
  return static_cast<size_t>(split_of(M, gates, kMostCtas).ctas) * static_cast<size_t>(vectors) *
         static_cast<size_t>(share_pitch(N)) * 4;
}

cudaError_t run_backward(const BackwardTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s

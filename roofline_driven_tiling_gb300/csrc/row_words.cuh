// row_words.cuh -- rows of 16-bit values in words of eight, wherever the rows start, arithmetic on the words in
// packed FP32 pairs, and sums over the threads of a row.
#pragma once

#include "drop.cuh"
#include "ff_math.cuh"
#include "t2s_device.cuh"

namespace t2s {
namespace row {

constexpr int kWord = 8;  // consecutive values of a row that a thread takes at a time: 16 bytes

// A matrix of 16-bit values as the kernels read and write it.
struct View {
  uint16_t* p;  // nullptr: absent
  int64_t ld;
  const uint16_t* end;  // after its last value
  int wide;             // every row starts on a 16-byte boundary

  // Row m from byte `at` on: sizes and strides are at most 2^30, so that 32-bit factors do.
  __device__ __forceinline__ uint16_t* row(int m, uint32_t at) const {
    return reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(p) +
                                       static_cast<uint64_t>(static_cast<uint32_t>(m)) * (2u * static_cast<uint32_t>(ld)) + at);
  }
};
// Whether a matrix consists of whole aligned words, or is absent.
inline bool whole_words(const View& v, int64_t cols) { return v.p == nullptr || (v.wide && cols % kWord == 0); }
inline View view_of(const uint16_t* p, int64_t ld, int64_t rows, int64_t cols) {
  View v;
  v.p = const_cast<uint16_t*>(p);
  v.ld = rows > 1 ? ld : 0;
  v.end = p == nullptr ? nullptr : p + (rows - 1) * v.ld + cols;
  v.wide = ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(v.ld * 2)) & 15u) == 0;
  return v;
}
// The first row whose aligned words may reach beyond the end of a matrix of `rows` rows. A row's words hold up to seven values
// before and after its own, which lie in the rows around it: in one, or in several rows of fewer than seven values. (At
// the matrix's start as many rows are meant; fetch_word's `inside` says how they are kept out.)
inline int64_t inner_end(const View& v, int64_t rows) {
  if (v.p == nullptr || v.ld == 0) return rows;
  return rows - (v.ld < kWord - 1 ? (kWord - 2 + v.ld) / v.ld : 1);
}

// The eight words' values from 32-bit words w[o] on: a shift by o = 1 to 7 values, the same for a whole row.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int o) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (o & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (o & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (o & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first `left` of eight values, the others 0.
__device__ __forceinline__ uint4 first_of(const uint4& v, int left) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = left >= 2 * i + 2 ? w[i] : left == 2 * i + 1 ? w[i] & 0xffffu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sixteen bytes from p to shared memory in the background, `bytes` of them read and the others 0.
__device__ __forceinline__ void copy_async(uint32_t to, const void* p, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A place in shared memory for a word of each thread: 16 bytes apart, and where words are not WIDE with room for one more
// after each warp's.
template <bool WIDE>
constexpr uint32_t kWarpBytes = WIDE ? 512u : 528u;
template <bool WIDE>
__device__ __forceinline__ uint32_t place_of_thread() {
  return threadIdx.x / 32 * kWarpBytes<WIDE> + threadIdx.x % 32 * 16u;
}

// Eight values of v's row from p on, `left` (perhaps none) of them inside the row, on their way to this thread's place in
// shared memory, where settle() puts them together after wait_copies(). WIDE: every row starts on a 16-byte boundary and
// holds whole words. Otherwise the lanes of a warp, which hold consecutive words of a row, bring the aligned words that
// their first values lie in, and the last of them one more, as far as the matrix reaches.
// Rows next to the matrix's ends are brought with care for what lies outside; that code is not inlined (the norm kernels
// fetch, read and write words at many places, and with the code for every case at each of them they were up to 130 KB long
// and bound by fetching it).
static __device__ __noinline__ void fetch_part(uint32_t to, const uint16_t* begin, const uint16_t* end, const uint16_t* p,
                                               int left) {
  const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1, n = min(left, kWord);
  const uint16_t* from = p - o;
  if (from >= begin) {
    copy_async(to, from, static_cast<int>(min(static_cast<int64_t>(16), 2 * (end - from))));
  } else {  // the first word of the matrix
    for (int i = 0; i < n && o + i < kWord; ++i)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 2u * static_cast<uint32_t>(o + i)), "h"(p[i]) : "memory");
  }
  if (o + n > kWord && (threadIdx.x % 32 == 31 || left <= kWord))
    copy_async(to + 16u, from + kWord, static_cast<int>(min(static_cast<int64_t>(16), 2 * (end - from - kWord))));
}
// `inside`: all of the row's aligned words lie within the matrix. The callers say so of the rows below inner_end() that a
// group takes after its first: rows of fewer than seven values are then the 16th or a later one, longer ones the second.
template <bool WIDE>
__device__ __forceinline__ void fetch_word(uint32_t to, const View& v, const uint16_t* p, int left, bool inside) {
  if (left <= 0) return;
  const char* from = reinterpret_cast<const char*>(p);
  if (!WIDE) {
    if (!inside) {
      fetch_part(to, v.p, v.end, p, left);
      return;
    }
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    from -= off;
    if ((threadIdx.x % 32 == 31 || left <= kWord) && static_cast<int>(off) + 2 * min(left, kWord) > 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16u), "l"(from + 16) : "memory");
  }
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// After wait_copies(), by all lanes of a warp: puts the words that fetch_word(to, v, p, left) brought together at `to`,
// zeros beyond the row's end, from where arrived() reads them as often as they are wanted.
template <bool WIDE>
__device__ __forceinline__ void settle(uint32_t to, const uint16_t* p, int left) {
  if (WIDE) return;
  const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;  // the same in a warp
  if (o == 0) {
    // Each lane's word lies in its place, which no other lane touches.
    if (left < kWord && left > 0) {
      const uint4 v = first_of(load_shared(to), left);
      st_shared_v4(to, v.x, v.y, v.z, v.w);
    }
    return;
  }
  __syncwarp();  // the lanes' copies, for one another
  uint4 v = make_uint4(0, 0, 0, 0);
  if (left > 0) v = shifted(load_shared(to), load_shared(to + 16u), o);
  if (left < kWord) v = first_of(v, left);
  __syncwarp();
  if (left > 0) st_shared_v4(to, v.x, v.y, v.z, v.w);
}
// WIDE: threads beyond the row's end have zeros in their places (clear_place(), before the first word is fetched), so that
// nothing is asked at each read. Otherwise the copies of the lane before may lie there.
template <bool WIDE>
__device__ __forceinline__ uint4 arrived(uint32_t to, int left) {
  return WIDE || left > 0 ? load_shared(to) : make_uint4(0, 0, 0, 0);
}
template <bool WIDE>
__device__ __forceinline__ void clear_place(uint32_t to, int left) {
  if (WIDE && left <= 0) st_shared_v4(to, 0u, 0u, 0u, 0u);
}

// The same at once, where there is no place for it.
static __device__ __noinline__ uint4 load_part(const uint16_t* p, int left, const uint16_t* begin, const uint16_t* end) {
  const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
  const uint16_t* from = p - o;
  const bool two = o + min(left, kWord) > kWord;
  if (from >= begin && from + (two ? 16 : 8) <= end) {
    const uint4 a = reinterpret_cast<const uint4*>(from)[0];
    const uint4 b = two ? reinterpret_cast<const uint4*>(from)[1] : make_uint4(0, 0, 0, 0);
    return first_of(o == 0 ? a : shifted(a, b, o), left);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 2 * i < left ? p[2 * i] : 0u;
    if (2 * i + 1 < left) w[i] |= static_cast<uint32_t>(p[2 * i + 1]) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool WIDE>
__device__ __forceinline__ uint4 load_word(const View& v, const uint16_t* p, int left) {
  if (left <= 0) return make_uint4(0, 0, 0, 0);
  if (WIDE || (v.wide && left >= kWord)) return *reinterpret_cast<const uint4*>(p);
  return load_part(p, left, v.p, v.end);
}

// The same in two steps, so that several words' loads are on their way before the first is put together.
template <bool WIDE>
struct RawWord {
  uint4 a, b;
  __device__ __forceinline__ static bool whole(const View& v, const uint16_t* p, int left, int o) {
    return p - o >= v.p && p - o + (o + min(left, kWord) > kWord ? 16 : 8) <= v.end;
  }
  __device__ __forceinline__ void load(const View& v, const uint16_t* p, int left) {
    a = b = make_uint4(0, 0, 0, 0);
    if (left <= 0) return;
    if (WIDE) {
      a = *reinterpret_cast<const uint4*>(p);
      return;
    }
    const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
    if (!whole(v, p, left, o)) return;
    a = reinterpret_cast<const uint4*>(p - o)[0];
    if (o + min(left, kWord) > kWord) b = reinterpret_cast<const uint4*>(p - o)[1];
  }
  __device__ __forceinline__ uint4 get(const View& v, const uint16_t* p, int left) const {
    if (WIDE || left <= 0) return a;
    const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;
    if (!whole(v, p, left, o)) return load_part(p, left, v.p, v.end);
    return first_of(o == 0 ? a : shifted(a, b, o), left);
  }
};

__device__ __forceinline__ void store_values(uint16_t* p, int first, int last, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < kWord; ++i)
    if (i >= first && i < last) p[i] = static_cast<uint16_t>(w[i / 2] >> 16 * (i & 1));
}

// Stores a word of each lane of a converged warp (`left` <= 0: none), consecutive lanes holding consecutive words of
// a row. Off 16-byte boundaries a lane writes the aligned word that its first values share with the lane before,
// and the lanes at the ends write the rest value by value.
static __device__ __noinline__ void store_some(uint16_t* p, int first, int last, uint4 x) { store_values(p, first, last, x); }
template <bool WIDE>
__device__ __forceinline__ void store_word(const View& v, uint16_t* p, int left, const uint4& x) {
  if (WIDE) {
    if (left > 0) *reinterpret_cast<uint4*>(p) = x;
    return;
  }
  const int o = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) >> 1;  // the same in a warp
  if (v.wide || o == 0) {
    if (left >= kWord) {
      *reinterpret_cast<uint4*>(p) = x;
    } else if (left > 0) {
      store_some(p, 0, left, x);
    }
    return;
  }
  const int lane = threadIdx.x & 31, head = kWord - o;  // this lane's values in the aligned word that holds p
  uint4 before;
  before.x = __shfl_up_sync(0xffffffffu, x.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, x.y, 1);
  before.z = __shfl_up_sync(0xffffffffu, x.z, 1);
  before.w = __shfl_up_sync(0xffffffffu, x.w, 1);
  const bool whole = lane > 0 && left >= head, next_whole = lane < 31 && left - kWord >= head;
  if (whole) *reinterpret_cast<uint4*>(p - o) = shifted(before, x, head);
  const int first = whole ? head : 0, last = next_whole ? head : min(left, kWord);
  if (first < last) store_some(p, first, last, x);
}

// ------------------------------------------------------------------ words as packed FP32 pairs
using ff::add2;
using ff::both;
using ff::fma2;
using ff::halves;
using ff::mul2;
using ff::pack2;

template <int KIND>
__device__ __forceinline__ void unpack(const uint4& v, uint64_t (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = ff::to_f32x2<KIND>(w[i]);
    f[i] = pack2(x.x, x.y);
  }
}
template <int KIND>
__device__ __forceinline__ uint4 pack(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = halves(f[i]);
    w[i] = ff::pack_f32<KIND>(x.x, x.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum(const uint64_t (&f)[4]) {
  const float2 s = halves(add2(add2(f[0], f[1]), add2(f[2], f[3])));
  return s.x + s.y;
}
__device__ __forceinline__ float dot(const uint64_t (&a)[4], const uint64_t (&b)[4]) {
  const float2 s = halves(fma2(a[0], b[0], fma2(a[1], b[1], fma2(a[2], b[2], mul2(a[3], b[3])))));
  return s.x + s.y;
}
// Values from `left` on become 0 (WIDE: all or none).
template <bool WIDE>
__device__ __forceinline__ void clear_from(uint64_t (&f)[4], int left) {
  if (left >= kWord) return;
  if (WIDE) left = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = halves(f[i]);
    f[i] = pack2(2 * i < left ? x.x : 0.0f, 2 * i + 1 < left ? x.y : 0.0f);
  }
}

// Which of a word's eight values stay, as bit masks; the word's first value is a multiple of 8 in its row.
struct Keep {
  uint32_t mask[kWord];

  __device__ __forceinline__ void draw(uint64_t key, uint64_t group, uint32_t dropped) {
    // A value's 16 bits, at the top of a word, are compared with whatever follows them. dropped = 65536: none stays.
    const uint32_t least = dropped << 16, ones = dropped < 65536u ? 0xffffffffu : 0u;
    const uint64_t first = key + group * kGamma;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t bits = mix64(first + i * kGamma);
      const uint32_t w[2] = {static_cast<uint32_t>(bits), static_cast<uint32_t>(bits >> 32)};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mask[4 * i + 2 * j] = (w[j] << 16) >= least ? ones : 0u;
        mask[4 * i + 2 * j + 1] = w[j] >= least ? ones : 0u;
      }
    }
  }
  // Kept values, the others 0.
  __device__ __forceinline__ void apply(uint64_t (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = halves(f[i]);
      f[i] = pack2(__uint_as_float(__float_as_uint(x.x) & mask[2 * i]), __uint_as_float(__float_as_uint(x.y) & mask[2 * i + 1]));
    }
  }
  // The same times `factor`.
  __device__ __forceinline__ void apply(uint64_t (&f)[4], float factor) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], both(factor));
    apply(f);
  }
};

// ------------------------------------------------------------------ sums over the threads of a row
// The threads that share a row: whole warps of a block that holds several such groups, each with a barrier of its
// own. Sums use two buffers in turn, so that one barrier a sum is enough: a buffer is written again only after the
// next sum's barrier, which every thread reaches after it has read.
struct Group {
  static constexpr int kMostSums = 4;
  int index, threads, rank;  // of the group in the block (the same in a warp, and shown to be); its threads; this one's
  float* room;               // 2 buffers of kMostSums floats for each of 32 warps
  uint32_t turn = 0;

  static constexpr int kRoomFloats = 2 * 32 * kMostSums;

  __device__ __forceinline__ Group(int threads_, float* rooms)
      : index(__shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / threads_, 0)), threads(threads_),
        rank(static_cast<int>(threadIdx.x) - index * threads_),
        room(rooms + (static_cast<int>(threadIdx.x) - rank) / 32 * kMostSums) {}

  __device__ __forceinline__ void barrier() const {
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
  }

  // V = 1, 2 or 4 sums, in every thread of the group and in the same order always. A lane first gives away half of
  // its sums at a step, until it holds one (of number lane % V); so four sums take 13 shuffles instead of 40.
  template <int V>
  __device__ __forceinline__ void sums(float (&v)[V]) {
    static_assert(V == 1 || V == 2 || V == 4, "sums of a lane");
    const int lane = rank & 31, warps = threads >> 5;
    float x = v[0];
    if constexpr (V == 4) {
      const bool high = lane & 2;
      const float a = high ? v[2] : v[0], b = high ? v[3] : v[1];
      v[0] = a + __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 2);
      v[1] = b + __shfl_xor_sync(0xffffffffu, high ? v[1] : v[3], 2);
    }
    if constexpr (V >= 2) {
      const bool odd = lane & 1;
      x = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
    }
#pragma unroll
    for (int d = 16; d >= V; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if (warps > 1) {
      float* buffer = room + (turn++ & 1u) * (32 * kMostSums);
      if (lane < V) buffer[(rank >> 5) * V + lane] = x;
      barrier();
      x = lane < warps * V ? buffer[lane] : 0.0f;
      for (int i = lane + 32; i < warps * V; i += 32) x += buffer[i];
#pragma unroll
      for (int d = 16; d >= V; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    }
    if constexpr (V == 1) {
      v[0] = x;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
    }
  }
};

}  // namespace row
}  // namespace t2s

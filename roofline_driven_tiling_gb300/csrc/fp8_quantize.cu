// fp8_quantize.cu -- 8-bit floating-point values with a scale for each block of 128: along rows, along
// columns (written transposed), or both from one read.
//
// A block's scale is the least power of two s with amax / s <= the type's largest value (448 = 1.75 2^8 for
// e4m3, 57344 = 1.75 2^15 for e5m2), at least 2^-126: an exponent off the bits of amax. x / s is then exact, and
// every value is rounded once. amax is taken over bit patterns, so that an infinity or NaN anywhere in a block
// makes the scale NaN and with it the whole block.
//
// Bound by memory, near enough by instructions that those were what the steps saved: 8192 x 8192 bfloat16 along rows 33 us
// (6.1 TB/s), 4096 x 8192 along rows 17.4 (5.8), columns 20.6 (4.9), both 27.8 (4.8; 4.5 rounds of three blocks to an SM),
// both with squares 25.5. FP32 values of 4096 x 8192 25.2 along rows (6.7 TB/s), both ways 39.3 (5.1; two blocks to an SM), with
// squares 36.4. Rows off 16-byte boundaries are loaded value by value: 4096 x 8191 bfloat16 29.3 along rows, both ways 50.
#include <cuda_runtime.h>

#include <cstdint>

#include "ff_device.cuh"
#include "ff_math.cuh"
#include "fp8_internal.h"

namespace t2s {
namespace fp8 {
namespace {

constexpr int kThreads = 256;

// Magnitudes are compared as the integers of their bits, and 16-bit ones two to a register (after unpacking to FP32, one by
// one, both ways over 4096 x 8192 took 34.2 us, rows 19.6).
template <int TYPE>
constexpr int kHeld = TYPE == kF32 ? 1 : 2;  // magnitudes in a register
template <int TYPE>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (TYPE == kF32) {
    return max(a, b);
  } else {
    return __vmaxs2(a, b);
  }
}
// The FP32 bits of magnitude i of a register.
template <int TYPE>
__device__ __forceinline__ uint32_t magnitude(uint32_t held, int i) {
  if constexpr (TYPE == kF32) {
    return held;
  } else if constexpr (TYPE == kBf16) {
    return i ? held & 0xffff0000u : held << 16;
  } else {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(held >> 16 * i & 0xffffu))));
  }
}
// The larger halves of a and of b.
template <int TYPE>
__device__ __forceinline__ uint32_t both_largest(uint32_t a, uint32_t b) {
  return larger<TYPE>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
}

// A block's scale and 1 / scale from the bits of its largest magnitude.
struct Scale {
  float value, inverse;
};
template <int FORMAT>
__device__ __forceinline__ Scale scale_of(uint32_t amax) {
  if (amax >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu)};
  // amax = f 2^e with 1 <= f < 2: the power is e - 8 (e5m2: e - 15), one more where f > 1.75.
  int e = static_cast<int>(amax >> 23) - (FORMAT == T2S_E4M3 ? 8 : 15) + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < 1) e = 1;
  return {__uint_as_float(static_cast<uint32_t>(e) << 23), __uint_as_float(static_cast<uint32_t>(254 - e) << 23)};
}

// Two values in 8 bits each, `lo` in the low byte.
template <int FORMAT>
__device__ __forceinline__ uint32_t pack_fp8x2(float lo, float hi) {
  uint16_t r;
  if constexpr (FORMAT == T2S_E4M3) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  } else {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  }
  return r;
}

template <int FORMAT>
__device__ __forceinline__ uint2 pack8(const uint64_t (&v)[4], float inverse) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = ff::halves(ff::mul2(v[i], ff::both(inverse)));
    w[i] = pack_fp8x2<FORMAT>(f.x, f.y);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Eight bytes of a row, fewer at its end or off 8-byte boundaries.
__device__ __forceinline__ void store8(uint8_t* p, int64_t left, bool wide, uint2 w) {
  if (wide && left >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> 8 * (i & 3));
  }
}

// The largest over a half-warp's 16 lanes, in all of them.
template <int TYPE>
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v = larger<TYPE>(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
// From maxima of a lane's rows (kHeld to a register) to the scales of the half-warp's: a lane first gives away half of its
// registers at a step, until it holds one, and only it turns that into scales, its rows' `value`s. In every lane v becomes
// the inverses, as inverse_of() reads them (powers of two and NaN, whose upper 16 bits say all).
template <int TYPE, int FORMAT, int W>
__device__ __forceinline__ void half_warp_scales(uint32_t (&v)[W], float (&value)[kHeld<TYPE>]) {
  const int lane = threadIdx.x & 31;
  uint32_t x[W];
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = v[i];
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) {
    const bool high = lane & d;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, high ? x[i] : x[i + d], d);
      x[i] = larger<TYPE>(high ? x[i + d] : x[i], other);
    }
  }
  // The lane holds register lane % W.
#pragma unroll
  for (int d = W; d <= 8; d *= 2) x[0] = larger<TYPE>(x[0], __shfl_xor_sync(0xffffffffu, x[0], d));
  uint32_t inverses = 0;
#pragma unroll
  for (int i = 0; i < kHeld<TYPE>; ++i) {
    const Scale s = scale_of<FORMAT>(magnitude<TYPE>(x[0], i));
    value[i] = s.value;
    inverses |= __float_as_uint(s.inverse) >> 16 << 16 * i;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = __shfl_sync(0xffffffffu, inverses, (lane & 16) + i);
}
__device__ __forceinline__ float inverse_of(uint32_t held, int i) {
  return __uint_as_float(i ? held & 0xffff0000u : held << 16);
}

// A thread's eight consecutive values of a row as they were read (16-bit ones take half the registers), zeros beyond its
// end. Nothing is done with them before all of a thread's loads are on their way.
template <int TYPE>
struct Eight {
  uint4 w;
  __device__ __forceinline__ void load(const void* x, int64_t at, int64_t left, bool wide) {
    const uint16_t* p = static_cast<const uint16_t*>(x) + at;
    if (wide && left >= 8) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = 2 * i < left ? p[2 * i] : 0u;
        if (2 * i + 1 < left) v[i] |= static_cast<uint32_t>(p[2 * i + 1]) << 16;
      }
      w = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  // Pairs of neighbours.
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = ff::to_f32x2<TYPE == kBf16 ? ff::kBf16 : ff::kF16>(u[i]);
      v[i] = ff::pack2(f.x, f.y);
    }
  }
  __device__ __forceinline__ void magnitudes(uint32_t (&a)[4]) const {
    a[0] = w.x & 0x7fff7fffu, a[1] = w.y & 0x7fff7fffu, a[2] = w.z & 0x7fff7fffu, a[3] = w.w & 0x7fff7fffu;
  }
};
template <>
struct Eight<kF32> {
  float f[8];
  __device__ __forceinline__ void load(const void* x, int64_t at, int64_t left, bool wide) {
    const float* p = static_cast<const float*>(x) + at;
    if (wide && left >= 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = i < left ? p[i] : 0.0f;
    }
  }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ff::pack2(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void magnitudes(uint32_t (&a)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(f[i]) & 0x7fffffffu;
  }
};

// The maxima of ROWS rows' eight values, kHeld rows to a register: magnitude<TYPE>(v[i / kHeld], i % kHeld) is row i's.
template <int TYPE, int ROWS>
__device__ __forceinline__ void row_maxima(const Eight<TYPE> (&x)[ROWS], uint32_t (&v)[ROWS / kHeld<TYPE>]) {
  constexpr int kWords = 8 / kHeld<TYPE>;
  uint32_t most[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    uint32_t a[kWords];
    x[i].magnitudes(a);
    most[i] = a[0];
#pragma unroll
    for (int j = 1; j < kWords; ++j) most[i] = larger<TYPE>(most[i], a[j]);
  }
#pragma unroll
  for (int i = 0; i < ROWS / kHeld<TYPE>; ++i) {
    if constexpr (TYPE == kF32) {
      v[i] = most[i];
    } else {
      v[i] = both_largest<TYPE>(most[2 * i], most[2 * i + 1]);
    }
  }
}

struct QuantizeParams {
  int64_t M, N, ldx;
  const void* X;
  Quantized rows, columns;
  int64_t row_tiles, column_tiles;
  int across;  // half-warps along a row
  int x_wide, rows_wide, columns_wide;
};

// Along rows: a half-warp takes a block of kAhead rows, all of them on their way at once; a CTA's 16 half-warps lie along
// a row (up to 4 KB of it) as far as it reaches, then down. (Down first, so that scales left in longer runs, the reads
// were 256 bytes of each row and 8192 x 8192 took 60 us.)
constexpr int kAhead = 4;

template <int TYPE, int FORMAT>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const __grid_constant__ QuantizeParams p) {
  ff::wait_for_earlier_kernels();
  const int half = threadIdx.x / 16, down = half / p.across;
  const int64_t tile = blockIdx.x, m0 = (tile / p.column_tiles * (16 / p.across) + down) * kAhead;
  const int64_t b = tile % p.column_tiles * p.across + (half - down * p.across), n0 = b * kBlock + threadIdx.x % 16 * 8;
  const int64_t left = p.N - n0;
  const int64_t from = m0 * p.ldx + n0;
  uint8_t* to = p.rows.q + m0 * p.rows.ld + n0;
  Eight<TYPE> x[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i].load(p.X, from + i * p.ldx, m0 + i < p.M ? left : 0, p.x_wide);
  uint32_t most[kAhead / kHeld<TYPE>];
  row_maxima<TYPE, kAhead>(x, most);
  float value[kHeld<TYPE>];
  half_warp_scales<TYPE, FORMAT>(most, value);
  const int lane = threadIdx.x % 16;
  if (lane < kAhead / kHeld<TYPE> && n0 - lane * 8 < p.N) {
#pragma unroll
    for (int i = 0; i < kHeld<TYPE>; ++i) {
      const int64_t m = m0 + lane * kHeld<TYPE> + i;
      if (m < p.M) p.rows.s.p[m * p.rows.s.row + b * p.rows.s.block] = value[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    uint64_t v[4];
    x[i].get(v);
    if (m0 + i < p.M && left > 0)
      store8(to, left, p.rows_wide, pack8<FORMAT>(v, inverse_of(most[i / kHeld<TYPE>], i % kHeld<TYPE>)));
    to += p.rows.ld;
  }
}

// Along columns, or both, or with a scale for 128 x 128: a CTA takes a tile of 128 x 128, a thread eight consecutive rows
// of eight consecutive columns. Maxima of columns go through shared memory, those of rows over a half-warp; the
// transposed values leave through shared memory too, eight bytes (a column's eight rows) at a time, so that they are
// written in rows of 128 bytes. The eight-byte words of a transposed row are stored in an order that differs from eight
// columns to the next, so that the lanes of a warp hit different banks both ways.
__device__ __forceinline__ uint32_t transposed_at(int column, int word) {
  return static_cast<uint32_t>(column * kBlock + ((word ^ (column / 8)) & 15) * 8);
}

template <int TYPE, int FORMAT, bool SQUARE>
__global__ void __launch_bounds__(kThreads, TYPE == kF32 ? 2 : 3) quantize_tile_kernel(const __grid_constant__ QuantizeParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kHeldHere = kHeld<TYPE>, kWords = 8 / kHeldHere;
  __shared__ __align__(16) uint32_t column_max[kWarps][kBlock / kHeldHere];
  __shared__ __align__(16) float column_inverse[kBlock];
  __shared__ __align__(16) uint8_t transposed[kBlock * kBlock];
  ff::wait_for_earlier_kernels();
  const int64_t tile = blockIdx.x, mb = tile % p.row_tiles, nb = tile / p.row_tiles;
  const int warp = threadIdx.x / 32, r0 = threadIdx.x / 16 * 8, c0 = threadIdx.x % 16 * 8;
  const int64_t m0 = mb * kBlock + r0, n0 = nb * kBlock + c0, left = p.N - n0;
  const bool columns = p.columns.q != nullptr;
  Eight<TYPE> x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i].load(p.X, m0 * p.ldx + n0 + i * p.ldx, m0 + i < p.M ? left : 0, p.x_wide);
  uint32_t row_max[kWords];  // eight rows too
  row_maxima<TYPE, 8>(x, row_max);
  Scale all = {};
  if (SQUARE) {
#pragma unroll
    for (int i = 1; i < kWords; ++i) row_max[0] = larger<TYPE>(row_max[0], row_max[i]);
    row_max[0] = half_warp_max<TYPE>(row_max[0]);
    if (threadIdx.x % 16 == 0) column_max[0][threadIdx.x / 16] = row_max[0];
    __syncthreads();
    uint32_t most = half_warp_max<TYPE>(column_max[0][threadIdx.x % 16]);
    if (TYPE != kF32) most = both_largest<TYPE>(most, most);
    all = scale_of<FORMAT>(magnitude<TYPE>(most, 0));
    if (threadIdx.x == 0) {
      if (p.rows.q != nullptr) p.rows.s.p[mb * p.rows.s.row + nb * p.rows.s.block] = all.value;
      if (columns) p.columns.s.p[nb * p.columns.s.row + mb * p.columns.s.block] = all.value;
    }
  } else if (columns) {
    uint32_t amax[kWords];
    x[0].magnitudes(amax);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      uint32_t a[kWords];
      x[i].magnitudes(a);
#pragma unroll
      for (int j = 0; j < kWords; ++j) amax[j] = larger<TYPE>(amax[j], a[j]);
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) amax[j] = larger<TYPE>(amax[j], __shfl_xor_sync(0xffffffffu, amax[j], 16));
    if ((threadIdx.x & 16) == 0) {
#pragma unroll
      for (int j = 0; j < kWords; j += 4)
        *reinterpret_cast<uint4*>(&column_max[warp][c0 / kHeldHere + j]) = make_uint4(amax[j], amax[j + 1], amax[j + 2], amax[j + 3]);
    }
    __syncthreads();
    if (threadIdx.x < kBlock) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) most = larger<TYPE>(most, column_max[i][threadIdx.x / kHeldHere]);
      const uint32_t a = magnitude<TYPE>(most, static_cast<int>(threadIdx.x) % kHeldHere);
      const Scale s = scale_of<FORMAT>(a);
      const int64_t n = nb * kBlock + threadIdx.x;
      column_inverse[threadIdx.x] = s.inverse;
      if (n < p.N) p.columns.s.p[n * p.columns.s.row + mb * p.columns.s.block] = s.value;
    }
    __syncthreads();
  }
  if (p.rows.q != nullptr) {
    if (!SQUARE) {
      float value[kHeldHere];
      half_warp_scales<TYPE, FORMAT>(row_max, value);
      const int lane = threadIdx.x % 16;
#pragma unroll
      for (int i = 0; i < kHeldHere; ++i) {
        const int64_t m = m0 + lane * kHeldHere + i;
        if (lane < kWords && m < p.M) p.rows.s.p[m * p.rows.s.row + nb * p.rows.s.block] = value[i];
      }
    }
    uint8_t* to = p.rows.q + m0 * p.rows.ld + n0;
#pragma unroll
    for (int i = 0; i < 8; ++i, to += p.rows.ld) {
      uint64_t v[4];
      x[i].get(v);
      if (m0 + i >= p.M) continue;
      const float inverse = SQUARE ? all.inverse : inverse_of(row_max[i / kHeldHere], i % kHeldHere);
      store8(to, left, p.rows_wide, pack8<FORMAT>(v, inverse));
    }
  }
  if (!columns) return;
  uint64_t inverse[4];
  if (SQUARE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) inverse[j] = ff::both(all.inverse);
  } else {
    const float4 lo = reinterpret_cast<const float4*>(column_inverse + c0)[0], hi = reinterpret_cast<const float4*>(column_inverse + c0)[1];
    inverse[0] = ff::pack2(lo.x, lo.y), inverse[1] = ff::pack2(lo.z, lo.w);
    inverse[2] = ff::pack2(hi.x, hi.y), inverse[3] = ff::pack2(hi.z, hi.w);
  }
  uint32_t bytes[8][2];  // a column's eight rows
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint64_t v[4], w[4];
    x[i].get(v);
    x[i + 1].get(w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = ff::halves(ff::mul2(v[j], inverse[j])), b = ff::halves(ff::mul2(w[j], inverse[j]));
      const uint32_t two[2] = {pack_fp8x2<FORMAT>(a.x, b.x), pack_fp8x2<FORMAT>(a.y, b.y)};
#pragma unroll
      for (int k = 0; k < 2; ++k) bytes[2 * j + k][i / 4] = i % 4 == 0 ? two[k] : bytes[2 * j + k][i / 4] | two[k] << 16;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint2*>(transposed + transposed_at(c0 + j, r0 / 8)) = make_uint2(bytes[j][0], bytes[j][1]);
  __syncthreads();
  // Sixteen threads to a transposed row of 128 bytes.
  const int word = threadIdx.x % 16;
  const int64_t rows_left = p.M - mb * kBlock - word * 8;
  uint8_t* to = p.columns.q + (nb * kBlock + threadIdx.x / 16) * p.columns.ld + mb * kBlock + word * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i, to += 16 * p.columns.ld) {
    const int c = threadIdx.x / 16 + 16 * i;
    if (nb * kBlock + c < p.N)
      store8(to, rows_left, p.columns_wide,
             *reinterpret_cast<const uint2*>(transposed + transposed_at(c, word)));
  }
}

template <int TYPE, int FORMAT>
cudaError_t launch(const QuantizeTask& t, cudaStream_t stream) {
  QuantizeParams p{t.M, t.N, t.ldx, t.X, t.rows, t.columns};
  const int64_t ld_bytes = t.ldx * (TYPE == kF32 ? 4 : 2);
  p.x_wide = ((reinterpret_cast<uintptr_t>(t.X) | static_cast<uintptr_t>(t.M > 1 ? ld_bytes : 0)) & 15u) == 0;
  p.rows_wide = ((reinterpret_cast<uintptr_t>(t.rows.q) | static_cast<uintptr_t>(t.rows.ld)) & 7u) == 0;
  p.columns_wide = ((reinterpret_cast<uintptr_t>(t.columns.q) | static_cast<uintptr_t>(t.columns.ld)) & 7u) == 0;
  const bool tiles = t.square || t.columns.q != nullptr;
  p.across = 1;
  while (p.across < 16 && p.across < blocks_of(t.N)) p.across *= 2;
  const int64_t rows = tiles ? kBlock : 16 / p.across * kAhead;
  p.row_tiles = (t.M + rows - 1) / rows;
  p.column_tiles = tiles ? blocks_of(t.N) : (blocks_of(t.N) + p.across - 1) / p.across;
  if (p.row_tiles > 0x7fffffff / p.column_tiles) return cudaErrorInvalidConfiguration;
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(p.row_tiles * p.column_tiles)), kThreads, 1, 0};
  if (!tiles) return ff::launch_early(stream, shape, quantize_rows_kernel<TYPE, FORMAT>, p);
  return t.square ? ff::launch_early(stream, shape, quantize_tile_kernel<TYPE, FORMAT, true>, p)
                  : ff::launch_early(stream, shape, quantize_tile_kernel<TYPE, FORMAT, false>, p);
}

template <int TYPE>
cudaError_t launch_format(const QuantizeTask& t, cudaStream_t stream) {
  return t.format == T2S_E4M3 ? launch<TYPE, T2S_E4M3>(t, stream) : launch<TYPE, T2S_E5M2>(t, stream);
}

}  // namespace

cudaError_t run_quantize(const QuantizeTask& t, cudaStream_t stream) {
  return t.type == kF32 ? launch_format<kF32>(t, stream)
                        : t.type == kBf16 ? launch_format<kBf16>(t, stream) : launch_format<kF16>(t, stream);
}

}  // namespace fp8
}  // namespace t2s

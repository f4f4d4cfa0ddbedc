// norm_device.cuh -- reductions, words and launch shapes shared by the norm and dropout kernels.
#pragma once

#include "drop.cuh"
#include "ff_device.cuh"
#include "ff_math.cuh"
#include "norm_internal.h"

namespace t2s {
namespace norm {

constexpr int kWord = 8;  // consecutive values of a row that a thread takes at a time: 16 bytes

template <int KIND>
__device__ __forceinline__ float at(const uint16_t* p, int64_t i, float absent) {
  return p == nullptr ? absent : ff::to_f32<KIND>(p[i]);
}

// Eight values of a row from p on, `left` of them inside the row, the others 0. `wide`: p lies on a 16-byte boundary.
__device__ __forceinline__ uint4 load_word(const uint16_t* p, int left, bool wide) {
  if (wide && left >= kWord) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 2 * i < left ? p[2 * i] : 0u;
    if (2 * i + 1 < left) w[i] |= static_cast<uint32_t>(p[2 * i + 1]) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_word(uint16_t* p, int left, bool wide, const uint4& v) {
  if (wide && left >= kWord) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < kWord; ++i)
    if (i < left) p[i] = static_cast<uint16_t>(w[i / 2] >> 16 * (i & 1));
}

template <int KIND>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kWord]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = ff::to_f32x2<KIND>(w[i]);
    f[2 * i] = x.x, f[2 * i + 1] = x.y;
  }
}

template <int KIND>
__device__ __forceinline__ uint4 pack(const float (&f)[kWord]) {
  return make_uint4(ff::pack_f32<KIND>(f[0], f[1]), ff::pack_f32<KIND>(f[2], f[3]), ff::pack_f32<KIND>(f[4], f[5]),
                    ff::pack_f32<KIND>(f[6], f[7]));
}

// Eight values of a parameter vector (`absent` where there is none).
template <int KIND>
__device__ __forceinline__ void parameter(const uint16_t* p, int64_t n, int left, bool wide, float absent,
                                          float (&f)[kWord]) {
  if (p != nullptr) {
    unpack<KIND>(load_word(p + n, left, wide), f);
  } else {
#pragma unroll
    for (int i = 0; i < kWord; ++i) f[i] = absent;
  }
}

// Drops among eight values whose first is a multiple of 8 in its row.
__device__ __forceinline__ void drop_word(const Dropout& d, uint64_t key, uint64_t group, float (&f)[kWord]) {
  const uint64_t lo = drop_bits(key, group), hi = drop_bits(key, group + 1);
#pragma unroll
  for (int i = 0; i < kWord; ++i) f[i] = drop(f[i], i < 4 ? lo : hi, i & 3, d.dropped, d.factor);
}

// Whether words of rows at p, ld values apart, can be read and written whole.
inline bool wide_rows(const void* p, int64_t ld, int64_t rows) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(rows > 1 ? ld * 2 : 0)) & 15u) == 0;
}

// Sums of V values over the block's threads, in every thread, in the same order always. `room`: 32 V floats.
template <int V>
__device__ __forceinline__ void block_sums(float (&v)[V], float* room) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  __syncthreads();  // what was last read here is done with
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) room[warp * V + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = lane < warps ? room[lane * V + i] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
}

// The threads that share a row: whole warps of a block that holds several such groups, each with a barrier of its
// own. Sums use two buffers in turn, so that one barrier a sum is enough: a buffer is written again only after the
// next sum's barrier, which every thread reaches after it has read.
struct Group {
  static constexpr int kMostSums = 4;
  int index, threads, rank;  // of the group in the block; its threads; this one among them
  float* room;               // 2 buffers of kMostSums floats for each of 32 warps
  uint32_t turn = 0;

  __device__ __forceinline__ Group(int threads_, float* rooms)
      : index(static_cast<int>(threadIdx.x) / threads_), threads(threads_),
        rank(static_cast<int>(threadIdx.x) - index * threads_),
        room(rooms + (static_cast<int>(threadIdx.x) - rank) / 32 * kMostSums) {}

  static constexpr int kRoomFloats = 2 * 32 * kMostSums;

  __device__ __forceinline__ void barrier() const {
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
  }
  template <int V>
  __device__ __forceinline__ void sums(float (&v)[V]) {
    static_assert(V <= kMostSums, "room");
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    const int warps = threads / 32, lane = rank & 31;
    if (warps == 1) return;
    float* buffer = room + (turn++ & 1u) * (32 * kMostSums);
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < V; ++i) buffer[(rank >> 5) * V + i] = v[i];
    barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lane < warps ? buffer[lane * V + i] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  }
};

}  // namespace norm
}  // namespace t2s

// norm_device.cuh -- what the norm kernels for rows of any length share.
#pragma once

#include <atomic>

#include "drop.cuh"
#include "ff_device.cuh"
#include "ff_math.cuh"
#include "norm_internal.h"
#include "row_words.cuh"

namespace t2s {
namespace norm {

template <int KIND>
__device__ __forceinline__ float at(const uint16_t* p, int64_t i, float absent) {
  return p == nullptr ? absent : ff::to_f32<KIND>(p[i]);
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

// Allows a kernel its dynamic shared memory, once on each device.
template <auto KERNEL>
cudaError_t prepare_smem(int bytes) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> prepared[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    prepared[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

}  // namespace norm
}  // namespace t2s

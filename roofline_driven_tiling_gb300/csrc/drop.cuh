// drop.cuh -- which values dropout drops, from a counter-based generator.
//
// The generator is SplitMix64 (Steele, Lea and Flood, "Fast splittable pseudorandom number generators", OOPSLA
// 2014): output i of seed s is mix(s + (i + 1) gamma). A call's key is output `sequence` of its seed, and four
// neighbouring values of a row share one output of the key, 16 bits each: value (m, n) of an M x N matrix takes
// bits 16 (n % 4) .. + 15 of output m ceil(N / 4) + n / 4. It is dropped where those are below `dropped`. So a
// value's fate depends on seed, sequence and place alone, and the mask is never stored. 16 bits a value, because
// a 64-bit output takes about 24 instructions: with 32 bits a value dropout would be bound by them, not by memory.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace t2s {

struct Dropout {
  const int64_t* seed_at = nullptr;  // device memory; nullptr: `seed`
  uint64_t seed = 0, sequence = 0;
  uint32_t dropped = 0;  // of 65536; 0: no dropout
  float factor = 1.0f;   // of the values that stay: 65536 / (65536 - dropped)
};

constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

__device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// The key of a call, plus gamma (that of output 0).
__device__ __forceinline__ uint64_t drop_key(const Dropout& d) {
  const uint64_t seed = d.seed_at != nullptr ? static_cast<uint64_t>(*d.seed_at) : d.seed;
  return mix64(seed + (d.sequence + 1) * kGamma) + kGamma;
}

// The bits of values 4 group .. 4 group + 3 counted over rows of ceil(N / 4) groups.
__device__ __forceinline__ uint64_t drop_bits(uint64_t key, uint64_t group) { return mix64(key + group * kGamma); }

// Value j of a group, or 0.
__device__ __forceinline__ float drop(float v, uint64_t bits, int j, uint32_t dropped, float factor) {
  return (static_cast<uint32_t>(bits >> (16 * j)) & 0xffffu) < dropped ? 0.0f : v * factor;
}

}  // namespace t2s

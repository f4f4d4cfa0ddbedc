// dropout.cu -- y = drop(x) + r over a matrix.
//
// Bound by memory with the generator's instructions (about 90 for a word of eight values) under the loads: 16384 x 4096 46 us
// (5.8 TB/s), with a residual 60 (6.7); 777 x 1003 with a residual, off 16-byte boundaries, 3.9 us (start-up and one round of
// blocks); 16384 x 4095 122 us, bound by putting words together and shifting them for the stores.
#include <cuda_runtime.h>

#include <cstdint>

#include "ff_device.cuh"
#include "norm_internal.h"
#include "row_words.cuh"

namespace t2s {
namespace norm {
namespace {

constexpr int kThreads = 256;

struct DropoutParams {
  row::View x, r, y;
  int64_t M, step;  // rows that all blocks take at once
  int N, across;    // threads along a row
  Dropout drop;
};

// A block takes 256 / across rows of up to `across` words each, a thread the same words of AHEAD rows at a time: so
// the place in a row is found once, and the generator's counter only moves on.
template <int KIND, bool WIDE, int AHEAD>
__global__ void __launch_bounds__(kThreads, WIDE ? 4 : 2) dropout_kernel(const __grid_constant__ DropoutParams p) {
  ff::wait_for_earlier_kernels();
  const int down = static_cast<int>(threadIdx.x) / p.across;
  const int n = (static_cast<int>(blockIdx.x) * p.across + static_cast<int>(threadIdx.x) - down * p.across) * row::kWord;
  const int left = p.N - n;
  const int64_t at_once = p.step / AHEAD;
  int64_t m = static_cast<int64_t>(blockIdx.y) * (kThreads / p.across) + down;
  const uint64_t groups = static_cast<uint64_t>((static_cast<int64_t>(p.N) + 3) / 4);
  const uint64_t key = drop_key(p.drop);
  const bool residual = p.r.p != nullptr;
  // Every lane of a warp stays for the stores' shuffles as long as one of its rows is left.
  const int64_t first_of_warp = __shfl_sync(0xffffffffu, m, 0);
  for (int64_t ahead = first_of_warp; ahead < p.M; ahead += p.step, m += p.step) {
    row::RawWord<WIDE> x[AHEAD], r[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t row = m + i * at_once;
      const int inside = row < p.M ? left : 0;
      x[i].load(p.x, p.x.p + row * p.x.ld + n, inside);
      if (residual) r[i].load(p.r, p.r.p + row * p.r.ld + n, inside);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t row = m + i * at_once;
      const int inside = row < p.M ? left : 0;
      uint64_t v[4];
      row::unpack<KIND>(x[i].get(p.x, p.x.p + row * p.x.ld + n, inside), v);
      row::Keep keep;
      keep.draw(key, static_cast<uint64_t>(row) * groups + static_cast<uint64_t>(n / 4), p.drop.dropped);
      keep.apply(v, p.drop.factor);
      if (residual) {
        uint64_t u[4];
        row::unpack<KIND>(r[i].get(p.r, p.r.p + row * p.r.ld + n, inside), u);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = row::add2(v[j], u[j]);
      }
      row::store_word<WIDE>(p.y, p.y.p + row * p.y.ld + n, inside, row::pack<KIND>(v));
    }
  }
}

template <int KIND>
cudaError_t run(const DropoutTask& t, cudaStream_t stream) {
  DropoutParams p;
  p.x = row::view_of(t.X.p, t.X.ld, t.M, t.N), p.r = row::view_of(t.R.p, t.R.ld, t.M, t.N);
  p.y = row::view_of(t.Y.p, t.Y.ld, t.M, t.N);
  p.M = t.M, p.N = static_cast<int>(t.N), p.drop = t.drop;
  // Threads along a row: a block, or a power of two where rows are short (whole warps unless rows are of whole aligned words: lanes
  // that follow each other then hold words that do).
  const int64_t words = (t.N + row::kWord - 1) / row::kWord;
  const bool wide = row::whole_words(p.x, t.N) && row::whole_words(p.r, t.N) && row::whole_words(p.y, t.N);
  p.across = wide ? 1 : 32;
  while (p.across < words && p.across < kThreads) p.across *= 2;
  const int64_t columns = (words + p.across - 1) / p.across, rows = kThreads / p.across;
  // Four rows of a thread at a time, or one where that leaves SMs without a block.
  const int ahead = columns * ((t.M + rows * 4 - 1) / (rows * 4)) < 2 * 152 ? 1 : 4;
  const int64_t blocks = (t.M + rows * ahead - 1) / (rows * ahead);
  int64_t most = 152 * 8 / columns;
  if (most < 1) most = 1;
  const int64_t grid = blocks < most ? blocks : most;
  p.step = grid * rows * ahead;
  const ff::LaunchShape shape{dim3(static_cast<unsigned>(columns), static_cast<unsigned>(grid)), kThreads, 1, 0};
  if (ahead == 1)
    return wide ? ff::launch_early(stream, shape, dropout_kernel<KIND, true, 1>, p)
                : ff::launch_early(stream, shape, dropout_kernel<KIND, false, 1>, p);
  return wide ? ff::launch_early(stream, shape, dropout_kernel<KIND, true, 4>, p)
              : ff::launch_early(stream, shape, dropout_kernel<KIND, false, 4>, p);
}

}  // namespace

cudaError_t run_dropout(const DropoutTask& t, cudaStream_t stream) {
  return t.kind == ff::kBf16 ? run<ff::kBf16>(t, stream) : run<ff::kF16>(t, stream);
}

}  // namespace norm
}  // namespace t2s

// fp8_api.cu -- C entry points of the 8-bit floating-point operators: argument checks.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_internal.h"
#include "matrix_args.h"
#include "t2s_internal.h"

namespace t2s {
namespace fp8 {
namespace {

bool bad_format(int f) { return f != T2S_E4M3 && f != T2S_E5M2; }

bool bad_scales(const Scales& s, int64_t rows, int64_t blocks) {
  if (rows == 0 || blocks == 0) return false;
  return s.p == nullptr || (reinterpret_cast<uintptr_t>(s.p) & 3u) != 0 || s.row < 0 || s.block < 0 ||
         s.row > T2S_MAX_DIM || s.block > T2S_MAX_DIM;
}

// Scales that are written: no two at the same place.
bool overlapping(const Scales& s, int64_t rows, int64_t blocks) {
  if (rows <= 1 && blocks <= 1) return false;
  if (rows <= 1) return s.block < 1;
  if (blocks <= 1) return s.row < 1;
  const int64_t small = s.row < s.block ? s.row : s.block, large = s.row < s.block ? s.block : s.row;
  return small < 1 || large < small * (s.row < s.block ? rows : blocks);
}

// Rows that the tensor cores' copies read: all on 16-byte boundaries.
bool bad_operand(const void* p, int64_t ld, int64_t rows, int64_t K) {
  if (rows == 0 || K == 0) return false;
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) != 0 || ld < K || ld > T2S_MAX_DIM ||
         (rows > 1 && ld % 16 != 0);
}

int quantize(Wide type, int64_t M, int64_t N, const void* X, int64_t ldx, int format, int square, uint8_t* Q,
             int64_t ldq, float* S, int64_t s_row, int64_t s_block, uint8_t* Qt, int64_t ldqt, float* St,
             int64_t st_row, int64_t st_block, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_format(format) || (square != 0 && square != 1)) return T2S_ERR_INVALID;
  const unsigned bytes = type == kF32 ? 4 : 2;
  if (bad_arguments({{X, ldx, M, N, bytes}}, {}, {{Q, ldq, M, N, 1}, {Qt, ldqt, N, M, 1}})) return T2S_ERR_INVALID;
  QuantizeTask t{type, M, N, X, ldx, format, square != 0, {Q, ldq, {S, s_row, s_block}},
                 {Qt, ldqt, {St, st_row, st_block}}};
  if (M == 0 || N == 0) return T2S_OK;
  if (Q == nullptr && Qt == nullptr) return T2S_ERR_INVALID;
  const int64_t mb = blocks_of(M), nb = blocks_of(N);
  if (Q != nullptr && (bad_scales(t.rows.s, square ? mb : M, nb) || overlapping(t.rows.s, square ? mb : M, nb)))
    return T2S_ERR_INVALID;
  if (Qt != nullptr && (bad_scales(t.columns.s, square ? nb : N, mb) || overlapping(t.columns.s, square ? nb : N, mb)))
    return T2S_ERR_INVALID;
  const void* const scales[2] = {Q != nullptr ? S : nullptr, Qt != nullptr ? St : nullptr};
  if (scales[0] == scales[1]) return T2S_ERR_INVALID;
  for (const void* w : scales)
    if (w != nullptr && (w == X || w == Q || w == Qt)) return T2S_ERR_INVALID;
  return done(run_quantize(t, reinterpret_cast<cudaStream_t>(stream)));
}

int product(Wide type, int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, int format_a, const float* SA,
            int64_t sa_row, int64_t sa_block, const uint8_t* B, int64_t ldb, int format_b, const float* SB,
            int64_t sb_row, int64_t sb_block, int b_group, void* C, int64_t ldc, t2s_stream_t stream) {
  if (bad_size(M) || bad_size(N) || bad_size(K) || bad_format(format_a) || bad_format(format_b) ||
      (b_group != 1 && b_group != kBlock))
    return T2S_ERR_INVALID;
  if (M == 0 || N == 0) return T2S_OK;
  const unsigned bytes = type == kF32 ? 4 : 2;
  if (C == nullptr || bad_arguments({}, {{A, lda, M, K, 1}, {B, ldb, N, K, 1}}, {{C, ldc, M, N, bytes}}) ||
      bad_operand(A, lda, M, K) || bad_operand(B, ldb, N, K))
    return T2S_ERR_INVALID;
  ProductTask t{type, M, N, K, A, B, lda, ldb, format_a, format_b, {const_cast<float*>(SA), sa_row, sa_block},
                {const_cast<float*>(SB), sb_row, sb_block}, b_group, C, ldc};
  const int64_t kb = blocks_of(K);
  if (bad_scales(t.sa, M, kb) || bad_scales(t.sb, (N + b_group - 1) / b_group, kb) ||
      (kb > 0 && (C == SA || C == SB)))
    return T2S_ERR_INVALID;
  return done(run_product(t, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace fp8
}  // namespace t2s

using namespace t2s::fp8;

extern "C" {

int t2s_quantize_fp8_bf16(int64_t M, int64_t N, const uint16_t* X, int64_t ldx, int format, int square, uint8_t* Q,
                          int64_t ldq, float* S, int64_t s_row, int64_t s_block, uint8_t* Qt, int64_t ldqt, float* St,
                          int64_t st_row, int64_t st_block, t2s_stream_t stream) {
  return quantize(kBf16, M, N, X, ldx, format, square, Q, ldq, S, s_row, s_block, Qt, ldqt, St, st_row, st_block,
                  stream);
}

int t2s_quantize_fp8_f16(int64_t M, int64_t N, const uint16_t* X, int64_t ldx, int format, int square, uint8_t* Q,
                         int64_t ldq, float* S, int64_t s_row, int64_t s_block, uint8_t* Qt, int64_t ldqt, float* St,
                         int64_t st_row, int64_t st_block, t2s_stream_t stream) {
  return quantize(kF16, M, N, X, ldx, format, square, Q, ldq, S, s_row, s_block, Qt, ldqt, St, st_row, st_block,
                  stream);
}

int t2s_quantize_fp8_f32(int64_t M, int64_t N, const float* X, int64_t ldx, int format, int square, uint8_t* Q,
                         int64_t ldq, float* S, int64_t s_row, int64_t s_block, uint8_t* Qt, int64_t ldqt, float* St,
                         int64_t st_row, int64_t st_block, t2s_stream_t stream) {
  return quantize(kF32, M, N, X, ldx, format, square, Q, ldq, S, s_row, s_block, Qt, ldqt, St, st_row, st_block,
                  stream);
}

int t2s_gemm_fp8_bf16(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, int format_a, const float* SA,
                      int64_t sa_row, int64_t sa_block, const uint8_t* B, int64_t ldb, int format_b, const float* SB,
                      int64_t sb_row, int64_t sb_block, int b_group, uint16_t* C, int64_t ldc, t2s_stream_t stream) {
  return product(kBf16, M, N, K, A, lda, format_a, SA, sa_row, sa_block, B, ldb, format_b, SB, sb_row, sb_block,
                 b_group, C, ldc, stream);
}

int t2s_gemm_fp8_f16(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, int format_a, const float* SA,
                     int64_t sa_row, int64_t sa_block, const uint8_t* B, int64_t ldb, int format_b, const float* SB,
                     int64_t sb_row, int64_t sb_block, int b_group, uint16_t* C, int64_t ldc, t2s_stream_t stream) {
  return product(kF16, M, N, K, A, lda, format_a, SA, sa_row, sa_block, B, ldb, format_b, SB, sb_row, sb_block,
                 b_group, C, ldc, stream);
}

int t2s_gemm_fp8_f32(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, int format_a, const float* SA,
                     int64_t sa_row, int64_t sa_block, const uint8_t* B, int64_t ldb, int format_b, const float* SB,
                     int64_t sb_row, int64_t sb_block, int b_group, float* C, int64_t ldc, t2s_stream_t stream) {
  return product(kF32, M, N, K, A, lda, format_a, SA, sa_row, sa_block, B, ldb, format_b, SB, sb_row, sb_block,
                 b_group, C, ldc, stream);
}

}  // extern "C"

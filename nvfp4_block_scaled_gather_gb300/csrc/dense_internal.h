// Host-side launchers of the dense operators; arguments are validated by
// dense_api.cu before these are called.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "moe_dense.h"

namespace moe {

int* status_ptr();  // as in attention_internal.h

constexpr int kFp8Block = 128;      // values that share a scale
constexpr int kMaxNormDim = 16384;
constexpr int kFp8MaxK = 1 << 20;
constexpr int kFp8MaxRows = (1 << 24) - 1;
constexpr long long kFp8MaxResults = 1LL << 38;  // tiles and the scale words of one CTA are counted in 32 bits

// Bytes that the scales of a row of K values take: four scales a word.
inline long long fp8_scale_bytes(long long K) { return 4 * ((K + 511) / 512); }

// The pieces of K whose sums are added in order: a rule on K alone, so that a
// row's bits do not depend on how a launch divides its work.
inline int fp8_piece(int K) { return 512 * ((K + 4095) / 4096); }

cudaError_t launch_residual_norm(const moe_residual_norm_t& a, int* status, cudaStream_t s);

cudaError_t launch_fp8_quantize(const uint16_t* x, long long x_stride, int rows, int K, int dtype,
                                const moe_fp8_rows_t& out, cudaStream_t s);

struct Fp8Gemm {
  moe_fp8_rows_t x, w;
  int T, N, K;
  void* y;
  long long y_stride;
  int y_dtype;
  int* status;
};
cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s);
// The same of 16-bit rows x; g.x is where their 8-bit rows go, if they go anywhere.
cudaError_t launch_fp8_linear(const uint16_t* x, long long x_stride, int dtype, const Fp8Gemm& g, cudaStream_t s);

}  // namespace moe

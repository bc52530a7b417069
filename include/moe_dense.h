/*
 * moe_dense.h -- C ABI of the dense operators of libmoe_nvfp4.so: what stands
 * between the attention of moe_attention.h and the routed experts of
 * moe_nvfp4.h in a decoder block. The residual stream takes up a block's
 * output and is normed for the next one; rows are held in 8-bit floating
 * point with a scale for each 128 values; such rows are multiplied with
 * weights held the same way.
 *
 * Conventions are those of moe_nvfp4.h: device pointers owned by the caller
 * (16-byte aligned), nothing allocated, every call asynchronous on `stream`,
 * arguments checked on the host before anything is enqueued, results
 * deterministic, and a row's result independent of the other rows of its
 * call, of their number too. Tensors are bf16 or fp16 (`dtype`, MOE_BF16 or
 * MOE_FP16 of moe_attention.h), 16-bit patterns; norms' weights are fp32.
 * Outputs overlap no input and no other output unless said otherwise.
 *
 * 8-bit rows: row r of K values is e4m3 codes (E4M3FN) at codes + r *
 * row_stride and e8m0 scales (a power of two, 2^(byte - 127)) at scales + r *
 * scale_stride, one for each 128 values (the last for what is left). Value k
 * is code[k] * 2^(scale[k / 128] - 127). Quantization takes for each block the
 * smallest power of two, from 2^-127 on, with which the largest magnitude is
 * at most 448, and rounds each value over it to nearest, ties to even. An
 * infinity or NaN becomes the code for NaN (0x7F) and does not count for the
 * scale. A power of two loses nothing against other scales (codes have their
 * own exponents), divides exactly, and is what the tensor cores apply
 * themselves.
 */
#ifndef MOE_DENSE_H
#define MOE_DENSE_H

#include "moe_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_FP32 = 2 }; /* beside MOE_BF16 and MOE_FP16: products only */

/* 8-bit rows. row_stride: bytes, a multiple of 16, at least K; scale_stride:
 * bytes, a multiple of 4 (scales are 4-byte aligned), at least 4 * ceil(K / 512). Scales past the last
 * block, up to the next multiple of four, belong to the row: they are written
 * as 127 and never read as scales. */
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  long long row_stride;
  long long scale_stride;
} moe_fp8_rows_t;

/* A factor for each element: that of (token t, head h, place d) at data[t *
 * token_stride + h * head_stride + d * dim_stride], strides in elements;
 * dim_stride is 1 (data 16-byte aligned, the other strides multiples of 8) or
 * 0 (one factor for a row; any other strides, data 2-byte aligned). */
typedef struct {
  const void* data;
  long long token_stride;
  long long head_stride;
  int dim_stride;
} moe_gate_t;

/* One call of moe_residual_norm. A null data (codes) pointer leaves that part
 * out. */
typedef struct {
  int tokens, heads, dim, dtype;
  moe_heads_t x;            /* the residual stream [tokens, heads, dim] */
  moe_heads_t block;        /* a block's output, like x; null: x is only normed */
  moe_gate_t gate;          /* null: 1 */
  float residual_scale;     /* finite */
  float eps;                /* finite, > 0 */
  int post_norm;            /* 1: the block's output is normed first */
  const float* post_weight; /* [dim]; null: 1 */
  const float* pre_weight;  /* [dim]; null: 1 */
  moe_heads_t y;            /* the stream after the block (needs a block) */
  moe_heads_t normed;       /* its norm */
  moe_fp8_rows_t quantized; /* its norm as 8-bit rows (heads == 1) */
} moe_residual_norm_t;

/* For each token and head, over the dim values of its row, with norm(v) = v /
 * sqrt(mean(v^2) + eps):
 *   b      = post_norm ? norm(block) * post_weight : block
 *   y      = x + residual_scale * gate * b       (x itself without a block)
 *   normed = norm(y) * pre_weight
 * held in fp32 (squares too: a row whose squares add up to more than fp32 holds
 * has norm 0); y is rounded as it is written, normed and quantized are made of
 * the unrounded y and rounded once. At least one output. y and normed may each
 * be x or block (same address and strides: other strides at the same address
 * are MOE_ERR_INVALID), not both the same one. dim % 8 == 0, dim <= 16384,
 * tokens * heads < 2^31; for quantized heads == 1 and dim % 16 == 0 (else
 * MOE_ERR_SHAPE). */
int moe_residual_norm(const moe_residual_norm_t* args /* host */, cudaStream_t stream);

/* x [rows, K] (row r at x + r * x_stride, in elements, a multiple of 8) as
 * 8-bit rows: activations, and weights at load time. K % 16 == 0, K >= 16. */
int moe_fp8_quantize_rows(const uint16_t* x, long long x_stride, int rows, int K, int dtype,
                          const moe_fp8_rows_t* out, cudaStream_t stream);

/* y[t, n] = sum_k x[t, k] w[n, k] over dequantized values, for T rows x and N
 * rows w of K values; y [T, N] bf16, fp16 or fp32 (y_dtype), row t at y + t *
 * y_stride (elements, at least N; y aligned to its elements). The sum runs over up to eight pieces of K (512
 * ceil(K / 4096) values each), each in fp32 on the tensor cores, the pieces added in fp32 in
 * ascending order: the bits of a row of y depend on that row of x and on w
 * alone. K % 16 == 0, K <= 2^20, T and N < 2^24, T * N <= 2^38 (else MOE_ERR_SHAPE). */
int moe_fp8_gemm(const moe_fp8_rows_t* x, int T, const moe_fp8_rows_t* w, int N, int K, void* y, long long y_stride,
                 int y_dtype, cudaStream_t stream);

/* moe_fp8_quantize_rows of x [T, K], then moe_fp8_gemm: the same bits.
 * workspace: moe_fp8_linear_workspace_size(T, K) bytes, 256-byte aligned, any
 * contents; calls that share one run in stream order. (Calls of few tokens
 * quantize on the way and leave it as it is.) */
size_t moe_fp8_linear_workspace_size(int T, int K);
int moe_fp8_linear(const uint16_t* x, long long x_stride, int T, int K, int dtype, const moe_fp8_rows_t* w, int N,
                   void* y, long long y_stride, int y_dtype, void* workspace, size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DENSE_H */

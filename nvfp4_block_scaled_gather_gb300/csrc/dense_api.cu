// C ABI of the dense operators (moe_dense.h): argument checks and launches.
// The kernels live in residual_norm.cu, fp8_rows.cu and fp8_gemm.cu.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "dense_internal.h"
#include "internal.h"

namespace moe {
namespace {

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool misaligned(const void* p, int to = 16) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16; }

bool heads_ok(const moe_heads_t& h) {
  return !misaligned(h.data) && h.token_stride >= 0 && h.head_stride >= 0 && h.token_stride % 8 == 0 &&
         h.head_stride % 8 == 0;
}
// Rows that are written do not overlap.
bool out_ok(const moe_heads_t& h, int tokens, int heads, int dim) {
  if (!heads_ok(h)) return false;
  if (heads > 1 && h.head_stride < dim) return false;
  if (tokens > 1 && h.token_stride < dim) return false;
  if (tokens > 1 && heads > 1 && h.token_stride < h.head_stride * (heads - 1) + dim &&
      h.head_stride < h.token_stride * (tokens - 1) + dim)
    return false;
  return true;
}

bool gate_ok(const moe_gate_t& g) {
  if (g.token_stride < 0 || g.head_stride < 0 || (g.dim_stride != 0 && g.dim_stride != 1)) return false;
  return g.dim_stride ? !misaligned(g.data) && g.token_stride % 8 == 0 && g.head_stride % 8 == 0
                      : !misaligned(g.data, 2);
}

bool rows_ok(const moe_fp8_rows_t* r, int rows, int K) {
  return r && r->codes && r->scales && !misaligned(r->codes) && !misaligned(r->scales, 4) && r->row_stride >= 0 &&
         r->scale_stride >= 0 && r->row_stride % 16 == 0 && r->scale_stride % 4 == 0 && r->row_stride < (1LL << 40) &&
         r->scale_stride < (1LL << 40) && (rows <= 1 || (r->row_stride >= K && r->scale_stride >= fp8_scale_bytes(K)));
}

bool same(const moe_heads_t& a, const moe_heads_t& b) {
  return a.data == b.data;
}
// An output over an input has the input's rows in their places: else some would be read after they were written. (A stride
// along one element says nothing.)
bool over_ok(const moe_heads_t& out, const moe_heads_t& in, int tokens, int heads) {
  return !out.data || !same(out, in) ||
         ((tokens <= 1 || out.token_stride == in.token_stride) && (heads <= 1 || out.head_stride == in.head_stride));
}

int norm_status(const moe_residual_norm_t* a) {
  if (!a || a->tokens < 0 || a->heads <= 0 || a->dim <= 0 || !dtype_ok(a->dtype)) return MOE_ERR_INVALID;
  if (!std::isfinite(a->eps) || !(a->eps > 0) || !std::isfinite(a->residual_scale)) return MOE_ERR_INVALID;
  if (a->post_norm != 0 && a->post_norm != 1) return MOE_ERR_INVALID;
  if (a->tokens > 0 && !a->block.data && (a->post_norm || a->gate.data || a->y.data)) return MOE_ERR_INVALID;
  if (a->post_weight && !a->post_norm) return MOE_ERR_INVALID;
  if (!a->y.data && !a->normed.data && !a->quantized.codes && a->tokens > 0) return MOE_ERR_INVALID;
  if (a->dim % 8 || a->dim > kMaxNormDim || (long long)a->tokens * a->heads > 0x7fffffffLL) return MOE_ERR_SHAPE;
  if (a->quantized.codes && (a->heads != 1 || a->dim % 16)) return MOE_ERR_SHAPE;
  if (a->tokens == 0) return MOE_OK;
  if (!a->x.data || !heads_ok(a->x) || (a->block.data && !heads_ok(a->block))) return MOE_ERR_INVALID;
  if (a->gate.data && !gate_ok(a->gate)) return MOE_ERR_INVALID;
  if (misaligned(a->post_weight) || misaligned(a->pre_weight)) return MOE_ERR_INVALID;
  if ((a->y.data && !out_ok(a->y, a->tokens, a->heads, a->dim)) ||
      (a->normed.data && !out_ok(a->normed, a->tokens, a->heads, a->dim)))
    return MOE_ERR_INVALID;
  if (a->y.data && a->normed.data && same(a->y, a->normed)) return MOE_ERR_INVALID;
  for (const moe_heads_t* in : {&a->x, &a->block})
    if (!over_ok(a->y, *in, a->tokens, a->heads) || !over_ok(a->normed, *in, a->tokens, a->heads)) return MOE_ERR_INVALID;
  if (a->quantized.codes && !rows_ok(&a->quantized, a->tokens, a->dim)) return MOE_ERR_INVALID;
  return MOE_OK;
}

int k_status(int K) { return K <= 0 ? MOE_ERR_INVALID : K % 16 || K > kFp8MaxK ? MOE_ERR_SHAPE : MOE_OK; }

int quantize_status(const uint16_t* x, long long x_stride, int rows, int K, int dtype) {
  if (rows < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID;
  const int st = k_status(K);
  if (st != MOE_OK) return st;
  if (rows > kFp8MaxRows) return MOE_ERR_SHAPE;
  if (rows > 0 && (!x || misaligned(x) || x_stride < 0 || x_stride % 8)) return MOE_ERR_INVALID;
  return MOE_OK;
}

// The sides of a product that do not depend on x's form.
int product_status(int T, const moe_fp8_rows_t* w, int N, int K, const void* y, long long y_stride, int y_dtype) {
  if (T < 0 || N < 0 || (!dtype_ok(y_dtype) && y_dtype != MOE_FP32)) return MOE_ERR_INVALID;
  const int st = k_status(K);
  if (st != MOE_OK) return st;
  if (T > kFp8MaxRows || N > kFp8MaxRows || (long long)T * N > kFp8MaxResults) return MOE_ERR_SHAPE;
  if (T == 0 || N == 0) return MOE_OK;
  if (!rows_ok(w, N, K) || !y || misaligned(y, y_dtype == MOE_FP32 ? 4 : 2) || y_stride < 0 || (T > 1 && y_stride < N)) return MOE_ERR_INVALID;
  return MOE_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_residual_norm(const moe_residual_norm_t* args, cudaStream_t stream) {
  const int st = norm_status(args);
  if (st != MOE_OK || args->tokens == 0) return st;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_residual_norm(*args, word, stream));
}

int moe_fp8_quantize_rows(const uint16_t* x, long long x_stride, int rows, int K, int dtype,
                          const moe_fp8_rows_t* out, cudaStream_t stream) {
  const int st = quantize_status(x, x_stride, rows, K, dtype);
  if (st != MOE_OK || rows == 0) return st;
  if (!rows_ok(out, rows, K)) return MOE_ERR_INVALID;
  return status_of(launch_fp8_quantize(x, x_stride, rows, K, dtype, *out, stream));
}

int moe_fp8_gemm(const moe_fp8_rows_t* x, int T, const moe_fp8_rows_t* w, int N, int K, void* y, long long y_stride,
                 int y_dtype, cudaStream_t stream) {
  const int st = product_status(T, w, N, K, y, y_stride, y_dtype);
  if (st != MOE_OK || T == 0 || N == 0) return st;
  if (!rows_ok(x, T, K)) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_fp8_gemm({*x, *w, T, N, K, y, y_stride, y_dtype, word}, stream));
}

size_t moe_fp8_linear_workspace_size(int T, int K) {
  if (T < 0 || T > kFp8MaxRows || k_status(K) != MOE_OK) return 0;
  const size_t rows = T > 0 ? T : 1;
  return align256(rows * K) + align256(rows * fp8_scale_bytes(K));
}

int moe_fp8_linear(const uint16_t* x, long long x_stride, int T, int K, int dtype, const moe_fp8_rows_t* w, int N,
                   void* y, long long y_stride, int y_dtype, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int st = quantize_status(x, x_stride, T, K, dtype);
  if (st == MOE_OK) st = product_status(T, w, N, K, y, y_stride, y_dtype);
  if (st != MOE_OK || T == 0 || N == 0) return st;
  if (!workspace || misaligned(workspace, 256)) return MOE_ERR_INVALID;
  if (ws_bytes < moe_fp8_linear_workspace_size(T, K)) return MOE_ERR_WORKSPACE;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  const moe_fp8_rows_t rows = {codes, codes + align256((size_t)T * K), K, fp8_scale_bytes(K)};
  return status_of(launch_fp8_linear(x, x_stride, dtype, {rows, *w, T, N, K, y, y_stride, y_dtype, word}, stream));
}

}  // extern "C"

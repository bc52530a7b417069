// y = x w^T over 8-bit rows (moe_fp8_gemm): y[t, n] = sum_k x[t, k] w[n, k].
//
// A CTA of 256 threads makes a tile of 64 tokens x 64 rows of w, 32 values of
// K at a time from shared memory, 4 x 4 sums a thread; the sum over each piece
// of K is added to the total where the piece ends.
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float e4m3_float(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

__global__ void __launch_bounds__(256) fp8_gemm_kernel(Fp8Gemm g, int piece, int tiles_n) {
  __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
  pdl_wait();
  pdl_trigger();
  const int t0 = (int)(blockIdx.x / tiles_n) * kTile, n0 = (int)(blockIdx.x % tiles_n) * kTile;
  const int tid = threadIdx.x, r = tid / 4, c = (tid % 4) * 8;
  const int tx = tid % 16, ty = tid / 16;
  float total[4][4] = {}, sum[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kStep) {
    auto fill = [&](const moe_fp8_rows_t& m, int row, int rows, float (*s)[kTile + 1]) {
      uint2 p = make_uint2(0, 0);
      float scale = 0.0f;
      if (row < rows && k0 + c < g.K) {
        p = ld_cg(reinterpret_cast<const uint2*>(m.codes + (long long)row * m.row_stride + k0 + c));
        const uint32_t e = __ldcg(m.scales + (long long)row * m.scale_stride + (k0 + c) / kFp8Block);
        scale = e ? __uint_as_float(e << 23) : __uint_as_float(1u << 22);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s[c + j][r] = e4m3_float(((j < 4 ? p.x : p.y) >> (8 * (j & 3))) & 0xff) * scale;
    };
    fill(g.x, t0 + r, g.T, xs);
    fill(g.w, n0 + r, g.N, ws);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], sum[i][j]);
    __syncthreads();
    if ((k0 + kStep) % piece == 0 || k0 + kStep >= g.K) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          total[i][j] += sum[i][j];
          sum[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (t >= g.T || n >= g.N) continue;
      const long long at = (long long)t * g.y_stride + n;
      if (g.y_dtype == MOE_FP32)
        static_cast<float*>(g.y)[at] = total[i][j];
      else
        static_cast<uint16_t*>(g.y)[at] = (uint16_t)(g.y_dtype == MOE_BF16 ? pack16x2<MOE_BF16>(total[i][j], 0.0f)
                                                                           : pack16x2<MOE_FP16>(total[i][j], 0.0f));
    }
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s) {
  const int tn = (g.N + kTile - 1) / kTile;
  const long long tiles = (long long)tn * ((g.T + kTile - 1) / kTile);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(fp8_gemm_kernel, dim3((unsigned)tiles), dim3(256), 0, s, g, fp8_piece(g.K), tn);
}

}  // namespace moe

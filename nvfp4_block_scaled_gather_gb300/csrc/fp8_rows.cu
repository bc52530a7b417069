// Rows of bf16 or fp16 to 8-bit rows (moe_fp8_quantize_rows).
//
// A warp takes 512 values of a row, the four blocks whose scales are one word:
// lane l has values 16 l .. 16 l + 15, eight lanes a block of 128. Its largest
// magnitude goes around by shuffles; dividing by a power of two is a product.
#include <cstdint>

#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <int kType>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const uint16_t* x, long long x_stride, int rows, int K,
                                                                int words, moe_fp8_rows_t out) {
  pdl_wait();
  pdl_trigger();
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= (long long)rows * words) return;
  const int row = (int)(unit / words), word = (int)(unit - (long long)row * words);
  const int k = word * 512 + lane * 16;
  float v[16];
  if (k < K) {
    const uint4* p = reinterpret_cast<const uint4*>(x + (long long)row * x_stride + k);
    const uint4 a = ld_cg(p), b = ld_cg(p + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<kType>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_size(v[i]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  const uint32_t scale = e8m0_of(amax);
  if (k < K) {
    const float inv = e8m0_inverse(scale);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x4_of(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
    *reinterpret_cast<uint4*>(out.codes + (long long)row * out.row_stride + k) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  const uint32_t mine = (word * 512 + (lane & ~7) * 16 < K ? scale : kNoScale) << (8 * (lane >> 3));
  uint32_t all = mine;
  all |= __shfl_xor_sync(~0u, all, 8);
  all |= __shfl_xor_sync(~0u, all, 16);
  if (lane == 0) *reinterpret_cast<uint32_t*>(out.scales + (long long)row * out.scale_stride + 4 * word) = all;
}

}  // namespace

cudaError_t launch_fp8_quantize(const uint16_t* x, long long x_stride, int rows, int K, int dtype,
                                const moe_fp8_rows_t& out, cudaStream_t s) {
  const int words = (K + 511) / 512;
  const long long units = (long long)rows * words;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto* kernel = dtype == MOE_BF16 ? fp8_quantize_kernel<MOE_BF16> : fp8_quantize_kernel<MOE_FP16>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, x, x_stride, rows, K, words, out);
}

}  // namespace moe

// Rows of bf16 or fp16 to 8-bit rows (moe_fp8_quantize_rows).
//
// A warp takes 512 values of a row, the four blocks whose scales are one word:
// lane l has values 16 l .. 16 l + 15, eight lanes a block of 128. Its largest
// magnitude goes around by shuffles; dividing by a power of two is a product.
// Bound by bytes: the next word's values are on their way meanwhile (16,384 x
// 4096 33 us, 6.1 TB/s; 8192 x 4096 18.3, 5.5).
#include <cstdint>

#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "internal.h"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kCtas = 6;  // of an SM: the values on their way fit its registers

struct Values {
  uint4 a, b;  // 16 of them
};

template <int kType>
__global__ void __launch_bounds__(kThreads, kCtas) fp8_quantize_kernel(const uint16_t* x, long long x_stride, int rows,
                                                                       int K, int words, moe_fp8_rows_t out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int step = gridDim.x * (kThreads / 32), step_row = step / words, step_word = step - step_row * words;
  // this warp's row and word, and the next one's (whose values are on their way)
  int row, word;
  {
    const int first = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    row = first / words;
    word = first - row * words;
  }
  auto ask = [&](int r, int w) {
    Values v = {};
    const int k = w * 512 + lane * 16;
    if (r < rows && k < K) {
      const uint4* p = reinterpret_cast<const uint4*>(x + (long long)r * x_stride + k);
      v.a = ld_cg(p);
      v.b = ld_cg(p + 1);
    }
    return v;
  };
  Values next = ask(row, word);
  while (row < rows) {
    const Values now = next;
    const int r = row, w = word, k = w * 512 + lane * 16;
    row += step_row;
    word += step_word;
    if (word >= words) {
      word -= words;
      ++row;
    }
    next = ask(row, word);
    const uint32_t words_now[8] = {now.a.x, now.a.y, now.a.z, now.a.w, now.b.x, now.b.y, now.b.z, now.b.w};
    const uint32_t most = block_max_bits<kType, 8>(words_now);
    float amax = unpack2<kType>(most).x;
    if (__any_sync(~0u, most >= kInfinityBits<kType>)) amax = finite_block_max<kType, 8>(words_now);
    const uint32_t scale = e8m0_of(amax);
    const float inv = e8m0_inverse(scale);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x4_of<kType>(words_now[2 * i], words_now[2 * i + 1], inv);
    if (k < K)
      *reinterpret_cast<uint4*>(out.codes + (long long)r * out.row_stride + k) = make_uint4(c[0], c[1], c[2], c[3]);
    uint32_t all = (w * 512 + (lane & ~7) * 16 < K ? scale : kNoScale) << (8 * (lane >> 3));
    all |= __shfl_xor_sync(~0u, all, 8);
    all |= __shfl_xor_sync(~0u, all, 16);
    if (lane == 0) *reinterpret_cast<uint32_t*>(out.scales + (long long)r * out.scale_stride + 4 * w) = all;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(const uint16_t* x, long long x_stride, int rows, int K, int dtype,
                                const moe_fp8_rows_t& out, cudaStream_t s) {
  const int words = (K + 511) / 512;
  const long long units = (long long)rows * words;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32), most = (long long)kCtas * num_sms();
  auto* kernel = dtype == MOE_BF16 ? fp8_quantize_kernel<MOE_BF16> : fp8_quantize_kernel<MOE_FP16>;
  return launch_pdl(kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, s, x, x_stride, rows, K, words, out);
}

}  // namespace moe

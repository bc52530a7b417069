// The residual stream's step between two blocks (moe_residual_norm):
//   b = norm(block) w_post,  y = x + scale gate b,  normed = norm(y) w_pre
// with norm(v) = v / sqrt(mean(v^2) + eps), in one pass: a row is read once,
// kept in registers as fp32 over both sums of squares, and written once.
#include <cstdint>

#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;  // of a CTA whose rows have 8, 16 or 32 threads each

template <int kType>
__device__ __forceinline__ void unpack8(const uint4& p, float* v) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<kType>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <int kType>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack16x2<kType>(v[0], v[1]), pack16x2<kType>(v[2], v[3]), pack16x2<kType>(v[4], v[5]),
                    pack16x2<kType>(v[6], v[7]));
}

// Sum over a row's threads: G of a warp, or all of a CTA (G == 0).
template <int G>
__device__ __forceinline__ float row_sum(float s, float* shared) {
  constexpr int width = G == 0 ? 32 : G;
#pragma unroll
  for (int o = 1; o < width; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
  if constexpr (G == 0) {
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = s;
    __syncthreads();
    s = shared[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) s += shared[w];
  }
  return s;
}

// NV groups of 8 values a thread: value 8 (i * threads + thread) + j of a row.
template <int kType, int G, int NV>
__global__ void __launch_bounds__(G == 0 ? 1024 : kRowThreads) residual_norm_kernel(moe_residual_norm_t a) {
  __shared__ float sums[2][32];
  pdl_wait();
  pdl_trigger();
  const int threads = G == 0 ? blockDim.x : G;
  const int at = G == 0 ? threadIdx.x : threadIdx.x % G;
  const long long row = G == 0 ? (long long)blockIdx.x
                               : (long long)blockIdx.x * (kRowThreads / (G == 0 ? 1 : G)) + threadIdx.x / (G == 0 ? 1 : G);
  const bool live = row < (long long)a.tokens * a.heads;
  const int t = live ? (int)(row / a.heads) : 0, h = live ? (int)(row - (long long)t * a.heads) : 0;
  const float n = (float)a.dim;
  auto place = [&](const moe_heads_t& m) {
    return static_cast<uint16_t*>(m.data) + (long long)t * m.token_stride + (long long)h * m.head_stride;
  };
  float y[NV][8], b[NV][8];
  const bool has_block = a.block.data != nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = 8 * (i * threads + at);
    uint4 px = make_uint4(0, 0, 0, 0), pb = px;
    if (live && d < a.dim) {
      px = ld_cg(reinterpret_cast<const uint4*>(place(a.x) + d));
      if (has_block) pb = ld_cg(reinterpret_cast<const uint4*>(place(a.block) + d));
    }
    unpack8<kType>(px, y[i]);
    unpack8<kType>(pb, b[i]);
  }
  if (has_block) {
    float r = 1.0f;
    if (a.post_norm) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += b[i][j] * b[i][j];
      r = 1.0f / sqrtf(row_sum<G>(s, sums[0]) / n + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int d = 8 * (i * threads + at);
      if (!live || d >= a.dim) continue;
      if (a.post_norm) {
        float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
        if (a.post_weight) {
          *reinterpret_cast<float4*>(w) = ld_cg(reinterpret_cast<const float4*>(a.post_weight + d));
          *reinterpret_cast<float4*>(w + 4) = ld_cg(reinterpret_cast<const float4*>(a.post_weight + d + 4));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * r * w[j];
      }
      if (a.gate.data) {
        const uint16_t* p = static_cast<const uint16_t*>(a.gate.data) + (long long)t * a.gate.token_stride +
                            (long long)h * a.gate.head_stride;
        float g[8];
        if (a.gate.dim_stride) {
          unpack8<kType>(ld_cg(reinterpret_cast<const uint4*>(p + d)), g);
        } else {
          const float one = unpack2<kType>(__ldcg(p)).x;
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = one;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] += a.residual_scale * b[i][j];
      if (a.y.data) *reinterpret_cast<uint4*>(place(a.y) + d) = pack8<kType>(y[i]);
    }
  }
  if (!a.normed.data && !a.quantized.codes) return;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += y[i][j] * y[i][j];
  const float r = 1.0f / sqrtf(row_sum<G>(s, sums[1]) / n + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = 8 * (i * threads + at);
    const bool mine = live && d < a.dim;
    float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
    if (mine && a.pre_weight) {
      *reinterpret_cast<float4*>(w) = ld_cg(reinterpret_cast<const float4*>(a.pre_weight + d));
      *reinterpret_cast<float4*>(w + 4) = ld_cg(reinterpret_cast<const float4*>(a.pre_weight + d + 4));
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[i][j] = y[i][j] * r * w[j];
      amax = fmaxf(amax, finite_size(y[i][j]));
    }
    if (mine && a.normed.data) *reinterpret_cast<uint4*>(place(a.normed) + d) = pack8<kType>(y[i]);
    if (a.quantized.codes) {
      // 16 threads (all of a row of 64 values at most) have a block of 128
      constexpr int width = G == 8 ? 8 : 16;
#pragma unroll
      for (int o = 1; o < width; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
      const uint32_t scale = e8m0_of(amax);
      if (mine) {
        const float inv = e8m0_inverse(scale);
        *reinterpret_cast<uint2*>(a.quantized.codes + (long long)t * a.quantized.row_stride + d) =
            make_uint2(e4m3x4_of(y[i][0], y[i][1], y[i][2], y[i][3], inv),
                       e4m3x4_of(y[i][4], y[i][5], y[i][6], y[i][7], inv));
      }
      uint8_t* scales = a.quantized.scales + (long long)t * a.quantized.scale_stride;
      if (mine && d % kFp8Block == 0) {
        scales[d / kFp8Block] = (uint8_t)scale;
        if (d + kFp8Block >= a.dim)  // the last block: the rest of its word
          for (int e = d / kFp8Block + 1; e % 4; ++e) scales[e] = (uint8_t)kNoScale;
      }
    }
  }
}

template <int kType, int G, int NV>
cudaError_t launch(const moe_residual_norm_t& a, cudaStream_t s) {
  const long long rows = (long long)a.tokens * a.heads;
  if constexpr (G > 0) {
    constexpr int per = kRowThreads / G;
    return launch_pdl(residual_norm_kernel<kType, G, NV>, dim3((unsigned)((rows + per - 1) / per)), dim3(kRowThreads), 0,
                      s, a);
  } else {
    const int threads = ((a.dim / 8 + NV - 1) / NV + 31) / 32 * 32;
    return launch_pdl(residual_norm_kernel<kType, 0, NV>, dim3((unsigned)rows), dim3((unsigned)threads), 0, s, a);
  }
}

template <int kType>
cudaError_t launch_typed(const moe_residual_norm_t& a, cudaStream_t s) {
  if (a.dim <= 64) return launch<kType, 8, 1>(a, s);
  if (a.dim <= 128) return launch<kType, 16, 1>(a, s);
  if (a.dim <= 256) return launch<kType, 32, 1>(a, s);
  if (a.dim <= 512) return launch<kType, 32, 2>(a, s);
  if (a.dim <= 8192) return launch<kType, 0, 1>(a, s);
  return launch<kType, 0, 2>(a, s);
}

}  // namespace

cudaError_t launch_residual_norm(const moe_residual_norm_t& a, cudaStream_t s) {
  return a.dtype == MOE_BF16 ? launch_typed<MOE_BF16>(a, s) : launch_typed<MOE_FP16>(a, s);
}

}  // namespace moe

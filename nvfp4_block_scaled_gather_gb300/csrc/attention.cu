// Attention over whole prompts and over a paged cache.
//
// One warp per (query token, head): online softmax over the keys that the
// query sees, in fp32, a lane holding every 32nd element of the head. This is
// the plainest form that is right for every case; it reads every key once per
// query and head, so it is bound by that re-reading.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_internal.h"
#include "internal.h"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

template <int kType>
__device__ __forceinline__ float to_f32(uint16_t bits) {
  return kType == MOE_BF16 ? __bfloat162float(__ushort_as_bfloat16(bits)) : __half2float(__ushort_as_half(bits));
}
template <int kType>
__device__ __forceinline__ uint16_t from_f32(float x) {
  return kType == MOE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ void report(int* status, int what) { atomicCAS(status, 0, what); }

template <int kType>
__global__ void __launch_bounds__(128) attention_kernel(AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(w / a.heads_q), h = (int)(w - (long long)t * a.heads_q);
  if (t >= a.total_q || t < ld_cg(a.cu_q) || t >= ld_cg(a.cu_q + a.n)) return;
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ld_cg(a.cu_q + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int first = max(ld_cg(a.cu_q + lo), 0), nq = min(ld_cg(a.cu_q + lo + 1), a.total_q) - first;
  const int i = t - first;
  if (i >= nq) return;
  const int kvh = h / (a.heads_q / a.heads_kv);
  int nk = 0, k0 = 0, seq = 0;
  if (a.paged) {
    seq = ld_cg(a.seqs + lo);
    if (seq >= 0 && seq < a.max_seqs) {
      nk = ld_cg(a.length + seq);
      if (nk < 0 || (long long)nk > (long long)a.max_pages * a.page_size) nk = 0;
    } else if (lane == 0) {
      report(a.status, MOE_ERR_INVALID);
    }
  } else {
    k0 = max(ld_cg(a.cu_k + lo), 0);
    nk = max(min(ld_cg(a.cu_k + lo + 1), a.total_k) - k0, 0);
  }
  const int context = nk - nq;  // keys before the queries' own
  constexpr int kPer = kMaxHeadDim / 32;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int d = lane + 32 * e;
    q[e] = d < a.head_dim ? to_f32<kType>(a.q.p[t * a.q.ts + h * a.q.hs + d]) * a.scale : 0.0f;
    o[e] = 0.0f;
  }
  bool seen_any = false;
  for (int j = 0; j < nk; ++j) {
    const int c = j - context;  // place among the drafted
    bool seen = c <= i;
    if (a.mask && c >= 0)
      seen = c < nq && (c >> 5) < a.mask_words && (ld_cg(a.mask + (long long)t * a.mask_words + (c >> 5)) >> (c & 31)) & 1;
    if (!seen) continue;
    long long row = k0 + j;
    if (a.paged) {
      const int p = ld_cg(a.table + (long long)seq * a.max_pages + j / a.page_size);
      if (p < 0 || p >= a.n_pages) {
        if (lane == 0) report(a.status, MOE_ERR_INVALID);
        continue;
      }
      row = (long long)p * a.page_size + j % a.page_size;
    }
    seen_any = true;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int d = lane + 32 * e;
      if (d < a.head_dim) s += q[e] * to_f32<kType>(a.k.p[row * a.k.ts + kvh * a.k.hs + d]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.0f : mn;
    const float alpha = __expf(m - base), p = __expf(s - base);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int d = lane + 32 * e;
      if (d < a.head_dim) o[e] = o[e] * alpha + p * to_f32<kType>(a.v.p[row * a.v.ts + kvh * a.v.hs + d]);
    }
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int d = lane + 32 * e;
    if (d < a.head_dim) a.out.p[t * a.out.ts + h * a.out.hs + d] = from_f32<kType>(seen_any ? o[e] / l : 0.0f);
  }
  if (a.lse && lane == 0) a.lse[(long long)t * a.heads_q + h] = seen_any ? m + __logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_attention(const AttnArgs& a, int dtype, cudaStream_t s) {
  const long long rows = (long long)a.total_q * a.heads_q;
  const dim3 grid((unsigned)((rows + 3) / 4));
  return dtype == MOE_BF16 ? launch_pdl(attention_kernel<MOE_BF16>, grid, dim3(128), 0, s, a)
                           : launch_pdl(attention_kernel<MOE_FP16>, grid, dim3(128), 0, s, a);
}

}  // namespace moe

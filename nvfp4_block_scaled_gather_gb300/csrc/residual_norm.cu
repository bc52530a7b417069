// The residual stream's step between two blocks (moe_residual_norm):
//   b = norm(block) w_post,  y = x + scale gate b,  normed = norm(y) w_pre
// with norm(v) = v / sqrt(mean(v^2) + eps), in one pass: a row is read once,
// kept in registers over both sums of squares, and written once. Bound by
// bytes (a row of 4096 moves 32 KB for 50,000 operations).
//
// A sum of squares is: eight values, a tree over the 32 threads that have 256
// values together, and a tree over those sums (for rows of more). It does not
// depend on how a launch spreads rows over threads, so a row's bits are the
// same in every call.
//
//  * Rows of at most 256: 8, 16 or 32 threads a row, several rows a thread in
//    flight (the heads of queries and keys; 3001 x 40 heads of 128: 14 us, where
//    a CTA a row took 46).
//  * Longer rows, few of them (decode): a CTA a row, eight values a thread,
//    everything asked for at once (one row of 4096 2.3 us, 152 rows 3.1: launch,
//    and one load, two sums and one store after the other).
//  * Longer rows, many of them: a CTA an SM stays, its groups of threads take row
//    after row, the next ones on their way while the present ones are worked on;
//    one copy of the norms' weights waits in shared memory (read from L2 for
//    every row they would be as many bytes again). The rows come to shared
//    memory by bulk copies: 16,384 x 4096 with both norms 84 to 90 us, 6.0 to 6.4
//    TB/s (120 with a CTA a row); to 8-bit rows 8192 x 4096 43 us, 5.4 TB/s,
//    short of issue slots.
//  * The longest, whose weights and rows would not fit shared memory, come to
//    registers.
#include <cstdint>

#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "internal.h"
#include "ldcg.cuh"
#include "mbar.cuh"
#include "pdl.cuh"
#include "row_slots.cuh"

namespace moe {
namespace {

constexpr int kSmallThreads = 256;

// What the host works out for a launch.
struct Shape {
  float inv_dim, eps;
  uint32_t magic;  // row / heads = row * magic >> shift, for rows below 2^31
  int shift;
  int* status;
};
__device__ __forceinline__ int token_of(int row, int heads, const Shape& s) {
  return heads == 1 ? row : (int)(((uint64_t)(uint32_t)row * s.magic) >> s.shift);
}

// Eight fp32 values in pairs: one instruction multiplies or adds both of a pair.
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t x) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(x));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int kType>
__device__ __forceinline__ F8 unpack8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<kType>(w[i]);
    f.p[i] = pair_of(u.x, u.y);
  }
  return f;
}
template <int kType>
__device__ __forceinline__ uint4 pack8(const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = split(f.p[i]);
    w[i] = pack16x2<kType>(u.x, u.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ F8 times(const F8& f, uint64_t by) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(f.p[i], by);
  return r;
}
__device__ __forceinline__ F8 times(const F8& f, const F8& by) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = mul2(f.p[i], by.p[i]);
  return r;
}
__device__ __forceinline__ float squares(const F8& f) {
  uint64_t s = mul2(f.p[0], f.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(f.p[i], f.p[i], s);
  const float2 u = split(s);
  return u.x + u.y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Until the row is there. Bounded: false, and the call is reported as failed, after that.
__device__ __forceinline__ bool wait_landed(uint32_t bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitCycles) {
      atomicExch(status, (int)MOE_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
template <int kWidth>
__device__ __forceinline__ float tree_sum(float s) {
#pragma unroll
  for (int o = 1; o < kWidth; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
  return s;
}

// 1 / sqrt(mean + eps) of a sum of squares (the approximate root is good to two ulps).
__device__ __forceinline__ float inverse_rms(float sum, const Shape& s) { return rsqrtf(fmaf(sum, s.inv_dim, s.eps)); }

// Where a row's eight values from d on are.
__device__ __forceinline__ uint16_t* place(const moe_heads_t& m, int t, int h, int d) {
  return static_cast<uint16_t*>(m.data) + (long long)t * m.token_stride + (long long)h * m.head_stride + d;
}
__device__ __forceinline__ uint4 load8(const moe_heads_t& m, int t, int h, int d) {
  return ld_cg(reinterpret_cast<const uint4*>(place(m, t, h, d)));
}
// The gate of eight values: as they are, or one for the row (its bits in .x).
__device__ __forceinline__ uint4 load_gate(const moe_gate_t& g, int t, int h, int d) {
  const uint16_t* p =
      static_cast<const uint16_t*>(g.data) + (long long)t * g.token_stride + (long long)h * g.head_stride;
  return g.dim_stride ? ld_cg(reinterpret_cast<const uint4*>(p + d)) : make_uint4(__ldcg(p), 0, 0, 0);
}
__device__ __forceinline__ F8 as_f8(const float4& a, const float4& b) {
  return {{pair_of(a.x, a.y), pair_of(a.z, a.w), pair_of(b.x, b.y), pair_of(b.z, b.w)}};
}
__device__ __forceinline__ F8 load_weights(const float* w, int d) {
  const float4 one = make_float4(1, 1, 1, 1);
  if (!w) return as_f8(one, one);
  return as_f8(ld_cg(reinterpret_cast<const float4*>(w + d)), ld_cg(reinterpret_cast<const float4*>(w + d + 4)));
}

// A block's values times one over their root mean square, then times the norm's weights. (In this order: with the weights, or
// a gate, first a product may pass fp32's largest value, which a factor of 0 makes NaN.)
__device__ __forceinline__ F8 norm_block(const F8& b, float r, const F8& w) { return times(times(b, pair_of(r, r)), w); }
// x + residual_scale gate b.
template <int kType>
__device__ __forceinline__ F8 add_block(const moe_residual_norm_t& a, const uint4& gate, F8 b, const uint4& x) {
  float by = a.residual_scale;
  if (a.gate.data) {
    if (a.gate.dim_stride) b = times(b, unpack8<kType>(gate));
    else by *= unpack2<kType>(gate.x).x;
  }
  const uint64_t by2 = pair_of(by, by);
  F8 y = unpack8<kType>(x);
#pragma unroll
  for (int i = 0; i < 4; ++i) y.p[i] = fma2(b.p[i], by2, y.p[i]);
  return y;
}

// normed = y r w of eight values to where it is asked for. `mine`: they are the row's. kWidth threads next to each other
// have a block of 128 (or the whole of a shorter row).
template <int kType, int kWidth>
__device__ __forceinline__ void write_normed(const moe_residual_norm_t& a, int t, int h, int d, bool mine, F8 y, float r,
                                             const F8& w) {
  y = times(times(y, pair_of(r, r)), w);
  if (mine && a.normed.data) *reinterpret_cast<uint4*>(place(a.normed, t, h, d)) = pack8<kType>(y);
  if (a.quantized.codes) {
    // (a maximum leaves NaN out; an infinity among a warp's takes it the way that leaves those out)
    float2 u[4];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = split(y.p[i]);
      most = fmaxf(most, fmaxf(fabsf(u[i].x), fabsf(u[i].y)));
    }
    if (!mine) most = 0.0f;
#pragma unroll
    for (int o = 1; o < kWidth; o <<= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
    uint32_t scale, lo, hi;
    if (!__any_sync(~0u, most == INFINITY)) {
      scale = e8m0_of(most);
      const float inv = e8m0_inverse(scale);
      const F8 v = times(y, pair_of(inv, inv));
      lo = e4m3x4(split(v.p[0]), split(v.p[1]));
      hi = e4m3x4(split(v.p[2]), split(v.p[3]));
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(finite_size(u[i].x), finite_size(u[i].y)));
      if (!mine) amax = 0.0f;
#pragma unroll
      for (int o = 1; o < kWidth; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
      scale = e8m0_of(amax);
      const float inv = e8m0_inverse(scale);
      lo = e4m3x4_of(u[0].x, u[0].y, u[1].x, u[1].y, inv);
      hi = e4m3x4_of(u[2].x, u[2].y, u[3].x, u[3].y, inv);
    }
    if (mine) {
      *reinterpret_cast<uint2*>(a.quantized.codes + (long long)t * a.quantized.row_stride + d) = make_uint2(lo, hi);
      if (d % kFp8Block == 0) {
        uint8_t* scales = a.quantized.scales + (long long)t * a.quantized.scale_stride;
        scales[d / kFp8Block] = (uint8_t)scale;
        if (d + kFp8Block >= a.dim)  // the last block: the rest of its word
          for (int e = d / kFp8Block + 1; e % 4; ++e) scales[e] = (uint8_t)kNoScale;
      }
    }
  }
}

// Rows of at most 8 G values, G threads each, kRows rows of a thread at a time. kBlock: with a block's output.
template <int kType, int G, int kRows, bool kBlock>
__global__ void __launch_bounds__(kSmallThreads, kBlock ? 4 : kRows == 4 ? 3 : 5)
    residual_norm_small(const __grid_constant__ moe_residual_norm_t a, const Shape shape) {
  pdl_wait();
  pdl_trigger();
  constexpr int kPer = kSmallThreads / G;
  const int d = 8 * (threadIdx.x % G);
  const int rows = a.tokens * a.heads, step = gridDim.x * kPer;
  const bool inside = d < a.dim;
  F8 pre = {}, post = {};
  if (inside) {
    pre = load_weights(a.pre_weight, d);
    if (kBlock && a.post_norm) post = load_weights(a.post_weight, d);
  }
  uint4 nx[kRows], nb[kRows];
  auto ask = [&](long long first) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long row = first + threadIdx.x / G + (long long)k * step;
      nx[k] = nb[k] = make_uint4(0, 0, 0, 0);
      if (inside && row < rows) {
        const int t = token_of((int)row, a.heads, shape), h = (int)row - t * a.heads;
        nx[k] = load8(a.x, t, h, d);
        if constexpr (kBlock) nb[k] = load8(a.block, t, h, d);
      }
    }
  };
  // (counted from the CTA's first row, so that all of a warp's threads go round together)
  ask((long long)blockIdx.x * kPer);
  for (long long first = (long long)blockIdx.x * kPer; first < rows; first += (long long)kRows * step) {
    uint4 x[kRows], b[kRows], g[kRows];
    int t[kRows], h[kRows];
    bool mine[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long row = first + threadIdx.x / G + (long long)k * step;
      mine[k] = inside && row < rows;
      t[k] = mine[k] ? token_of((int)row, a.heads, shape) : 0;
      h[k] = mine[k] ? (int)row - t[k] * a.heads : 0;
      g[k] = make_uint4(0, 0, 0, 0);
      if (kBlock && mine[k] && a.gate.data) g[k] = load_gate(a.gate, t[k], h[k], d);
      x[k] = nx[k];
      b[k] = nb[k];
    }
    ask(first + (long long)kRows * step);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      F8 y;
      if constexpr (kBlock) {
        F8 v = unpack8<kType>(b[k]);
        if (a.post_norm) v = norm_block(v, inverse_rms(tree_sum<G>(squares(v)), shape), post);
        y = add_block<kType>(a, g[k], v, x[k]);
        if (mine[k] && a.y.data) *reinterpret_cast<uint4*>(place(a.y, t[k], h[k], d)) = pack8<kType>(y);
      } else {
        y = unpack8<kType>(x[k]);
      }
      if (a.normed.data || a.quantized.codes) {  // (values past a row are 0)
        const float r = inverse_rms(tree_sum<G>(squares(y)), shape);
        write_normed<kType, (G < 16 ? G : 16)>(a, t[k], h[k], d, mine[k], y, r, pre);
      }
    }
  }
}

// The threads that have a row together: all of a CTA's, or a group of its warps with a barrier of its own.
struct Group {
  int threads, thread, barrier;  // barrier 0: the CTA's
};
__device__ __forceinline__ void sync(const Group& g) {
  if (g.barrier == 0) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(g.barrier), "r"(g.threads) : "memory");
}

// The sum over a row: a tree over the trees' sums of all its 256-value pieces (64 at most). `sums` is not written again
// before the call after the next one.
template <int NV>
__device__ __forceinline__ float row_sum(const Group& g, const float (&s)[NV], float* sums) {
  const int warps = g.threads >> 5, warp = g.thread >> 5, lane = threadIdx.x & 31, pieces = NV * warps;
  // NV trees in one: a lane sends half of the sums that it has and goes on with the others (lane l ends with sum l % NV)
  float part[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) part[i] = s[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int left = NV / (2 * o);  // sums of a lane after this step
    if (left >= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < left; ++i) {
        const float keep = up ? part[2 * i + 1] : part[2 * i], send = up ? part[2 * i] : part[2 * i + 1];
        part[i] = keep + __shfl_xor_sync(~0u, send, o);
      }
    } else {
      part[0] += __shfl_xor_sync(~0u, part[0], o);
    }
  }
  if (lane < NV) sums[lane * warps + warp] = part[0];
  sync(g);
  float mine = lane < pieces ? sums[lane] : 0.0f;
  if (pieces > 32 && 32 + lane < pieces) mine += sums[32 + lane];
  return tree_sum<32>(mine);
}

// Longer rows, a CTA each: eight values 8 (i * threads + thread) .. of a row, i < NV. kStay: CTAs go from row to row.
template <int kType, int NV, bool kStay>
__global__ void __launch_bounds__(kStay ? 512 : 1024)
    residual_norm_rows(const __grid_constant__ moe_residual_norm_t a, const Shape shape) {
  extern __shared__ float4 weights[];  // kStay: post (each eight values' first four, then their others), then pre
  __shared__ float sums[2][2][64];
  const int threads = blockDim.x, rows = a.tokens * a.heads;
  const Group all = {threads, (int)threadIdx.x, 0};
  const bool has_block = a.block.data != nullptr;
  auto at = [&](int i) { return 8 * (i * threads + (int)threadIdx.x); };
  pdl_wait();
  pdl_trigger();
  uint4 x[NV], b[NV], g[NV];
  auto ask = [&](int row, uint4* px, uint4* pb) {
    const int t = token_of(row, a.heads, shape), h = row - t * a.heads;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      px[i] = pb[i] = make_uint4(0, 0, 0, 0);
      if (at(i) < a.dim) {
        px[i] = load8(a.x, t, h, at(i));
        if (has_block) pb[i] = load8(a.block, t, h, at(i));
      }
    }
  };
  int row = blockIdx.x;
  ask(row, x, b);
  F8 post[kStay ? 1 : NV], pre[kStay ? 1 : NV];
  const int eights = a.dim / 8;
  if constexpr (kStay) {
    for (int d = 4 * threadIdx.x; d < a.dim; d += 4 * threads) {
      const float4 one = make_float4(1, 1, 1, 1);
      const int to = d / 8 + (d & 4 ? eights : 0);
      weights[to] = a.post_weight ? ld_cg(reinterpret_cast<const float4*>(a.post_weight + d)) : one;
      weights[2 * eights + to] = a.pre_weight ? ld_cg(reinterpret_cast<const float4*>(a.pre_weight + d)) : one;
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at(i) < a.dim) {
        post[i] = load_weights(a.post_weight, at(i));
        pre[i] = load_weights(a.pre_weight, at(i));
      } else {
        post[i] = pre[i] = {};
      }
  }
  auto held = [&](const F8* own, int i, int from) {
    if constexpr (!kStay) return own[i];
    const int e = from * eights + i * threads + threadIdx.x;
    return at(i) < a.dim ? as_f8(weights[e], weights[e + eights]) : F8{};
  };
  for (int turn = 0;; turn ^= 1) {
    const int t = token_of(row, a.heads, shape), h = row - t * a.heads;
    if (has_block && a.gate.data) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        g[i] = at(i) < a.dim ? load_gate(a.gate, t, h, at(i)) : make_uint4(0, 0, 0, 0);
    }
    uint4 nx[NV], nb[NV];
    const bool more = kStay && row + (int)gridDim.x < rows;
    if (more) ask(row + gridDim.x, nx, nb);
    F8 y[NV];
    float s[NV];
    if (has_block) {
      float r = 1.0f;
      if (a.post_norm) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = squares(unpack8<kType>(b[i]));
        r = inverse_rms(row_sum<NV>(all, s, sums[turn][0]), shape);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        F8 v = unpack8<kType>(b[i]);
        if (a.post_norm) v = norm_block(v, r, held(post, i, 0));
        y[i] = add_block<kType>(a, g[i], v, x[i]);
        if (a.y.data && at(i) < a.dim) *reinterpret_cast<uint4*>(place(a.y, t, h, at(i))) = pack8<kType>(y[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) y[i] = unpack8<kType>(x[i]);
    }
    if (a.normed.data || a.quantized.codes) {  // (values past the row are 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = squares(y[i]);
      const float r = inverse_rms(row_sum<NV>(all, s, sums[turn][1]), shape);
#pragma unroll
      for (int i = 0; i < NV; ++i) write_normed<kType, 16>(a, t, h, at(i), at(i) < a.dim, y[i], r, held(pre, i, 2));
    }
    if (!more) break;
    row += gridDim.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = nx[i];
      b[i] = nb[i];
    }
  }
}

// Rows of 257 to kMaxStreamDim, many of them: the same with the rows brought to shared memory by bulk copies, kSlots of
// them on their way or being worked on, which leaves the registers to the arithmetic. A CTA is an SM's: groups of threads
// with a row each, beside one copy of the weights.
constexpr int kSlots = 2;
constexpr int kMaxStreamDim = 14080;  // weights and slots within 225,280 bytes
constexpr int kMostGroups = 15;       // barriers 1 .. 15
template <int NV>
constexpr int kMostThreads = NV == 4 ? 512 : 1024;  // (a row's of more than 8192 values are one group)
template <int kType, int NV>
__global__ void __launch_bounds__(kMostThreads<NV>, 1)
    residual_norm_stream(const __grid_constant__ moe_residual_norm_t a, const Shape shape, const int group_threads) {
  extern __shared__ float4 weights[];  // post (each eight values' first four, then their others), pre, then the slots
  __shared__ float sums[2][2][NV * kMostThreads<NV> / 32];
  __shared__ uint64_t all_landed[kMostGroups][kSlots];
  __shared__ int all_gave_up[kMostGroups][2];  // a wait of this turn's row
  const int threads = NV == 4 ? blockDim.x : group_threads;
  const int rows = a.tokens * a.heads, eights = a.dim / 8, bytes = 2 * a.dim;
  const int group = NV == 4 ? 0 : __shfl_sync(~0u, (int)threadIdx.x / threads, 0);
  const Group own_group = {threads, (int)threadIdx.x - group * threads, NV == 4 ? 0 : group + 1};
  const int own = group * NV * (threads / 32);  // of sums
  uint64_t(&landed)[kSlots] = all_landed[group];
  volatile int* gave_up = all_gave_up[group];
  const bool has_block = a.block.data != nullptr;
  uint8_t* slots = reinterpret_cast<uint8_t*>(weights + 4 * eights) + group * kSlots * 2 * bytes;
  auto eighth = [&](int i) { return i * threads + own_group.thread; };
  // (rows go over the CTAs first)
  const long long first = blockIdx.x + (long long)group * gridDim.x;
  const long long step = (NV == 4 ? 1LL : (long long)(blockDim.x / threads)) * gridDim.x;
  if (own_group.thread == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(smem_u32(landed + i), 1);
    gave_up[0] = gave_up[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  auto bring = [&](int slot, long long row) {  // by one thread
    const int t = token_of((int)row, a.heads, shape), h = (int)row - t * a.heads;
    const uint32_t bar = smem_u32(landed + slot), to = smem_u32(slots) + (uint32_t)(slot * 2 * bytes);
    mbar_expect_tx(bar, has_block ? 2 * bytes : bytes);
    bulk_load(to, place(a.x, t, h, 0), bytes, bar);
    if (has_block) bulk_load(to + bytes, place(a.block, t, h, 0), bytes, bar);
  };
  RowSlots<kSlots> on_way(step, rows);
  if (own_group.thread == 0) on_way.start(first, bring);
  for (int d = 4 * threadIdx.x; d < a.dim; d += 4 * (int)blockDim.x) {
    const float4 one = make_float4(1, 1, 1, 1);
    const int to = d / 8 + (d & 4 ? eights : 0);
    weights[to] = a.post_weight ? ld_cg(reinterpret_cast<const float4*>(a.post_weight + d)) : one;
    weights[2 * eights + to] = a.pre_weight ? ld_cg(reinterpret_cast<const float4*>(a.pre_weight + d)) : one;
  }
  __syncthreads();
  int turn = 0;
  // (a thread behind the row's end does the last values' work again, for nobody: it has no part in sums and writes nothing)
  int e[NV];
  bool mine[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    mine[i] = eighth(i) < eights;
    e[i] = mine[i] ? eighth(i) : eights - 1;
  }
  // the gate, asked for a row ahead (16,384 x 4096, a factor for each element: 104 us, 107 where it was asked for with its
  // own row)
  uint4 g[NV];
  auto ask_gate = [&](long long row) {
    if (!has_block || !a.gate.data || row >= rows) return;
    const int t = token_of((int)row, a.heads, shape), h = (int)row - t * a.heads;
#pragma unroll
    for (int i = 0; i < NV; ++i) g[i] = load_gate(a.gate, t, h, 8 * e[i]);
  };
  ask_gate(first);
  for (long long row = first; row < rows; row += step) {
    const int t = token_of((int)row, a.heads, shape), h = (int)row - t * a.heads;
    if (!wait_landed(smem_u32(landed + on_way.slot), on_way.parity, shape.status)) gave_up[turn] = 1;
    const uint4* x = reinterpret_cast<const uint4*>(slots + on_way.slot * 2 * bytes);
    const uint4* b = x + eights;
    F8 y[NV];
    float s[NV];
    if (has_block) {
      float r = 1.0f;
      if (a.post_norm) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          y[i] = unpack8<kType>(b[e[i]]);
          s[i] = mine[i] ? squares(y[i]) : 0.0f;
        }
        r = inverse_rms(row_sum<NV>(own_group, s, sums[turn][0] + own), shape);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const F8 v = a.post_norm ? norm_block(y[i], r, as_f8(weights[e[i]], weights[e[i] + eights])) : unpack8<kType>(b[e[i]]);
        y[i] = add_block<kType>(a, g[i], v, x[e[i]]);
        if (a.y.data && mine[i]) *reinterpret_cast<uint4*>(place(a.y, t, h, 8 * e[i])) = pack8<kType>(y[i]);
      }
      ask_gate(row + step);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) y[i] = unpack8<kType>(x[e[i]]);
    }
    const bool more = a.normed.data || a.quantized.codes;
    float r = 0.0f;
    if (more) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = mine[i] ? squares(y[i]) : 0.0f;
      r = inverse_rms(row_sum<NV>(own_group, s, sums[turn][1] + own), shape);  // (everyone has read the slot)
    } else {
      sync(own_group);
    }
    // A group in which a wait gave up ends here, all of its threads alike (the next row's flag is the other one): nothing
    // more is asked for, and what is on its way is waited for.
    if (gave_up[turn]) {
      if (own_group.thread == 0)
        on_way.leave(row, [&](int slot, uint32_t parity) { wait_landed(smem_u32(landed + slot), parity, shape.status); });
      break;
    }
    if (own_group.thread == 0) on_way.again(row, bring);
    if (more) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const F8 w = as_f8(weights[2 * eights + e[i]], weights[3 * eights + e[i]]);
        write_normed<kType, 16>(a, t, h, 8 * e[i], mine[i], y[i], r, w);
      }
    }
    turn ^= 1;
    on_way.next();
  }
}

template <int kType, int G, int kRows, bool kBlock>
cudaError_t launch_small_by(int per_sm, const moe_residual_norm_t& a, const Shape& shape, cudaStream_t s) {
  constexpr int per = kSmallThreads / G * kRows;
  const long long turns = ((long long)a.tokens * a.heads + per - 1) / per, most = (long long)per_sm * num_sms();
  return launch_pdl(residual_norm_small<kType, G, kRows, kBlock>, dim3((unsigned)(turns < most ? turns : most)),
                    dim3(kSmallThreads), 0, s, a, shape);
}
// A CTA's start and end take as long as several turns of its loop, so few CTAs that stay: with a block one an SM, more for
// rows that keep each busy for twelve turns (3000 rows of 256: one an SM 5.8 us, two 6.9, three 10.4; 30,000: 23.6, 18.3 and
// 19.7; 300,000 of 128: 96, 64, 59 and with four 55). Without one, two rows of a thread at a time where all run at once
// (200 tokens of 40 heads of 128: 3.1 us, four rows 0.2 more; 64 tokens 2.0 and 2.6), else four and three CTAs an SM (3001
// tokens 14 us, two rows and five CTAs 16).
template <int kType, int G>
cudaError_t launch_small(const moe_residual_norm_t& a, const Shape& shape, cudaStream_t s) {
  const long long rows = (long long)a.tokens * a.heads;
  constexpr int per = kSmallThreads / G;
  if (a.block.data) {
    const long long busy = rows / (12LL * per * num_sms());
    return launch_small_by<kType, G, 1, true>(busy < 1 ? 1 : busy > 4 ? 4 : (int)busy, a, shape, s);
  }
  if (rows <= 4LL * per * num_sms()) return launch_small_by<kType, G, 2, false>(2, a, shape, s);
  return launch_small_by<kType, G, 4, false>(3, a, shape, s);
}

template <int kType, int NV>
cudaError_t launch_stream(const moe_residual_norm_t& a, const Shape& shape, cudaStream_t s) {
  const int threads = ((a.dim / 8 + NV - 1) / NV + 31) / 32 * 32;
  constexpr int most_smem = kMaxStreamDim * (8 + 4 * kSlots);
  const cudaError_t err = allow_smem<residual_norm_stream<kType, NV>, most_smem>();
  if (err != cudaSuccess) return err;
  const long long rows = (long long)a.tokens * a.heads, grid = rows < num_sms() ? rows : num_sms();
  long long groups = (most_smem - 8 * a.dim) / (4 * kSlots * a.dim);
  groups = groups < kMostThreads<NV> / threads ? groups : kMostThreads<NV> / threads;
  groups = groups < kMostGroups ? groups : kMostGroups;
  // Beyond what memory keeps up with, more rows at a time make reads and writes get in each other's way: two outputs of 16
  // bits take 12,288 values at a time (30,000 x 2048: five groups 77 us, six 86, eight 90; 12,000 x 5120: two 80, three 90;
  // 16,384 x 4096: two 92, three 91, four 97), with a gate, which is more to do, 15,360 (4001 x 5120, a factor for each
  // token: two 33.7, three 32.1). 8-bit outputs have fewer bytes and more to do (8192 x 4096: three groups 48 us, four 44).
  const int most = a.gate.data ? 15360 : 12288;
  if (a.normed.data && groups > 2 && groups * a.dim > most) groups = most / a.dim < 2 ? 2 : most / a.dim;
  groups = groups < (rows + grid - 1) / grid ? groups : (rows + grid - 1) / grid;
  return launch_pdl(residual_norm_stream<kType, NV>, dim3((unsigned)grid), dim3((unsigned)(groups * threads)),
                    (size_t)a.dim * (8 + 4 * kSlots * groups), s, a, shape, threads);
}

template <int kType>
cudaError_t launch_typed(const moe_residual_norm_t& a, const Shape& shape, cudaStream_t s) {
  if (a.dim <= 64) return launch_small<kType, 8>(a, shape, s);
  if (a.dim <= 128) return launch_small<kType, 16>(a, shape, s);
  if (a.dim <= 256) return launch_small<kType, 32>(a, shape, s);
  const long long rows = (long long)a.tokens * a.heads;
  const int threads = (a.dim / 8 + 31) / 32 * 32;
  // a CTA a row where all run at one time, up to four an SM (one row of 4096 2.3 us, 2.9 by groups; 304 rows 3.9 and 4.4;
  // but 400 rows 6.0 and 5.1, 180 of 7168 6.4 and 5.3, 1000 of 512 3.2 and 3.0)
  const int at_once = threads > 1024 ? 0 : threads > 256 ? 1024 / threads : 4;
  if (rows <= (long long)at_once * num_sms())
    return launch_pdl(residual_norm_rows<kType, 1, false>, dim3((unsigned)rows), dim3(threads), 0, s, a, shape);
  // (sixteen values a thread: 30,000 x 2048 78 us, 93 with eight; x 1024 44.5 and 49.7; but 50,000 x 520 62.5 and 57.4)
  if (a.dim <= 768) return launch_stream<kType, 1>(a, shape, s);
  if (a.dim <= 8192) return launch_stream<kType, 2>(a, shape, s);
  if (a.dim <= kMaxStreamDim) return launch_stream<kType, 4>(a, shape, s);
  // rows whose weights and slots would not fit shared memory
  const size_t smem = (size_t)a.dim * 8;
  const cudaError_t err = allow_smem<residual_norm_rows<kType, 4, true>, 8 * kMaxNormDim>();
  if (err != cudaSuccess) return err;
  return launch_pdl(residual_norm_rows<kType, 4, true>, dim3((unsigned)(rows < num_sms() ? rows : num_sms())),
                    dim3(((a.dim / 8 + 3) / 4 + 31) / 32 * 32), smem, s, a, shape);
}

}  // namespace

cudaError_t launch_residual_norm(const moe_residual_norm_t& a, int* status, cudaStream_t s) {
  Shape shape = {1.0f / (float)a.dim, a.eps, 0, 31, status};
  // rounded up: off by less than heads / 2^shift a row, which 2^31 rows do not add up to one
  while ((1LL << (shape.shift - 31)) < a.heads) ++shape.shift;
  shape.magic = (uint32_t)((1ULL << shape.shift) / (unsigned)a.heads + 1);
  return a.dtype == MOE_BF16 ? launch_typed<MOE_BF16>(a, shape, s) : launch_typed<MOE_FP16>(a, shape, s);
}

}  // namespace moe

// y = x w^T over 8-bit rows (moe_fp8_gemm): y[t, n] = sum_k x[t, k] w[n, k].
//
// tcgen05.mma.kind::mxf8f6f4 with the rows of w as the M side (128 a CTA) and
// tokens as the N side, so that one token costs a 16-wide product and not a
// 128-row one, and every number of tokens runs through the same code. The
// tensor cores apply the scales: a block of 128 values is four instructions
// (K = 32) with the same scale byte; a word of a row's scales, four blocks,
// lies in tensor memory, and the instruction's descriptor says which byte.
//
//  * K is cut into up to eight pieces (fp8_piece), a rule on K alone. A piece
//    is summed in tensor memory; the pieces' sums are added in fp32 in
//    ascending order. So a launch may give the pieces of a tile to the CTAs
//    of a cluster (few tiles: decode) or run them one after the other (many
//    tiles) with the same bits.
//  * Warp roles: four warps load scale words (a lane a row) and store them to
//    tensor memory, all four lane quarters alike; four warps an accumulator's
//    columns (one group, or two for wide tiles) add up pieces and write y;
//    one warp loads tiles by TMA (128-byte swizzle) into a ring; one issues
//    the MMAs, into two accumulators in turn.
//  * A cluster's CTAs send their pieces' sums to the CTA that adds a row up
//    (distributed shared memory; CTA r has 128 / split of the tile's rows).
//  * Every wait is bounded; on expiry the kernel records MOE_ERR_TIMEOUT,
//    waits for its copies and MMAs, frees tensor memory and returns.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "dense_internal.h"
#include "fp8_codec.cuh"
#include "internal.h"
#include "ldcg.cuh"
#include "mbar.cuh"
#include "pdl.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kRows = 128;         // rows of w of a CTA's tile
constexpr int kStageK = 128;       // values (bytes) of K of a stage: one scale block
constexpr int kWBytes = kRows * kStageK;
constexpr int kHeader = 1024;
constexpr int kMaxStages = 12;
constexpr int kMaxTokens = 240;    // of a tile: two accumulators and the scales fill tensor memory

// kCols: tokens of a tile at most.
template <int kCols>
struct Shape {
  static constexpr bool wide = kCols > 64;
  static constexpr int groups = wide ? 2 : 1;                  // of four warps that read accumulators
  static constexpr int acc = kCols / groups;                   // sums of a thread
  static constexpr int warps = 4 + 4 * groups + (wide ? 4 : 2);
  static constexpr int threads = 32 * warps;
  static constexpr int load_warp = 4 + 4 * groups, mma_warp = load_warp + 1;
  static constexpr int per_sm = wide ? 1 : 2;
  static constexpr int smem = wide ? 232448 : 115712;          // 227 KB; half an SM's 228 KB less 1 KB each
  static constexpr int acc_cols = kCols;                       // of one accumulator
  static constexpr int scale_bufs = wide ? 2 : 4;
  static constexpr int xs_words = (kCols + 31) / 32;           // columns that the tokens' scales take
  static constexpr int scale_cols = 16;                        // tokens' scales, then (at 8) those of w
  static constexpr int tmem = wide ? 512 : 2 * acc_cols + scale_bufs * scale_cols <= 128 ? 128 : 256;
};

struct Args {
  const uint8_t *ws, *xs;
  long long ws_stride, xs_stride;
  void* y;
  long long y_stride;
  int y_dtype;
  int T, N, K;
  int tn;                 // tokens of a tile, a multiple of 16
  int tiles_t;
  long long tiles;        // of w rows x tokens
  int split;              // CTAs of a cluster that share a tile
  int piece, pieces;      // values of K of a piece; pieces
  int stages;
  int* status;
};

// ------------------------------- PTX helpers --------------------------------
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tc_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tc_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same place in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Shared-memory descriptor, K-major operand in the 128-byte swizzle: rows of
// 128 bytes, 8-row groups 1024 bytes apart, descriptor version 1, mode 2.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor, kind::mxf8f6f4: A and B e4m3 (format 0), K-major,
// e8m0 scales, M = 128, N = n; `byte` of each scale word is used.
__device__ __forceinline__ uint32_t idesc_mxf8(int n) {
  return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_byte(uint32_t idesc, int byte) {
  return idesc | ((uint32_t)byte << 4) | ((uint32_t)byte << 29);
}

// ------------------------------- bounded waits -------------------------------
struct Ctl {
  volatile int* abort_flag;
  int* status;
};
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Ctl& c) {
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *c.abort_flag = 1;
      atomicExch(c.status, (int)MOE_ERR_TIMEOUT);
      return false;
    }
  }
}
// By one thread.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, const Ctl& c) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, c);
}
// By a whole warp, the same answer in every lane.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Ctl& c) {
  return __all_sync(~0u, wait_one(bar, parity, c));
}

__device__ __forceinline__ void store_y(const Args& a, int t, int n, float v) {
  const long long at = (long long)t * a.y_stride + n;
  if (a.y_dtype == MOE_FP32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<uint16_t*>(a.y)[at] =
        (uint16_t)(a.y_dtype == MOE_BF16 ? pack16x2<MOE_BF16>(v, 0.0f) : pack16x2<MOE_FP16>(v, 0.0f));
}

template <int kCols>
__global__ void __launch_bounds__(Shape<kCols>::threads, Shape<kCols>::per_sm)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ Args a) {
  using S = Shape<kCols>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  auto full_bar = [&](int s) { return base + 8u * s; };
  auto empty_bar = [&](int s) { return base + 8u * (kMaxStages + s); };
  auto sfull_bar = [&](int i) { return base + 8u * (2 * kMaxStages + i); };
  auto sempty_bar = [&](int i) { return base + 8u * (2 * kMaxStages + 4 + i); };
  auto afull_bar = [&](int i) { return base + 8u * (2 * kMaxStages + 8 + i); };
  auto aempty_bar = [&](int i) { return base + 8u * (2 * kMaxStages + 10 + i); };
  const uint32_t drain_bar = base + 8u * (2 * kMaxStages + 12);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  const uint32_t s_w = base + kHeader, s_x = s_w + (uint32_t)a.stages * kWBytes;
  const uint32_t x_bytes = (uint32_t)a.tn * kStageK;
  // the sums that this CTA's rows get from its cluster: [pieces][tokens][128 / split]
  const uint32_t recv_off = kHeader + (uint32_t)a.stages * (kWBytes + x_bytes);
  float* recv = reinterpret_cast<float*>(smem + recv_off);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < S::scale_bufs; ++i) {
      mbar_init(sfull_bar(i), 4);
      mbar_init(sempty_bar(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(afull_bar(i), 1);
      mbar_init(aempty_bar(i), 4 * S::groups);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == S::mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(S::tmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const long long first = blockIdx.x / a.split, step = gridDim.x / a.split;
  const int per = (a.pieces + a.split - 1) / a.split;
  const int p0 = min(a.pieces, rank * per), p1 = min(a.pieces, p0 + per);
  // blocks of 128 values of K: all of them, and this CTA's
  const int blocks = (a.K + kStageK - 1) / kStageK, per_piece = a.piece / kStageK;
  const int b0 = min(blocks, p0 * per_piece), b1 = min(blocks, p1 * per_piece);
  if (warp == S::load_warp && lane == 0) {
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&xmap);
    // the rows of w may be those that the kernel before this one writes: they are asked for in L2 only
    if (first < a.tiles)
      for (int b = b0; b < b1 && b < b0 + a.stages; ++b)
        tma_prefetch_l2(&wmap, b * kStageK, (int)(first / a.tiles_t) * kRows);
  }
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (a.split > 1) cluster_sync();  // a CTA's sums go to peers that have begun
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, a.status};
  pdl_wait();
  pdl_trigger();

  if (warp < 4) {
    // ============================ scales to tensor memory ============================
    // Lane l of each warp has rows l, 32 + l, ...: column c of its quarter takes row 32 c + l's word.
    uint32_t n = 0;
    bool ok = true;
    for (long long i = first; i < a.tiles && ok; i += step) {
      const int n0 = (int)(i / a.tiles_t) * kRows, t0 = (int)(i % a.tiles_t) * a.tn;
      for (int b = b0; b < b1 && ok; b += 4, ++n) {
        uint32_t w[4], x[S::xs_words];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = n0 + 32 * c + lane;
          w[c] = r < a.N ? ld_cg(reinterpret_cast<const uint32_t*>(a.ws + r * a.ws_stride + b)) : 0u;
        }
#pragma unroll
        for (int c = 0; c < S::xs_words; ++c) {
          const int r = t0 + 32 * c + lane;
          x[c] = 32 * c < a.tn && r < a.T ? ld_cg(reinterpret_cast<const uint32_t*>(a.xs + r * a.xs_stride + b)) : 0u;
        }
        const int buf = n % S::scale_bufs;
        ok = wait_warp(sempty_bar(buf), ((n / S::scale_bufs) & 1) ^ 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t col = tmem + ((uint32_t)(warp * 32) << 16) + 2 * S::acc_cols + buf * S::scale_cols;
        tc_st4(col + 8, w);
#pragma unroll
        for (int c = 0; c < S::xs_words; ++c) tc_st1(col + c, x[c]);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull_bar(buf));
      }
    }
  } else if (warp == S::load_warp) {
    // ================================ tiles by TMA ================================
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (long long i = first; i < a.tiles && ok; i += step) {
        const int n0 = (int)(i / a.tiles_t) * kRows, t0 = (int)(i % a.tiles_t) * a.tn;
        for (int b = b0; b < b1; ++b, ++n) {
          ok = wait_one(empty_bar(stage), phase ^ 1u, ctl);
          if (!ok) break;
          mbar_expect_tx(full_bar(stage), kWBytes + x_bytes);
          tma_load(s_w + stage * kWBytes, &wmap, b * kStageK, n0, full_bar(stage));
          tma_load(s_x + stage * x_bytes, &xmap, b * kStageK, t0, full_bar(stage));
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok || *abort_flag) {  // nothing of ours may be in flight at exit: the last loads of every stage
        const uint32_t s = (uint32_t)a.stages;
        for (uint32_t j = n > s ? n - s : 0; j < n; ++j) {
          const long long t = clock64();
          while (!mbar_try_wait(full_bar(j % s), (j / s) & 1u) && clock64() - t < kWaitCycles) {
          }
        }
      }
    }
  } else if (warp == S::mma_warp) {
    // ==================================== MMAs ====================================
    if (lane == 0) {
      const uint32_t idesc = idesc_mxf8(a.tn);
      int stage = 0;
      uint32_t phase = 0, ns = 0, na = 0;
      bool ok = true;
      for (long long i = first; i < a.tiles && ok; i += step) {
        for (int p = p0; p < p1 && ok; ++p, ++na) {
          ok = wait_one(aempty_bar(na & 1), ((na >> 1) & 1) ^ 1u, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (na & 1) * S::acc_cols;
          const int end = min(b1, (p + 1) * per_piece);
          for (int b = p * per_piece; b < end; ++b) {
            const int buf = ns % S::scale_bufs;
            if ((b & 3) == 0) {
              ok = wait_one(sfull_bar(buf), (ns / S::scale_bufs) & 1, ctl);
              if (!ok) break;
            }
            ok = wait_one(full_bar(stage), phase, ctl);
            if (!ok) break;
            tc_fence_after();
            const uint32_t col = tmem + 2 * S::acc_cols + buf * S::scale_cols;
            const uint64_t wd = desc_kmajor(s_w + stage * kWBytes), xd = desc_kmajor(s_x + stage * x_bytes);
            const uint32_t id = with_byte(idesc, b & 3);
            const int steps = min(4, (a.K - b * kStageK + 31) / 32);
            for (int j = 0; j < steps; ++j)  // 32 bytes on: 2 in a descriptor's address
              tc_mma(d, wd + 2 * j, xd + 2 * j, id, col + 8, col, b > p * per_piece || j > 0);
            tc_commit(empty_bar(stage));
            if ((b & 3) == 3 || b + 1 == end) {
              tc_commit(sempty_bar(buf));
              ++ns;
            }
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
          }
          if (ok) tc_commit(afull_bar(na & 1));
        }
      }
      if (!ok || *abort_flag) {
        tc_commit(drain_bar);
        const long long t = clock64();
        while (!mbar_try_wait(drain_bar, 0) && clock64() - t < kWaitCycles) {
        }
      }
    }
  } else if (warp < 4 + 4 * S::groups) {
    // ============================ sums of pieces, and y ============================
    const int quad = warp & 3, group = (warp - 4) >> 2;
    const int mine = a.tn / S::groups, c0 = group * mine;  // this group's columns: a multiple of 8
    const int slice = kRows / a.split, row = quad * 32 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + c0;
    uint32_t na = 0;
    bool ok = true;
    for (long long i = first; i < a.tiles && ok; i += step) {
      const int n = (int)(i / a.tiles_t) * kRows + row, t0 = (int)(i % a.tiles_t) * a.tn + c0;
      float sum[S::acc];
      for (int p = p0; p < p1; ++p, ++na) {
        ok = wait_warp(afull_bar(na & 1), (na >> 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = taddr + (na & 1) * S::acc_cols;
        const uint32_t to = a.split > 1 ? peer(base + recv_off, row / slice) + 4u * ((uint32_t)(p * a.tn) * slice + row % slice) : 0;
#pragma unroll
        for (int c = 0; c < S::acc; c += 8) {
          if (c < mine) {
            uint32_t v[8];
            tc_ld8(from + c, v);
            tc_wait_ld();
            if (a.split > 1) {
#pragma unroll
              for (int j = 0; j < 8; ++j) st_peer(to + 4u * (uint32_t)((c + j) * slice), __uint_as_float(v[j]));
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) sum[c + j] = p == p0 ? __uint_as_float(v[j]) : sum[c + j] + __uint_as_float(v[j]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(aempty_bar(na & 1));
      }
      if (ok && a.split == 1 && n < a.N) {
#pragma unroll
        for (int c = 0; c < S::acc; ++c)
          if (c < mine && t0 + c < a.T) store_y(a, t0 + c, n, sum[c]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == S::mma_warp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::tmem) : "memory");
  }
  if (a.split > 1) {
    __syncwarp();
    cluster_sync();
    if (*abort_flag) return;
    const int slice = kRows / a.split;
    const int n0 = (int)(first / a.tiles_t) * kRows + rank * slice, t0 = (int)(first % a.tiles_t) * a.tn;
    for (int i = threadIdx.x; i < slice * a.tn; i += S::threads) {
      const int n = n0 + i % slice, t = t0 + i / slice;
      if (n >= a.N || t >= a.T) continue;
      float v = recv[i];
      for (int p = 1; p < a.pieces; ++p) v += recv[p * slice * a.tn + i];
      store_y(a, t, n, v);
    }
  }
}

// 128 bytes x `rows` of 8-bit rows of K values.
bool make_map(CUtensorMap* map, const moe_fp8_rows_t& m, int rows, int K, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? m.row_stride : K)};
  const cuuint32_t box[2] = {kStageK, (cuuint32_t)box_rows};
  const cuuint32_t steps[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int kCols>
cudaError_t launch(const Fp8Gemm& g, Args a, cudaStream_t s) {
  using S = Shape<kCols>;
  const long long slots = (long long)num_sms() * S::per_sm;
  const int tiles_n = (g.N + kRows - 1) / kRows;
  a.tiles_t = (g.T + kCols - 1) / kCols;
  a.tn = ((g.T + a.tiles_t - 1) / a.tiles_t + 15) / 16 * 16;
  a.tiles_t = (g.T + a.tn - 1) / a.tn;
  a.tiles = (long long)tiles_n * a.tiles_t;
  a.split = 1;
  // a cluster's CTAs share a tile where there are too few tiles; what they send each other is held in 32 KB
  if (!S::wide)
    while (a.split < 8 && a.split < a.pieces && a.tiles * a.split * 2 <= slots) a.split *= 2;
  if (a.split > 1 && a.tn > 8 * a.split) a.split = 1;
  const int recv = a.split > 1 ? a.pieces * a.tn * (kRows / a.split) * 4 : 0;
  const int room = (S::smem - 1024 - kHeader - recv) / (kWBytes + a.tn * kStageK);
  a.stages = room < kMaxStages ? room : kMaxStages;
  CUtensorMap wmap, xmap;
  if (!make_map(&wmap, g.w, g.N, g.K, kRows) || !make_map(&xmap, g.x, g.T, g.K, a.tn)) return cudaErrorInvalidValue;
  const cudaError_t err =
      cudaFuncSetAttribute(fp8_gemm_kernel<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
  if (err != cudaSuccess) return err;
  const long long grid = a.split > 1 ? a.tiles * a.split : a.tiles < slots ? a.tiles : slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::threads);
  cfg.dynamicSmemBytes = S::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<kCols>, wmap, xmap, a);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s) {
  Args a = {};
  a.ws = g.w.scales;
  a.xs = g.x.scales;
  a.ws_stride = g.w.scale_stride;
  a.xs_stride = g.x.scale_stride;
  a.y = g.y;
  a.y_stride = g.y_stride;
  a.y_dtype = g.y_dtype;
  a.T = g.T;
  a.N = g.N;
  a.K = g.K;
  a.piece = fp8_piece(g.K);
  a.pieces = (g.K + a.piece - 1) / a.piece;
  a.status = g.status;
  if (g.T <= 16) return launch<16>(g, a, s);
  if (g.T <= 32) return launch<32>(g, a, s);
  if (g.T <= 64) return launch<64>(g, a, s);
  return launch<kMaxTokens>(g, a, s);
}

}  // namespace moe

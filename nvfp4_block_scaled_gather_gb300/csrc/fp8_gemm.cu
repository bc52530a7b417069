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
//  * Tiles: 16, 32 or 64 tokens x 128 rows of w, two CTAs an SM; or 240 tokens
//    x 256 rows, two CTAs that share each MMA (a pair), one an SM.
//  * Warp roles: one warp loads tiles by TMA (128-byte swizzle) into a ring;
//    four bring scale words to shared memory (a lane a row), and where the
//    tokens come as 16-bit rows, quantize them on the way; one issues the
//    MMAs, into two accumulators in turn, and before a word's first one the
//    copy of its scales to tensor memory; four, or eight of wide tiles, add up
//    the pieces (a lane a row of w) and write y.
//  * A cluster's CTAs send their pieces' sums to the CTA that adds a row up
//    (distributed shared memory; CTA r has 128 / split of the tile's rows).
//  * Every wait is bounded; on expiry the kernel records MOE_ERR_TIMEOUT,
//    waits for its copies and MMAs, frees tensor memory and returns.
//
// What bounds it: of many tokens the tensor cores and the power limit. Between
// stores a stage takes 965 cycles of the 960 that its MMAs need; a tile's 61 KB
// of results hold the next tile up by an eighth of that at K = 4096, and the
// clock falls (1.7 GHz with random codes, less with real ones): 8192 x 10240 x
// 4096 takes 205 to 245 us, 2800 to 3350 TFLOP/s, where a large library product
// of the same 8-bit values, without scales, takes 190 to 212 and with a scale
// for each 32 values 216 to 220. Of decode batches over many rows of w the reads
// of w (32 tokens x 100,003 x 4096: 67 us, 6.3 TB/s). Of small ones the chain
// from the launch over the first tiles, the MMAs and the joined sums to the
// store: 3.4 us for 256 x 1024, 6.8 for 5120 x 4096, one token.
#include <atomic>
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
constexpr int kBlockK = 128;       // values (bytes) of K that share a scale: a row of a swizzled tile
constexpr int kWBytes = kRows * kBlockK;
constexpr int kMaxStages = 5;
constexpr int kScaleSlots = 2;     // words of scales on their way
constexpr int kStageAtoms = 1024 + kScaleSlots * 1536;  // an atom for each stage, of tokens that are quantized here
constexpr int kHeader = 7168;
static_assert(kStageAtoms + kMaxStages * 512 <= kHeader, "");
constexpr int kMostSplit = 8;      // CTAs of a cluster, and pieces
constexpr int kMaxTokens = 240;    // of a tile: two accumulators and the scales fill tensor memory

// kCols: tokens of a tile at most. kPair: two CTAs share a tile of 256 rows of
// w, one MMA over both; each loads its own rows and half of the tokens.
template <int kCols, bool kPair>
struct Shape {
  static constexpr bool wide = kCols > 64;
  static constexpr int ctas = kPair ? 2 : 1;
  static constexpr int tile_rows = kRows * ctas;
  static constexpr int groups = wide ? 2 : 1;                  // of four warps that read accumulators
  static constexpr int acc = kCols / groups;                   // sums of a thread
  static constexpr int warps = 4 + 4 * groups + (wide ? 4 : 2);
  static constexpr int threads = 32 * warps;
  static constexpr int load_warp = 4 + 4 * groups, mma_warp = load_warp + 1;
  static constexpr int per_sm = wide ? 1 : 2;
  // blocks of 128 values of K of a stage: a stage's waits and arrivals cost the issuing warp as much as four MMAs, so
  // that with one block it could not keep the tensor cores busy (8192 x 10240 x 4096: 384 us)
  static constexpr int deep = wide ? 2 : 1;
  // A word of scales is four blocks: so many stages. The columns that a word's scales are copied to were those of the
  // word before the last one, whose MMAs have to be done: they are where the ring has come round to a word's first
  // stage, if it has no more stages than a word and one more.
  static constexpr int word_stages = 4 / deep, most_stages = word_stages + 1;
  static constexpr int asked = wide ? 32 : 16;                 // columns that are read from tensor memory together
  // registers a thread of the two warpgroups that hold sums and of the other two: 256 x 184 + 256 x 72 of the launch's 512 x 128
  static constexpr int many = wide ? 184 : 0, few = wide ? 72 : 0;
  static constexpr int smem = wide ? 232448 : 115712;          // 227 KB; half an SM's 228 KB less 1 KB each
  static constexpr int acc_cols = kCols;                       // of one accumulator
  // a word of scales of 32 rows: a column of tensor memory; 128 rows: an atom of 512 bytes in shared memory
  static constexpr int xs_words = (kCols + 31) / 32, xs_atoms = (xs_words + 3) / 4;
  static constexpr int slot_bytes = (1 + xs_atoms) * 512;      // w's atom, then the tokens'
  static constexpr int scale_cols = 16;                        // tokens' scales, then (at 8) those of w; two such
  static constexpr int tmem = wide ? 512 : 2 * acc_cols + 2 * scale_cols + 32 <= 128 ? 128 : 256;
};

struct Args {
  const uint8_t *ws, *xs;
  long long ws_stride, xs_stride;
  const uint16_t* x16;    // rows to be quantized on the way (kFrom)
  long long x16_stride;
  void* y;
  long long y_stride;
  int y_dtype;
  int pairs;              // 16-bit results of two rows of w can be written together
  int T, N, K;
  int tn;                 // tokens of a tile, a multiple of 16
  int tiles_n, tiles_t;
  int tiles;              // of w rows x tokens
  int split;              // CTAs of a cluster that share a tile
  int piece, pieces;      // values of K of a piece; pieces
  int stages;
  int* status;
};

// ------------------------------- PTX helpers --------------------------------
// (of a pair: `bar` may be the other CTA's)
template <bool kPair>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst),
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
// Arrives on the barrier (of a pair: on both CTAs') once this thread's MMAs are done.
template <bool kPair>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (tensor memory) += A B over a block of 128 values of K, or its first 32 `steps`: 32 bytes of the tiles' rows, 2 in a
// descriptor's address, each. The first step overwrites D where `accumulate` is 0.
#define MOE_MMA_BLOCK(GROUP)                                                                                          \
  if (steps == 4) {                                                                                                   \
    asm volatile(                                                                                                     \
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"                                                                \
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"                                                          \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t" \
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"                                                                 \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%5], [%6], q;\n\t" \
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"                                                                 \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%5], [%6], q;\n\t" \
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"                                                                 \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %3, [%5], [%6], q;\n\t}\n" ::"r"(d), \
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)                                       \
        : "memory");                                                                                                  \
  } else {                                                                                                            \
    for (int j = 0; j < steps; ++j, adesc += 2, bdesc += 2, accumulate = 1)                                           \
      asm volatile(                                                                                                   \
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                          \
          "tcgen05.mma.cta_group::" GROUP ".kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d), \
          "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)                                     \
          : "memory");                                                                                                \
  }
template <bool kPair>
__device__ __forceinline__ void tc_mma_block(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate, int steps) {
  if constexpr (kPair) {
    MOE_MMA_BLOCK("2")
  } else {
    MOE_MMA_BLOCK("1")
  }
}
template <bool kPair>
__device__ __forceinline__ void tc_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tc_dealloc(uint32_t tmem, uint32_t cols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// An atom of 128 rows' scale words to four columns of tensor memory, all lane quarters alike (of a pair: in both CTAs).
template <bool kPair>
__device__ __forceinline__ void tc_copy_atom(uint32_t taddr, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// This warpgroup's registers a thread, up or down from the launch's 128.
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// (without waiting for this thread's stores)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of the same place in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Four values to another CTA's shared memory, whose barrier counts their bytes. (A warp's go next to each other: with each
// lane's in a row of its own 32 tokens took 17 us instead of 10.)
__device__ __forceinline__ void send(uint32_t addr, const uint32_t* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
               : "memory");
}

// An arrival that may be on another CTA's barrier. (What it tells of is in tensor memory, or in shared memory that the
// other CTA's MMAs read through the async proxy: fences of those have come before it. With cluster scope it would wait
// for all of the warp's loads and stores.)
__device__ __forceinline__ void arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Shared-memory descriptor, K-major operand in the 128-byte swizzle: rows of
// 128 bytes, 8-row groups 1024 bytes apart, descriptor version 1, mode 2.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Descriptor of an atom of scale words: 32 rows of 16 bytes (row r: those of rows r, 32 + r, 64 + r, 96 + r), no
// swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t desc_atom(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// Instruction descriptor, kind::mxf8f6f4: A and B e4m3 (format 0), K-major,
// e8m0 scales, M = m, N = n; bytes a and b of A's and B's scale words are used.
__device__ __forceinline__ uint32_t idesc_mxf8(int m, int n) {
  return ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_bytes(uint32_t idesc, int a, int b) {
  return idesc | ((uint32_t)b << 4) | ((uint32_t)a << 29);
}

// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// ------------------------------- bounded waits -------------------------------
struct Ctl {
  volatile int* abort_flag;
  int* status;
};
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Ctl& c) {
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
// By a whole warp, which goes on where the wait gave up (the flag is up then, and no later wait waits).
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, const Ctl& c) {
  if (!mbar_try_wait(bar, parity)) wait_slow(bar, parity, c);
  __syncwarp();
}
// By a whole warp, the same answer in every lane. (Inlined: a kernel that moves registers between its warps makes no
// calls. The other CTA's arrivals need no wider scope: what they tell of is in tensor memory, ordered by tcgen05
// fences; a wait with cluster scope took 500 cycles when it had nothing to wait for.)
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Ctl& c) {
  return __all_sync(~0u, mbar_try_wait(bar, parity) || wait_slow(bar, parity, c));
}

// Tile i's place. Tiles that run at one time are eight rows of tiles of w high, so that both operands come from L2.
struct Place {
  int n, t;
};
__device__ __forceinline__ Place place_of(int i, const Args& a) {
  constexpr int kHigh = 8;
  if (a.tiles_n <= kHigh) return {i % a.tiles_n, i / a.tiles_n};
  const int full = kHigh * a.tiles_t;
  const int group = i / full, in = i - group * full;
  const int high = min(kHigh, a.tiles_n - group * kHigh), t = in / high;
  return {group * kHigh + in - t * high, t};
}

// Two sums in one instruction.
__device__ __forceinline__ void add_pair(float& a, float& b, uint32_t x, uint32_t y) {
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}\n"
      : "+f"(a), "+f"(b)
      : "r"(x), "r"(y));
}
__device__ __forceinline__ void store_y(const Args& a, int t, int n, float v) {
  const long long at = (long long)t * a.y_stride + n;
  if (a.y_dtype == MOE_FP32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<uint16_t*>(a.y)[at] =
        (uint16_t)(a.y_dtype == MOE_BF16 ? pack16x2<MOE_BF16>(v, 0.0f) : pack16x2<MOE_FP16>(v, 0.0f));
}

// The pieces' sums at `p`, `apart` from each other, in ascending order (all are asked for first).
__device__ __forceinline__ float sum_pieces(const float* p, int apart, int pieces) {
  float part[kMostSplit];
#pragma unroll
  for (int i = 0; i < kMostSplit; ++i)
    if (i < pieces) part[i] = p[i * apart];
  float v = part[0];
#pragma unroll
  for (int i = 1; i < kMostSplit; ++i)
    if (i < pieces) v += part[i];
  return v;
}

// One row of w's results for `there` tokens, a warp's lanes next to each other.
template <int kAcc, typename To, typename Round>
__device__ __forceinline__ void store_column(To* y, long long stride, const float (&sum)[kAcc], int there, Round round) {
#pragma unroll
  for (int c = 0; c < kAcc; c += 8) {
    if (c >= there) break;
    if (c + 8 <= there) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j * stride] = round(sum[c + j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < there) y[j * stride] = round(sum[c + j]);
    }
    y += 8 * stride;
  }
}
// The same for 16-bit results two rows of w at a time (N and the stride even, y 4-byte aligned): lanes 2 l and 2 l + 1
// exchange, the even one then has both rows' results for tokens 0, 2, ..., the odd one for 1, 3, ... By the whole warp;
// `in`: this lane's row is one of w's.
template <int kAcc, int kType>
__device__ __forceinline__ void store_pairs(uint16_t* y, long long stride, const float (&sum)[kAcc], int there, bool in,
                                            int lane) {
  const bool odd = lane & 1;
  y += odd ? stride - 1 : 0;
#pragma unroll
  for (int c = 0; c < kAcc; c += 8) {
    if (c >= there) break;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float mine = odd ? sum[c + j + 1] : sum[c + j];
      const float other = __shfl_xor_sync(~0u, odd ? sum[c + j] : sum[c + j + 1], 1);
      const uint32_t v = pack16x2<kType>(odd ? other : mine, odd ? mine : other);
      if (in && c + j + (odd ? 1 : 0) < there) *reinterpret_cast<uint32_t*>(y + j * stride) = v;
    }
    y += 8 * stride;
  }
}

// kFrom: what the tokens come as, 8-bit rows or (narrow tiles) a 16-bit type, MOE_BF16 or MOE_FP16: then the warps that
// bring scales quantize the tokens' values as they go.
constexpr int kFromRows = -1;
template <int kCols, bool kPair, int kFrom>
__global__ void __launch_bounds__(Shape<kCols, kPair>::threads, Shape<kCols, kPair>::per_sm)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ Args a) {
  using S = Shape<kCols, kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  auto full_bar = [&](int s) { return base + 8u * s; };
  auto empty_bar = [&](int s) { return base + 8u * (kMaxStages + s); };
  auto afull_bar = [&](int i) { return base + 8u * (2 * kMaxStages + i); };
  auto aempty_bar = [&](int i) { return base + 8u * (2 * kMaxStages + 2 + i); };
  const uint32_t drain_bar = base + 8u * (2 * kMaxStages + 4), join_bar = base + 8u * (2 * kMaxStages + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  const uint32_t s_scales = base + 1024, s_w = base + kHeader, s_x = s_w + (uint32_t)a.stages * S::deep * kWBytes;
  const uint32_t x_bytes = (uint32_t)(a.tn / S::ctas) * kBlockK;  // a block's tokens in this CTA
  // the sums that this CTA's rows get from its cluster: [pieces][tokens / 4][128 / split][4]
  const uint32_t recv_off = kHeader + (uint32_t)a.stages * S::deep * (kWBytes + x_bytes);
  float* recv = reinterpret_cast<float*>(smem + recv_off);

  // (known to be the same over a warp: tensor-core and copy instructions take their operands from uniform registers)
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full_bar(s), 1 + 4 * S::ctas);  // the tiles' bytes, and the warps that bring scales
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(afull_bar(i), 1);
      mbar_init(aempty_bar(i), 4 * S::groups * S::ctas);
    }
    mbar_init(drain_bar, 1);
    mbar_init(join_bar, 1);
    if (!kPair && a.split > 1) {
      const int t0 = place_of(blockIdx.x / a.split, a).t * a.tn;
      mbar_expect_tx(join_bar, 4 * a.pieces * (kRows / a.split) * ((min(a.tn, a.T - t0) + 3) / 4 * 4));
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == S::mma_warp) {
    tc_alloc<kPair>(smem_u32(tmem_slot), S::tmem);
    tc_fence_before();
  }
  const int ctas = kPair ? 2 : a.split;  // of a cluster
  const int rank = ctas > 1 ? (int)cluster_rank() : 0;
  const int first = blockIdx.x / ctas, step = gridDim.x / ctas;
  const int per = (a.pieces + a.split - 1) / a.split;
  const int p0 = kPair ? 0 : min(a.pieces, rank * per), p1 = kPair ? a.pieces : min(a.pieces, p0 + per);
  const int half = kPair ? rank : 0;  // which of a pair
  // blocks of 128 values of K: all of them, and this CTA's
  const int blocks = (a.K + kBlockK - 1) / kBlockK, per_piece = a.piece / kBlockK;
  const int b0 = min(blocks, p0 * per_piece), b1 = min(blocks, p1 * per_piece);
  const int b2 = b0 + (b1 - b0 + 3) / 4 * 4;  // in whole words: the last stages may be empty
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (ctas > 1) cluster_arrive();
  if (kPair) cluster_wait();  // the other CTA has begun, its barriers are set up
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const Ctl ctl{abort_flag, a.status};
  if (warp == S::load_warp) {
    if (elect_one()) {
      tma_prefetch_map(&wmap);
      if constexpr (kFrom == kFromRows) tma_prefetch_map(&xmap);
      // the rows of w may be those that the kernel before this one writes: they are asked for in L2 only
      if (first < a.tiles) {
        const int n0 = place_of(first, a).n * S::tile_rows + half * kRows;
        for (int b = b0; b < b1 && b < b0 + a.stages * S::deep; ++b) tma_prefetch_l2(&wmap, b * kBlockK, n0);
      }
    }
    __syncwarp();
  }
  pdl_wait();
  pdl_trigger();

  if (warp < 4) {
    if constexpr (S::wide) give_registers<S::few>();
    if constexpr (kFrom != kFromRows) {
      // ========================== scale words of w, and the tokens ==========================
      // (One tile a CTA.) Warp g has the scale words of w's rows 32 g .. 32 g + 31. Of the tokens thread i has, of tokens
      // i / 16, 8 on and so on, values 8 (i % 16) .. of a block: 16 threads its largest magnitude. A stage's scales are an
      // atom of their own, in the first byte. Values are asked for kAhead blocks ahead. (Kept short: with a word's four
      // blocks worked on at once, 36 KB of instructions that run once, one token took 9.6 us instead of 7.6.)
      static_assert(kCols <= 32 && S::deep == 1, "at most four tokens a thread, a block a stage");
      constexpr int kTokens = kCols / 8, kAhead = 8 / kTokens;
      struct Values {
        uint4 x[kTokens];
        uint32_t w;
      };
      const int part = threadIdx.x & 15, token = threadIdx.x >> 4;
      const Place at = place_of(min(first, a.tiles - 1), a);
      const int left = min(a.tn, a.T - at.t * a.tn);  // tokens
      const uint16_t* x0 = a.x16 + (at.t * a.tn + token) * a.x16_stride + 8 * part;
      const int n = at.n * kRows + 32 * warp + lane;
      const uint8_t* w0 = n < a.N ? a.ws + n * a.ws_stride : nullptr;
      auto ask = [&](int b, Values& v) {
        if ((b & 3) == 0) v.w = w0 && b < b1 ? ld_cg(reinterpret_cast<const uint32_t*>(w0 + b)) : 0u;
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
          v.x[u] = make_uint4(0, 0, 0, 0);
          if (token + 8 * u < left && b < b1 && b * kBlockK + 8 * part < a.K)
            v.x[u] = ld_cg(reinterpret_cast<const uint4*>(x0 + 8 * u * a.x16_stride + b * kBlockK));
        }
      };
      Values q[kAhead];
      if (first < a.tiles) {
#pragma unroll
        for (int set = 0; set < kAhead; ++set) ask(b0 + set, q[set]);
      }
      int stage = 0;
      uint32_t phase = 0;
      bool ok = first < a.tiles;
#pragma unroll 1
      for (int b = b0; b < b2 && ok; b += kAhead) {  // (b2 - b0 is a multiple of four)
#pragma unroll
        for (int two = 0; two < kAhead; two += 2) {  // two blocks' maxima at a time: their chains go side by side
          uint32_t scales[2][kTokens];
#pragma unroll
          for (int u = 0; u < kTokens; ++u) {
            if (2 * warp + 8 * u >= left) break;  // none of this warp's
            uint32_t most[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4 x = q[two + j].x[u];
              const uint32_t words[4] = {x.x, x.y, x.z, x.w};
              most[j] = block_max_bits<kFrom, 16>(words);
              scales[j][u] = e8m0_of(unpack2<kFrom>(most[j]).x);
            }
            if (__any_sync(~0u, max(most[0], most[1]) >= kInfinityBits<kFrom>)) {
#pragma unroll 1
              for (int j = 0; j < 2; ++j) {
                const uint4 x = j ? q[two + 1].x[u] : q[two].x[u];
                const uint32_t words[4] = {x.x, x.y, x.z, x.w};
                const uint32_t scale = e8m0_of(finite_block_max<kFrom, 16>(words));
                if (j) scales[1][u] = scale;
                else scales[0][u] = scale;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            Values& v = q[two + j];
            ok = ok && wait_warp(empty_bar(stage), phase ^ 1u, ctl);
            if (!ok) break;
            const int now = b + two + j;
            if ((now & 3) == 0)  // (the copies of the word before the last one, from this slot, are done as its MMAs are)
              *reinterpret_cast<uint32_t*>(smem + 1024 + ((now - b0) >> 2) % kScaleSlots * S::slot_bytes + lane * 16 +
                                           warp * 4) = v.w;
            uint8_t* atom = smem + kStageAtoms + stage * 512 + token * 16;
            // 16-byte piece c of row r at piece c ^ (r % 8); the other tokens' rows are 8 on
            uint8_t* tile = smem + (s_x - base) + stage * x_bytes + token * kBlockK + (((part >> 1) ^ token) << 4) +
                            (part & 1) * 8;
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
              if (2 * warp + 8 * u >= left) break;
              const uint4 x = v.x[u];
              const float inv = e8m0_inverse(scales[j][u]);
              if (part == 0) *reinterpret_cast<uint32_t*>(atom + u * 128) = scales[j][u];
              *reinterpret_cast<uint2*>(tile + u * 8 * kBlockK) =
                  make_uint2(e4m3x4_of<kFrom>(x.x, x.y, inv), e4m3x4_of<kFrom>(x.z, x.w, inv));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full_bar(stage));
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
            ask(now + kAhead, v);
          }
        }
      }
    } else {
      // ================================ scale words ================================
      // Group g of 32 rows is warp g % 4's: w's rows, then the tokens'. A lane has a row's word, in its place of the atom
      // that the MMA warp copies to tensor memory. (Stores from here to tensor memory wait for the MMAs that are queued.)
      // Words are asked for kAhead ahead, each set in registers of its own (moving them would wait for them).
      constexpr int kMine = (4 + S::xs_words + 3) / 4;
      struct Words {
        uint32_t v[kMine];
      };
      constexpr int kAhead = 4;
      Words q[kAhead];
      int i = b0 < b1 ? first : a.tiles, b = b0;  // of the next words to ask for
      const uint8_t* from[kMine];                 // this lane's rows' scales, or none
      auto enter = [&] {
        const Place at = place_of(i, a);
        const int n = at.n * S::tile_rows + half * kRows + 32 * warp + lane;
        from[0] = n < a.N ? a.ws + n * a.ws_stride : nullptr;
#pragma unroll
        for (int c = 1; c < kMine; ++c) {
          const int first_row = 32 * (warp + 4 * (c - 1)), t = at.t * a.tn + first_row + lane;
          from[c] = first_row < a.tn && t < a.T ? a.xs + t * a.xs_stride : nullptr;
        }
      };
      auto ask = [&](Words& r) {
        if (i >= a.tiles) return;
#pragma unroll
        for (int c = 0; c < kMine; ++c) r.v[c] = from[c] ? ld_cg(reinterpret_cast<const uint32_t*>(from[c] + b)) : 0u;
        b += 4;
        if (b >= b1) {
          b = b0;
          i += step;
          if (i < a.tiles) enter();
        }
      };
      if (i < a.tiles) enter();
#pragma unroll
      for (int u = 0; u < kAhead; ++u) ask(q[u]);
      const uint32_t mine = first < a.tiles ? (uint32_t)((a.tiles - first + step - 1) / step * ((b2 - b0) / 4)) : 0u;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (uint32_t n = 0; n < mine && ok;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u, ++n) {
          if (n >= mine) break;
          for (int j = 0; j < S::word_stages; ++j) {
            ok = wait_warp(empty_bar(stage), phase ^ 1u, ctl);
            if (!ok) break;
            if (j == 0) {
              // (the copies of the word before the last one, from this slot, are done as its MMAs are)
              uint8_t* atoms = smem + 1024 + (n % kScaleSlots) * S::slot_bytes + lane * 16 + warp * 4;
#pragma unroll
              for (int c = 0; c < kMine; ++c) *reinterpret_cast<uint32_t*>(atoms + c * 512) = q[u].v[c];
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
            if (lane == 0) {
              if constexpr (kPair) arrive_peer(peer(full_bar(stage), 0));
              else mbar_arrive(full_bar(stage));
            }
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          ask(q[u]);
        }
      }
    }
  } else if (warp >= S::load_warp) {
    if constexpr (S::wide) give_registers<S::few>();
    if (warp == S::load_warp) {
      // ================================ tiles by TMA ================================
      // (This warp and the next go through their loops whole, one lane issues: under a lane's own branch each
      // instruction would be a loop over the lanes that may be in it.)
      uint32_t n = 0;
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      for (int i = first; i < a.tiles && ok; i += step) {
        const Place at = place_of(i, a);
        const int n0 = at.n * S::tile_rows + half * kRows, t0 = at.t * a.tn + half * (a.tn / 2);
        for (int b = b0; b < b2; b += S::deep, ++n) {
          ok = wait_warp(empty_bar(stage), phase ^ 1u, ctl);
          if (!ok) break;
          if (elect_one()) {
            const int here = min(S::deep, b1 - b);  // (none: only the arrival)
            // a pair's loads are all counted by the first CTA, whose MMAs read both CTAs' stages
            const uint32_t bar = kPair ? peer(full_bar(stage), 0) : full_bar(stage);
            if (half == 0)
              mbar_expect_tx(full_bar(stage), S::ctas * max(here, 0) * (kWBytes + (kFrom == kFromRows ? x_bytes : 0)));
#pragma unroll
            for (int h = 0; h < S::deep; ++h) {
              if (h >= here) break;
              tma_load<kPair>(s_w + (stage * S::deep + h) * kWBytes, &wmap, (b + h) * kBlockK, n0, bar);
              if constexpr (kFrom == kFromRows)
                tma_load<kPair>(s_x + (stage * S::deep + h) * x_bytes, &xmap, (b + h) * kBlockK, t0, bar);
            }
          }
          __syncwarp();
          if (++stage == a.stages) { stage = 0; phase ^= 1u; }
        }
      }
      // nothing of ours may be in flight at exit: the last loads of every stage (a pair's by the first CTA, before the
      // cluster's last barrier)
      if (half == 0 && (!ok || *abort_flag)) {
        const uint32_t s = (uint32_t)a.stages;
        for (uint32_t j = n > s ? n - s : 0; j < n; ++j) {
          const long long t = clock64();
          while (!mbar_try_wait(full_bar(j % s), (j / s) & 1u) && clock64() - t < kWaitCycles) {
          }
        }
      }
    } else if (warp == S::mma_warp && half == 0) {
      // ==================================== MMAs ====================================
      const uint32_t idesc = idesc_mxf8(S::tile_rows, a.tn);
      const uint64_t w_desc = desc_kmajor(s_w), x_desc = desc_kmajor(s_x), atom_desc = desc_atom(s_scales);
      int stage = 0;
      uint32_t phase = 0, ns = 0, na = 0;
      bool ok = true;
      for (int i = first; i < a.tiles && ok; i += step) {
        for (int p = p0; p < p1 && ok; ++p, ++na) {
          ok = wait_warp(aempty_bar(na & 1), ((na >> 1) & 1) ^ 1u, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (na & 1) * S::acc_cols;
          const int begin = p * per_piece, end = min(b1, begin + per_piece), whole = begin + (end - begin + 3) / 4 * 4;
          for (int b = begin; b < whole; b += S::deep) {
            const uint32_t col = tmem + 2 * S::acc_cols + (ns & 1) * S::scale_cols;
            wait_on(full_bar(stage), phase, ctl);
            tc_fence_after();
            // the columns of the tokens' scales, w's are 8 on; of tokens quantized here a stage's own (eight by turns, more
            // than stages)
            uint32_t xcol = col;
            if constexpr (kFrom != kFromRows) xcol = tmem + 2 * S::acc_cols + 2 * S::scale_cols + (b - b0) % 8 * 4;
            if (elect_one()) {
              const uint64_t from = atom_desc + (uint64_t)((ns % kScaleSlots) * (S::slot_bytes >> 4));
              if ((b & 3) == 0) {
                tc_copy_atom<kPair>(col + 8, from);
                if constexpr (kFrom == kFromRows)
#pragma unroll
                  for (int c = 0; c < S::xs_atoms; ++c) tc_copy_atom<kPair>(col + 4 * c, from + 32 * (c + 1));
              }
              if constexpr (kFrom != kFromRows)
                tc_copy_atom<kPair>(xcol, atom_desc + (uint64_t)((kStageAtoms - 1024 + stage * 512) >> 4));
              const uint64_t wd = w_desc + (uint64_t)(stage * S::deep * (kWBytes >> 4));
              const uint64_t xd = x_desc + (uint64_t)(stage * S::deep * (x_bytes >> 4));
              const uint32_t id = with_bytes(idesc, b & 3, kFrom == kFromRows ? b & 3 : 0);
              constexpr uint32_t kNext = (1u << 29) | (1u << 4);  // both bytes on (a stage of more than one block)
              if ((b + S::deep) * kBlockK <= a.K) {
#pragma unroll
                for (int h = 0; h < S::deep; ++h)
                  tc_mma_block<kPair>(d, wd + h * (kWBytes >> 4), xd + h * (x_bytes >> 4), id + h * kNext, col + 8, xcol,
                                      b + h > begin, 4);
              } else {  // the end of K
                for (int h = 0; b + h < end && h < S::deep; ++h)
                  tc_mma_block<kPair>(d, wd + h * (kWBytes >> 4), xd + h * (x_bytes >> 4), id + h * kNext, col + 8, xcol,
                                      b + h > begin, min(4, (a.K - (b + h) * kBlockK + 31) / 32));
              }
              tc_commit<kPair>(empty_bar(stage));
              if (b + S::deep >= whole) tc_commit<kPair>(afull_bar(na & 1));
            }
            __syncwarp();
            if (((b + S::deep) & 3) == 0) ++ns;
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (!ok || *abort_flag) {
        if (elect_one()) tc_commit<kPair>(drain_bar);
        __syncwarp();
        const long long t = clock64();
        while (!mbar_try_wait(drain_bar, 0) && clock64() - t < kWaitCycles) {
        }
      }
    }
  } else {
    if constexpr (S::wide) take_registers<S::many>();
    // ============================ sums of pieces, and y ============================
    const int quad = warp & 3, group = (warp - 4) >> 2;
    const int mine = a.tn / S::groups, c0 = group * mine;  // this group's columns: a multiple of 8
    const int slice = kRows / a.split, row = quad * 32 + lane;
    const uint32_t freed = kPair ? peer(aempty_bar(0), 0) : aempty_bar(0);
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + c0;
    uint32_t na = 0;
    bool ok = true;
    if (!kPair && a.split > 1) cluster_wait();  // peers have begun, their barriers are set up
    for (int i = first; i < a.tiles && ok; i += step) {
      const Place at = place_of(i, a);
      const int n = at.n * S::tile_rows + half * kRows + row, t0 = at.t * a.tn + c0;
      const int sent = (min(a.tn, a.T - t0) + 3) / 4 * 4;  // tokens whose sums go to peers
      float sum[S::acc];
#pragma unroll
      for (int c = 0; c < S::acc; ++c) sum[c] = 0.0f;
      for (int p = p0; p < p1; ++p, ++na) {
        ok = wait_warp(afull_bar(na & 1), (na >> 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = taddr + (na & 1) * S::acc_cols;
        uint32_t v[S::asked];
        if (S::wide || a.split == 1) {
#pragma unroll
          for (int c = 0; c < S::acc; c += S::asked) {
            if (c >= mine) break;
            // (columns past the tile's are read and added too: nobody looks at their sums)
#pragma unroll
            for (int j = 0; j < S::asked; j += 8)
              if (c + j < S::acc) tc_ld8(from + c + j, v + j);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < S::asked; j += 2)
              if (c + j < S::acc) add_pair(sum[c + j], sum[c + j + 1], v[j], v[j + 1]);
          }
        } else {
          const uint32_t cta = row / slice;
          const uint32_t to = peer(base + recv_off, cta) + 4u * (uint32_t)(p * a.tn * slice) + 16u * (row % slice);
          const uint32_t bar = peer(join_bar, cta);
          for (int c = 0; c < sent; c += 8) {
            tc_ld8(from + c, v);
            tc_wait_ld();
            send(to + 4u * (uint32_t)(c * slice), v, bar);
            if (c + 4 < sent) send(to + 4u * (uint32_t)((c + 4) * slice), v + 4, bar);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) arrive_peer(freed + 8u * (na & 1));
          else mbar_arrive(freed + 8u * (na & 1));
        }
      }
      if (!ok) break;
      if (!S::wide && a.split > 1) {
        // a row of this CTA's for a token: its pieces' sums, in ascending order
        ok = wait_warp(join_bar, 0, ctl);
        if (!ok) break;
        const int n0 = n - row + rank * slice, tokens = min(a.tn, a.T - t0), shift = 31 - __clz(slice);
        const int worker = (int)threadIdx.x - 128;
        if (sent << shift <= 128) {  // one each
          const int j = worker, r = (j >> 2) & (slice - 1), t = (j & 3) + (j >> (shift + 2) << 2);
          if (n0 + r < a.N && t < tokens) store_y(a, t0 + t, n0 + r, sum_pieces(recv + j, a.tn * slice, a.pieces));
          continue;
        }
        // four tokens at a time (16 x 6144 x 4096 7.6 us, 8.2 with one; 64 x 4096 x 4096 8.2 and 9.5; but 8 x 1024 x 1024 3.6
        // and 3.4)
        for (int j = worker; j < sent / 4 << shift; j += 128) {
          const int r = j & (slice - 1), t = 4 * (j >> shift);
          if (n0 + r >= a.N) continue;
          const float4* piece = reinterpret_cast<const float4*>(recv) + j;
          float4 v = piece[0];
          for (int p = 1; p < a.pieces; ++p) {
            const float4 more = piece[p * (a.tn / 4) * slice];
            v = make_float4(v.x + more.x, v.y + more.y, v.z + more.z, v.w + more.w);
          }
          store_y(a, t0 + t, n0 + r, v.x);
          if (t + 1 < tokens) store_y(a, t0 + t + 1, n0 + r, v.y);
          if (t + 2 < tokens) store_y(a, t0 + t + 2, n0 + r, v.z);
          if (t + 3 < tokens) store_y(a, t0 + t + 3, n0 + r, v.w);
        }
        continue;
      }
      const int there = min(mine, a.T - t0);  // tokens
      const long long at_y = (long long)t0 * a.y_stride + n;
      uint16_t* y16 = static_cast<uint16_t*>(a.y) + at_y;
      if (a.y_dtype == MOE_FP32) {
        if (n < a.N)
          store_column<S::acc>(static_cast<float*>(a.y) + at_y, a.y_stride, sum, there, [](float v) { return v; });
      } else if (a.pairs) {
        if (a.y_dtype == MOE_BF16) store_pairs<S::acc, MOE_BF16>(y16, a.y_stride, sum, there, n < a.N, lane);
        else store_pairs<S::acc, MOE_FP16>(y16, a.y_stride, sum, there, n < a.N, lane);
      } else if (n < a.N) {
        if (a.y_dtype == MOE_BF16)
          store_column<S::acc>(y16, a.y_stride, sum, there, [](float v) { return (uint16_t)pack16x2<MOE_BF16>(v, 0.0f); });
        else
          store_column<S::acc>(y16, a.y_stride, sum, there, [](float v) { return (uint16_t)pack16x2<MOE_FP16>(v, 0.0f); });
      }
    }
  }
  __syncwarp();
  if (!kPair && a.split > 1) {
    if (warp < 4 || warp >= S::load_warp) cluster_wait();  // (the others have)
    cluster_arrive_relaxed();                              // nothing more is sent from here
    // A CTA that has its sums needs its peers no more, nor they it. One that gave up may still be sent some.
    if (__any_sync(~0u, *abort_flag)) cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // the pair's MMAs are done in both CTAs
  }
  if (warp == S::mma_warp) {
    tc_fence_after();
    tc_dealloc<kPair>(tmem, S::tmem);
  }
}

// 128 bytes x `rows` of 8-bit rows of K values.
bool make_map(CUtensorMap* map, const moe_fp8_rows_t& m, int rows, int K, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? m.row_stride : K)};
  const cuuint32_t box[2] = {kBlockK, (cuuint32_t)box_rows};
  const cuuint32_t steps[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Clusters of `ctas` CTAs of this footprint that run at one time on the current device, asked of the runtime: a cluster lies in
// one GPC, and GPCs differ in their SMs.
int clusters_of(const void* kernel, int ctas, int threads, int smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * 2 * num_sms());
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

// Of pairs. (A GPC with an odd number of SMs leaves one out.)
template <int kCols>
int pairs_at_once() {
  static std::atomic<int> known[64];  // (zero)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (known[dev] == 0) {
    using S = Shape<kCols, true>;
    known[dev] = clusters_of((const void*)fp8_gemm_kernel<kCols, true, kFromRows>, 2, S::threads, S::smem);
  }
  return known[dev];
}

// Of 2, 4 or 8 CTAs of narrow tiles. The runtime counts one CTA an SM for a kernel that allocates tensor memory, however
// little, where two of these run: one of the same footprint stands in, which is not launched. (74 of 4 and 36 of 8 where 304
// CTAs' room would be 76 and 38: 36 of 8, 64 tokens x 4608 rows of w x 4096, 9.4 us, 37 of them, x 4736, 14.0, in pairs 11.2;
// 74 of 4, one token x 9472 x 4096, 9.3, 75, x 9600, 13.5, 75 of 2 10.4.)
using Narrow = Shape<16, false>;
__global__ void __launch_bounds__(Narrow::threads, Narrow::per_sm) narrow_footprint() {}
int clusters_at_once(int ctas) {
  static std::atomic<int> known[64][kMostSplit + 1];  // (zero)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& n = known[dev][ctas];
  if (n == 0 && allow_smem<narrow_footprint, Narrow::smem>() == cudaSuccess)
    n = clusters_of((const void*)narrow_footprint, ctas, Narrow::threads, Narrow::smem);
  return n;
}

// CTAs that share a tile of tn tokens, where there are no more tiles than clusters that run at one time; what they send each
// other is held in 32 KB.
int split_of(long long tiles, int pieces, int tn) {
  int split = 1;
  if (pieces > 1)
    while (split < kMostSplit && tiles <= clusters_at_once(2 * split)) split *= 2;
  return tn > 8 * split ? 1 : split;
}

template <int kCols, bool kPair, int kFrom = kFromRows>
cudaError_t launch(const Fp8Gemm& g, Args a, cudaStream_t s) {
  using S = Shape<kCols, kPair>;
  const cudaError_t err = allow_smem<fp8_gemm_kernel<kCols, kPair, kFrom>, S::smem>();
  if (err != cudaSuccess) return err;
  long long slots = (long long)num_sms() * S::per_sm;
  if constexpr (kPair) slots = pairs_at_once<kCols>();
  if (slots < 1) return cudaErrorInvalidConfiguration;
  a.tiles_n = (g.N + S::tile_rows - 1) / S::tile_rows;
  auto width = [&](int tiles_t) { return ((g.T + tiles_t - 1) / tiles_t + 15) / 16 * 16; };
  const int least = (g.T + kCols - 1) / kCols;
  int best = least;
  if (S::wide) {
    // the number of rounds of tiles times a tile's time (its MMAs, and what each stage and its end cost beside them):
    // more and narrower tiles may fill the last round
    long long cost = 0;
    for (int n = least; n <= 2 * least + 2; ++n) {
      const int tn = width(n), tiles_t = (g.T + tn - 1) / tn;
      const long long c = ((long long)a.tiles_n * tiles_t + slots - 1) / slots * (tn + 200);
      if (n == least || c < cost) {
        cost = c;
        best = n;
      }
    }
  }
  a.tn = width(best);
  a.tiles_t = (g.T + a.tn - 1) / a.tn;
  a.tiles = a.tiles_n * a.tiles_t;
  a.split = 1;
  if (!S::wide) a.split = split_of(a.tiles, a.pieces, a.tn);
  const int recv = a.split > 1 ? a.pieces * a.tn * (kRows / a.split) * 4 : 0;
  const int room = (S::smem - 1024 - kHeader - recv) / (S::deep * (kWBytes + a.tn / S::ctas * kBlockK));
  a.stages = room < S::most_stages ? room : S::most_stages;
  CUtensorMap wmap, xmap = {};
  if (!make_map(&wmap, g.w, g.N, g.K, kRows) ||
      (kFrom == kFromRows && !make_map(&xmap, g.x, g.T, g.K, a.tn / S::ctas)))
    return cudaErrorInvalidValue;
  const int ctas = kPair ? 2 : a.split;
  const long long grid = a.split > 1 ? (long long)a.tiles * a.split : (a.tiles < slots ? a.tiles : slots) * ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::threads);
  cfg.dynamicSmemBytes = S::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<kCols, kPair, kFrom>, wmap, xmap, a);
}

}  // namespace

namespace {

Args common_args(const Fp8Gemm& g) {
  Args a = {};
  a.ws = g.w.scales;
  a.xs = g.x.scales;
  a.ws_stride = g.w.scale_stride;
  a.xs_stride = g.x.scale_stride;
  a.y = g.y;
  a.y_stride = g.y_stride;
  a.y_dtype = g.y_dtype;
  a.pairs = g.y_dtype != MOE_FP32 && g.N % 2 == 0 && g.y_stride % 2 == 0 && reinterpret_cast<uintptr_t>(g.y) % 4 == 0;
  a.T = g.T;
  a.N = g.N;
  a.K = g.K;
  a.piece = fp8_piece(g.K);
  a.pieces = (g.K + a.piece - 1) / a.piece;
  a.status = g.status;
  return a;
}

// Whether all tiles of so many tokens run at one time, a cluster each.
bool clusters_fit(const Fp8Gemm& g, int cols) {
  const long long rows = (g.N + kRows - 1) / kRows;
  return rows * ((g.T + cols - 1) / cols) <= clusters_at_once(kMostSplit);
}

}  // namespace

// The narrowest tiles that hold all tokens of a decode batch (every row of w is read once), or of which a cluster each
// runs at one time; else pairs. A pair's time goes with K (from 3 us, and 1.3 for each 1024 values), a cluster's with the
// sums that it sends, T N: 64 tokens x 4096 x 11008 take 13.4 us in clusters and 21.8 in pairs, 40 x 1024 x 4096 4.9 and 8.9,
// 64 x 1024 x 2048 5.3 and 5.7, 64 x 512 x 1024 3.9 and 4.3, but 64 x 2048 x 1024 5.8 and 4.4, 32 x 4096 x 1024 5.8 and 4.5,
// 200 x 1024 x 1536 6.5 and 5.4. Many rows of w for few tokens are read faster by more CTAs (16 x 8192 x 2048 6.2 us and 7.5,
// 32 x 8192 x 2048 6.8 and 7.4; but 16 x 4096 x 1536 5.8 and 5.5). Tiles that no CTAs share read w at least as fast as pairs
// (32 x 20,000 x 1024 6.8 and 7.2). The border T N = K^2 / 36 + 8000, and K of 1536, are drawn between such sizes; they follow
// from no count of cycles or bytes.
cudaError_t launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s) {
  const Args a = common_args(g);
  const long long rows = (g.N + kRows - 1) / kRows;
  // clusters rather than pairs (of one tile of w half of a pair's rows would be none)
  const bool pays = (g.T + 7) / 8 * 8LL * g.N <= (long long)g.K * g.K / 36 + 8000 || g.N <= kRows;
  const bool by_itself = split_of(rows, a.pieces, (g.T + 15) / 16 * 16) == 1;
  const bool few = pays || by_itself || g.K > 1536;
  auto fits = [&](int cols) { return (pays || a.pieces == 1) && clusters_fit(g, cols); };
  if (g.T <= 16 ? few : fits(16)) return launch<16, false>(g, a, s);
  if (g.T <= 32 ? few : fits(32)) return launch<32, false>(g, a, s);
  if (g.N <= kRows || fits(64)) return launch<64, false>(g, a, s);
  return launch<kMaxTokens, true>(g, a, s);
}

cudaError_t launch_fp8_linear(const uint16_t* x, long long x_stride, int dtype, const Fp8Gemm& g, cudaStream_t s) {
  // Where a cluster shares a tile each CTA quantizes its part of K on the way; CTAs that go from tile to tile would do it
  // again for each. (One token x 5120 x 4096 7.5 us, 10.0 with a launch before it; 16 tokens 9.0 and 10.5; 32 tokens x 4096
  // x 4096, 512 values of K a CTA, 9.2 and 9.9, but x 11008, 1536 values, 16.9 and 14.8 when tried: the quantizing takes longer
  // than the tiles of w.)
  Args a = common_args(g);
  a.x16 = x;
  a.x16_stride = x_stride;
  const long long rows = (g.N + kRows - 1) / kRows;
  // Values of K that a CTA would quantize. 1024 take it about 5 us, during which the GPU reads 32 MB: more are worth it as far
  // as w's bytes, and the four that a launch before this one moves for each value of x, take longer (16 tokens x 512 x 16,384
  // 9.6 us with a launch before it, 12.9 without, x 65,536 21.7 and 45.6; but one token x 4096 x 11,008 13.1 and 11.1, x 8192
  // x 16,384 26.1 and 24.0).
  const int split16 = split_of(rows * ((g.T + 15) / 16), a.pieces, 16);
  const int values = (a.pieces + split16 - 1) / split16 * a.piece;
  const bool hidden = values <= 1024 + (g.N + 4LL * g.T) * g.K / 32768;
  if (((g.T <= 16 && split16 > 1) || clusters_fit(g, 16)) && hidden)
    return dtype == MOE_BF16 ? launch<16, false, MOE_BF16>(g, a, s) : launch<16, false, MOE_FP16>(g, a, s);
  // (32 x 12,800 x 1024, whose tiles no CTAs share, 7.7 us with a launch before it, 10.3 without)
  const int split = split_of(rows, a.pieces, 32);
  if (g.T <= 32 && split > 1 && (a.pieces + split - 1) / split * a.piece <= 512)
    return dtype == MOE_BF16 ? launch<32, false, MOE_BF16>(g, a, s) : launch<32, false, MOE_FP16>(g, a, s);
  const cudaError_t e = launch_fp8_quantize(x, x_stride, g.T, g.K, dtype, g.x, s);
  return e != cudaSuccess ? e : launch_fp8_gemm(g, s);
}

}  // namespace moe

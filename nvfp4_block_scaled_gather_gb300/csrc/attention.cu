// Attention over whole prompts and over a paged cache, on tcgen05 (sm_103a).
//
// For a tile of 128 query rows and a block of 128 keys:
//   S = Q K^T                     (tensor cores, fp32 in tensor memory)
//   m' = max(m, rowmax S), P = exp2(c S - c m'), l = l 2^(c m - c m') + rowsum P      with c = scale log2 e
//   O = O 2^(c m - c m') + P V    (tensor cores, P in 16 bits from tensor memory)
// and at the end out = O / l. One pass over the keys; S and P never leave the
// SM. P is rounded to 16 bits because the tensor cores take it so: its error
// is that of the output's own rounding, 2^-8 or 2^-11 of it at most. l sums the
// unrounded ones. fp16 ends at 2^-24, where bf16 has fp32's range: there all of
// P and l are 2^7 larger (the factor cancels in O / l; P <= 2^15), so that
// weights down to 2^-21 of the largest keep their 11 bits and none above 2^-32
// is lost (a million such are 2^-12 of the row). m follows the running maximum lazily:
// as long as no score of the row exceeds m by 8 powers of two, P <= 256 is
// held against the old m (exact: the factor cancels in O / l) and O is not
// touched.
//
//  * A query row is a (token, head of the group): the heads that share a kv
//    head fill a tile together (128 / group tokens a tile), so a decode step
//    reads each key once for all of them.
//  * A work item is a pair of query tiles of one sequence and kv head (or one
//    tile: few rows) against a run of key blocks. There are two S and two O in
//    tensor memory, and the steps (a tile against a block) take them in turn,
//    so that the MMAs of one step run under the softmax of the other: with two
//    tiles each has its own S and O over the same blocks; with one tile each
//    has every other block, and the two O are joined at the end.
//  * Long sequences with few rows are cut into pieces (cut_of), whose partial
//    O, m, l a second kernel joins in order.
//  * Persistent CTAs, one per SM, walk the items, which are dealt out in order
//    of size (item_of).
//  * Warp roles: warps 0-7 softmax and the items' outputs; warp 8 loads tiles
//    by TMA into a ring (128-byte swizzle; a box is the rows of a page, or all
//    128); warp 9 hands out the items and cleans values (below); warps 10 and
//    11 issue the MMAs of one S and O each. Pages whose size is no multiple of
//    8 rows, and strides of 0, cannot be boxes: there warps 8 and 9 copy the
//    tiles by 16-byte cp.async.
//  * Blocks in which some row sees a key that another does not are masked, and
//    values there that are not finite are zeroed before the MMA (0 * NaN would
//    reach rows that do not see them); the rows that do see them get them
//    added at the end.
//  * Pages whose id is out of range are not loaded: their rows of a tile hold
//    what was there before, and every item that meets one gives its rows no
//    result (0 and -inf; so do the other pieces of a cut sequence, by the join).
//  * Every wait is bounded; on expiry the kernel records MOE_ERR_TIMEOUT,
//    drains its copies and MMAs, frees tensor memory and returns.
//
// What bounds it: of long prompts the MMAs (two of 128 x 128 x 128 a step) and
// the way from a step's weights to the next scores: 8192 tokens, 32 query and 8
// kv heads of 128, take 362 us over the same inputs again and 383 to 400 over
// new ones, 1520 and 1376 to 1436 TFLOP/s counting what the causal mask leaves,
// 80% and 72 to 75% of a large matrix product's rate (heads of 64: 354 us, for
// half the products). Of decode batches the reads of the cache (32 streams over
// 500..6000 keys, 8 kv heads: 82 us, 5.5 TB/s); of single short calls the chain
// from the plan over the first loads, S, P and O to the store (12 us, launch
// and all).
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_internal.h"
#include "internal.h"
#include "ldcg.cuh"
#include "mbar.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;       // query rows of a tile, keys of a block
constexpr int kThreads = 384;
constexpr int kLoaders = 64;     // threads that load by cp.async
constexpr int kPlan = 256;       // sequences whose plan is kept in shared memory, a thread each
constexpr int kClasses = 256;    // classes that items are put in by size
constexpr int kItems = 4;        // work items between the loader and the other roles
constexpr int kPoisoned = 8;     // more than the items that a loader can be ahead by
constexpr int kNoKey = -1, kNoPage = -2;  // for a key's row: past the sequence's end, in no page of the pool
constexpr int kItemReaders = 12;  // every warp
constexpr int kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // the two S (P goes over it) and the two O, 128 columns each
constexpr int kHeader = 16384;
constexpr float kLazy = 8.0f;    // powers of two that a score may exceed the running maximum by
template <int kType>
constexpr float kRaise = kType == MOE_FP16 ? 7.0f : 0.0f;  // powers of two that P and l are held larger by
constexpr float kUndone = -1.0f;  // in place of a piece's sum: the sequence has a bad page

template <int DP>
struct Sizes {
  static constexpr int tile = kTile * DP * 2;       // bytes of 128 rows
  static constexpr int stages = DP == 128 ? 4 : 8;  // 128 KB in flight
  static constexpr int smem = 2 * tile + stages * tile + kHeader;
};

// ------------------------------- PTX helpers --------------------------------
// One arrival for a whole warp.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// 16 bytes global -> shared through L2; zeros where there is no source.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// One arrival on the barrier once all of this thread's earlier copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One box of a 3-d tensor (head dimension, heads, rows) to shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// 32 bytes, a whole sector.
__device__ __forceinline__ void store32(void* to, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (tensor memory) += A B, 16-bit operands, A and B in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}
// 32 columns of this warp's 32 lanes (a thread: its row's 32 values). The whole
// warp has to execute these together: a __syncwarp() stands before them where
// lanes may have gone separate ways, which also keeps the compiler from pulling
// a lane's condition out of a loop around them.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// The two warps that share 32 rows meet (named barrier `id`); whether any thread says so.
__device__ __forceinline__ bool pair_any(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(any)
      : "r"(id), "r"(mine ? 1u : 0u)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors, 128-byte swizzle (16-byte piece c of row r
// at piece c ^ (r % 8) of its 128 bytes), descriptor version 1, swizzle mode
// 2. A tile of 128 rows is stored as halves of 64 columns, 128 bytes a row.
// K-major (Q and K: the head dimension is summed over): 8-row groups 1024
// bytes apart (stride offset).
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major (V: the rows are summed over): 64-column halves 128 * 128 bytes
// apart (leading offset), 8-row groups 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((kTile * 128) >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor, kind::f16: fp32 accumulators, both operands bf16 or
// both fp16, M = 128, N = n; B MN-major if mn.
__device__ __forceinline__ uint32_t idesc_f16(int type, int n, bool mn) {
  const uint32_t f = type == MOE_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTile >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in one 64-bit register: one instruction multiplies or adds both.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_pair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 1 / x to one ulp or so.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int kType>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (kType == MOE_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int kType>
__device__ __forceinline__ float to_f32(uint16_t bits) {
  return kType == MOE_BF16 ? __bfloat162float(__ushort_as_bfloat16(bits)) : __half2float(__ushort_as_half(bits));
}
// Clears the halves of a word that are not finite; whether there were any.
template <int kType>
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w) {
  constexpr uint32_t kLo = kType == MOE_BF16 ? 0x7F80u : 0x7C00u, kHi = kLo << 16;
  const bool lo = (w & kLo) == kLo, hi = (w & kHi) == kHi;
  if (lo) w &= 0xFFFF0000u;
  if (hi) w &= 0x0000FFFFu;
  return lo || hi;
}

__device__ __forceinline__ void report(int* status, int what) { atomicCAS(status, 0, what); }

// ------------------------------- bounded waits -------------------------------
struct Ctl {
  volatile int* abort_flag;
  int* status;
};

__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Ctl c) {
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
// By a whole warp, the same answer in every lane: false if this or another role gave up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Ctl& c) {
  return __all_sync(~0u, mbar_try_wait(bar, parity) || wait_slow(bar, parity, c));
}

// ---------------------------------- the plan ----------------------------------
struct Seq {
  int first, nq;   // queries: first row, count
  int k0, nk;      // keys: first packed row or row of the table, count
};

// Rows first .. end - 1 within total: how many (0 where they run backwards; no
// difference of offsets that could pass 32 bits is taken).
__device__ __forceinline__ int rows_between(int first, int end, int total) {
  return max(min(end, total), first) - first;
}
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  s.first = max(ld_cg(a.cu_q + b), 0);
  s.nq = rows_between(s.first, ld_cg(a.cu_q + b + 1), a.total_q);
  s.nk = 0;
  if (a.paged) {
    s.k0 = ld_cg(a.seqs + b);
    if (s.k0 >= 0 && s.k0 < a.max_seqs) {
      s.nk = ld_cg(a.length + s.k0);
      if (s.nk < 0 || (long long)s.nk > (long long)a.max_pages * a.page_size) {
        s.nk = 0;
        report(a.status, MOE_ERR_INVALID);
      }
    } else {
      s.k0 = 0;
      if (s.nq > 0) report(a.status, MOE_ERR_INVALID);
    }
  } else {
    s.k0 = max(ld_cg(a.cu_k + b), 0);
    s.nk = rows_between(s.k0, ld_cg(a.cu_k + b + 1), a.total_k);
  }
  return s;
}

struct __align__(16) Planned {
  Seq seq;
  int pairs;     // query tile pairs
  Cut cut;
  int items;     // pairs x pieces
};
static_assert(sizeof(Planned) == 32, "two 16-byte reads");
__device__ __forceinline__ Planned plan_of(const AttnArgs& a, int b, int tokens_per_tile) {
  Planned w;
  w.seq = seq_of(a, b);
  w.pairs = (w.seq.nq + 2 * tokens_per_tile - 1) / (2 * tokens_per_tile);
  const int blocks = (w.seq.nk + kTile - 1) / kTile;
  w.cut = a.part_o && w.seq.nq > 0 ? cut_of(blocks, w.pairs * a.heads_kv) : Cut{1, blocks};
  w.items = w.pairs * w.cut.pieces;
  return w;
}
__device__ __forceinline__ long long part_rows_of(const AttnArgs& a, const Planned& w) {
  return w.cut.pieces > 1 ? (long long)w.seq.nq * a.heads_q * w.cut.pieces : 0;
}
// Items of a sequence (for one kv head) of at least n key blocks: all alike,
// or (causal) those of the later query tile pairs.
__device__ __forceinline__ int items_from(const AttnArgs& a, const Planned& w, int n, int tokens_per_tile) {
  if (w.items == 0 || n > w.cut.blocks) return 0;
  if (n <= 0 || w.cut.pieces > 1 || a.mask) return w.items;
  // pair p sees the keys before nk - nq + (p + 1) * 2 * tokens_per_tile
  const int rest = (n - 1) * kTile - (w.seq.nk - w.seq.nq);
  if (rest <= 0) return w.pairs;
  const int tokens = 2 * tokens_per_tile;
  const int shorter = (tokens & (tokens - 1)) == 0 ? rest >> (31 - __clz(tokens)) : rest / tokens;
  return w.pairs - min(shorter, w.pairs - 1);
}

struct __align__(16) Item {
  int first, tokens;      // first query row (token) of the pair, its tokens
  int i0, nq;             // place of the first token in its sequence, the sequence's queries
  int k0, nk;             // as Seq
  int b0, blocks;         // run of key blocks
  int kvh, two;           // kv head; 1: two tiles
  int pieces, end;        // pieces of the sequence; 1: no more items (nothing else holds)
  long long part;         // first partial row of the piece
  int rows, piece;        // the sequence's partial rows per piece; which piece
};
static_assert(sizeof(Item) == 64, "four 16-byte reads");

// How many of the first keys a query sees: all up to its own (chain), or those
// before the drafted ones (tree; the rest is in its bits).
__device__ __forceinline__ int limit_of(const AttnArgs& a, int nk, int nq, int i) {
  const int l = nk - nq + (a.mask ? 0 : i + 1);
  return min(max(l, 0), nk);
}

// Bits of the keys pos .. pos + 31 that query i (row t) of the sequence sees.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs& a, int t, int nk, int nq, int limit, int pos) {
  const int n = limit - pos;
  uint32_t w = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
  if (!a.mask) return w;
  const int j = pos - (nk - nq);  // place of key pos among the drafted
  if (j <= -32 || j >= nq) return w;
  const int* row = a.mask + (long long)t * a.mask_words;
  uint32_t bits;
  if (j < 0) {
    bits = (uint32_t)ld_cg(row) << -j;
  } else {
    const int i = j >> 5;
    const uint32_t lo = i < a.mask_words ? (uint32_t)ld_cg(row + i) : 0u;
    const uint32_t hi = i + 1 < a.mask_words ? (uint32_t)ld_cg(row + i + 1) : 0u;
    bits = __funnelshift_r(lo, hi, j & 31);
  }
  const int left = nq - j;  // drafted tokens from here on
  if (left < 32) bits &= (1u << left) - 1u;
  return w | bits;
}
__device__ __forceinline__ bool sees_any(const AttnArgs& a, int t, int nk, int nq, int limit) {
  bool any = limit > 0;
  if (a.mask && !any)
    for (int pos = 0; pos < nk; pos += 32) any |= seen_bits(a, t, nk, nq, limit, pos) != 0;
  return any;
}

// What the plan leaves in shared memory.
struct Plan {
  union {
    Planned seq[kPlan];                // of up to kPlan sequences
    int group[kPlan + 1];              // of more: items before each group of 32 * per sequences
  };
  long long part[kPlan];               // partial rows before a sequence (or group)
  int from[kClasses + 1];              // items of class c (2^shift blocks) and above
  int total;                           // items for one kv head
  int shift, classes;
  int per;
};

// By a whole warp: this CTA's item of a round. The items stand in order of
// falling size (number of key blocks), a kv head after the other, and are
// dealt to the CTAs forth and back, which comes within a few per cent of the
// best there is: 992 items of 9 ragged prompts, 992 / 152 to a CTA, end after
// 82 steps instead of the 112 that dealing them out as they stand takes (80
// where each CTA takes the longest that is left). Counts of the sizes, made
// once, tell the size of an item; then a pass over the sequences finds its own
// (1600 cycles for 9 sequences, 3800 for 256; without the counts 9000, which
// short items waited for: 256 streams over 300..1500 keys 206 us, so 179). With
// more sequences than the plan holds the items are dealt in the order of the
// call, and 32 sequences are read again for an item (1024 streams over
// 300..1500 keys: 660 us, 5.7 TB/s; searched from the first one on 1870).
__device__ __forceinline__ Item item_of(const AttnArgs& a, const Plan& plan, int round, int tpt) {
  const int lane = threadIdx.x & 31;
  Item x = {};
  // (below 2^32: an item has a row of a tile at least, or of a partial result, and both are counted in 31 bits; up to
  // kPlan sequences may share rows: each has less than 2^23 items)
  const uint32_t next = (uint32_t)round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  // (a CTA's last round can miss it, but then no later one is left)
  x.end = next >= (unsigned long long)plan.total * a.heads_kv;
  if (x.end) return x;
  int u = (int)(next / (uint32_t)a.heads_kv);  // item of this kv head
  const int kvh = (int)(next - (uint32_t)u * a.heads_kv);
  int b = 0, first = 0;                        // its sequence, and where the sequence's items of this size begin
  Planned w;
  long long part;
  if (a.n == 1) {
    w = plan.seq[0];
    part = 0;
  } else if (a.n <= kPlan) {
    // the class c with from[c + 1] <= u < from[c]
    int c = 0, above = plan.classes;
    while (above - c > 1) {
      const int mid = (c + above) >> 1;
      if (plan.from[mid] > u) c = mid;
      else above = mid;
    }
    u -= plan.from[c + 1];
    const int least = c << plan.shift, more_than = (c + 1) << plan.shift;
    // the sequence among those with items of this class
    for (int i0 = 0;; i0 += 32) {
      int more = 0, count = 0;
      if (i0 + lane < a.n) {
        more = items_from(a, plan.seq[i0 + lane], more_than, tpt);
        count = items_from(a, plan.seq[i0 + lane], least, tpt) - more;
      }
      const int all = __reduce_add_sync(~0u, count);
      if (u >= all && i0 + 32 < a.n) {
        u -= all;
        continue;
      }
      int sum = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t reach = __ballot_sync(~0u, sum > u);
      const int at = reach ? __ffs(reach) - 1 : 0;
      b = i0 + at;
      u -= __shfl_sync(~0u, sum - count, at);
      first = __shfl_sync(~0u, more, at);
      break;
    }
    w = plan.seq[b];
    part = plan.part[b];
  } else {
    int g = 0, above = kPlan;  // the group with group[g] <= u < group[g + 1]
    while (above - g > 1) {
      const int mid = (g + above) >> 1;
      if (plan.group[mid] <= u) g = mid;
      else above = mid;
    }
    u -= plan.group[g];
    part = plan.part[g];
    // its sequences, 32 at a time
    for (long long i0 = (long long)g * 32 * plan.per;; i0 += 32) {
      Planned mine = {};
      if (i0 + lane < a.n) mine = plan_of(a, (int)i0 + lane, tpt);
      int sum = mine.items;
      long long rows = part_rows_of(a, mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, sum, o);
        const long long z = __shfl_up_sync(~0u, rows, o);
        if (lane >= o) {
          sum += y;
          rows += z;
        }
      }
      const uint32_t reach = __ballot_sync(~0u, sum > u);
      if (reach || i0 + 32 >= a.n) {
        const int at = reach ? __ffs(reach) - 1 : 0;
        u -= __shfl_sync(~0u, sum - mine.items, at);
        part += __shfl_sync(~0u, rows - part_rows_of(a, mine), at);
        w = plan_of(a, min((int)i0 + at, a.n - 1), tpt);
        break;
      }
      u -= __shfl_sync(~0u, sum, 31);
      part += __shfl_sync(~0u, rows, 31);
    }
  }
  u += first;
  const Seq& s = w.seq;
  const int pair = max(w.pairs - 1 - u / w.cut.pieces, 0);
  x.piece = u % w.cut.pieces;
  x.i0 = pair * 2 * tpt;
  x.first = s.first + x.i0;
  x.tokens = min(2 * tpt, s.nq - x.i0);
  x.two = x.tokens > tpt;
  x.nq = s.nq;
  x.k0 = s.k0;
  x.nk = s.nk;
  x.kvh = kvh;
  // the keys that any row of the pair sees end here
  const int keys = a.mask ? s.nk : limit_of(a, s.nk, s.nq, x.i0 + x.tokens - 1);
  x.b0 = x.piece * w.cut.blocks;
  x.blocks = max(0, min((keys + kTile - 1) / kTile - x.b0, w.cut.blocks));
  x.pieces = w.cut.pieces;
  x.rows = s.nq * a.heads_q;
  x.part = part + (long long)x.piece * x.rows;
  return x;
}

// By a whole warp: whether any of the page ids first .. last of a row of the
// table is out of range. Rarely needed, and kept out of line: within the
// loader's code it made decode_one 13.8 us instead of 12.6 and trees of 16
// streams 48.7 instead of 41.2, where it never runs.
__device__ __noinline__ bool any_bad(const int* row, int first, int last, int n_pages) {
  bool bad = false;
  for (int at = first + (threadIdx.x & 31); at <= last; at += 32) {
    const int p = ld_cg(row + at);
    bad |= p < 0 || p >= n_pages;
  }
  return __any_sync(~0u, bad);
}

// The tensor maps of a call (boxes of 64 columns).
struct Maps {
  CUtensorMap q, k, v;
  int use;       // 0: the tiles are copied by cp.async
  int box;       // rows of a box of K and V
  int wide;      // the output's rows are whole sectors of 32 bytes
};

// A place in the ring of tiles and the parity of its round.
template <int kStages>
struct Place {
  int slot;
  uint32_t parity;
  __device__ __forceinline__ void step(int by) {  // by <= kStages
    slot += by;
    if (slot >= kStages) {
      slot -= kStages;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int by) {
    slot += by;
    parity ^= (uint32_t)(slot / kStages) & 1u;
    slot %= kStages;
  }
};

template <int kType, int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnArgs a,
                                                                  const __grid_constant__ Maps maps) {
  using Sz = Sizes<DP>;
  constexpr int kStages = Sz::stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle needs it; the same for every thread
    if (threadIdx.x == 0) report(a.status, MOE_ERR_CUDA);
    return;
  }
  const uint32_t sQ = smem_u32(smem), sKV = sQ + 2 * Sz::tile;
  uint8_t* head = smem + (2 + kStages) * Sz::tile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(head);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (8 + s); };
  auto qfull_bar = [&](int s) { return bar0 + 8u * (16 + s); };
  auto qempty_bar = [&](int s) { return bar0 + 8u * (18 + s); };
  auto sfull_bar = [&](int w) { return bar0 + 8u * (20 + w); };
  auto pfull_bar = [&](int w, int part) { return bar0 + 8u * (part ? 47 + w : 22 + w); };  // 2 x 32 keys of P each
  auto ofull_bar = [&](int w) { return bar0 + 8u * (24 + w); };
  auto oempty_bar = [&](int w) { return bar0 + 8u * (26 + w); };
  const uint32_t drain_bar = bar0 + 8u * 29, drain2_bar = bar0 + 8u * 46;
  auto ifull_bar = [&](int i) { return bar0 + 8u * (30 + i); };
  auto iempty_bar = [&](int i) { return bar0 + 8u * (34 + i); };
  auto land_bar = [&](int s) { return bar0 + 8u * (38 + s); };  // values that are cleaned before they are full
  // after the barriers (49 of them, 392 bytes)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(head + 392);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(head + 396);
  volatile int* poisoned = reinterpret_cast<volatile int*>(head + 416);    // [kPoisoned]
  Item* s_item = reinterpret_cast<Item*>(head + 448);                      // [kItems]
  float* s_top = reinterpret_cast<float*>(head + 704);                     // [2][128]
  int* s_wsum = reinterpret_cast<int*>(head + 1728);                       // [warps] items, then sizes
  long long* s_wpart = reinterpret_cast<long long*>(head + 1856);          // [warps] partial rows; of many sequences, queries
  volatile int* undone = reinterpret_cast<volatile int*>(head + 1952);     // [kPoisoned]
  Plan& plan = *reinterpret_cast<Plan*>(head + 1984);
  static_assert(1984 % alignof(Plan) == 0 && 1984 + sizeof(Plan) <= kHeader, "the header holds it");

  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  if (warp == 0) {  // a barrier or two to a lane
    auto arrivals = [&](int i) -> int {
      if (i < 8) return maps.use ? 1 : kLoaders;         // full
      if (i < 16) return 2;                              // empty: both MMA warps
      if (i < 18) return maps.use ? 1 : kLoaders;        // query tiles full
      if (i < 20) return 2;                              // query tiles empty
      if (i < 22) return 1;                              // scores full
      if (i < 24 || i == 47 || i == 48) return 8;        // weights full: warps
      if (i < 26) return 1;                              // O full
      if (i < 28) return 8;                              // O empty: warps
      if (i >= 30 && i < 34) return 1;                   // items full
      if (i >= 34 && i < 38) return kItemReaders;        // items empty
      return 1;                                          // landed values, drains
    };
    for (int i = lane; i < 49; i += 32) mbar_init(bar0 + 8u * i, arrivals(i));
    if (lane < kPoisoned) poisoned[lane] = undone[lane] = 0;
    if (lane == 0) *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8 && maps.use && lane < 3) tma_prefetch(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v);
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  pdl_wait();
  pdl_trigger();
  const int group = a.group, tpt = a.tile_tokens;
  // the plan, a thread to a sequence
  const bool kept = a.n <= kPlan;
  const int groups = (a.n + 31) / 32, per = (groups + kPlan - 1) / kPlan;  // of more sequences
  if (!kept) {
    if (tid < kPlan) plan.group[tid + 1] = 0, plan.part[tid] = 0;
    __syncthreads();
  }
  int count = 0, size = 0;
  long long part = 0, many = 0;
  for (int b0 = warp * 32; b0 < a.n; b0 += kThreads) {
    Planned w = {};
    if (b0 + lane < a.n) w = plan_of(a, b0 + lane, tpt);
    if (kept) {
      if (b0 + lane < a.n) plan.seq[b0 + lane] = w;
    } else {
      const int g = b0 / 32 / per, items = __reduce_add_sync(~0u, w.items);
      many += w.seq.nq;
      long long rows = part_rows_of(a, w);
      for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(~0u, rows, o);
      if (lane == 0) {
        atomicAdd(&plan.group[g + 1], items);
        if (g + 1 < kPlan) atomicAdd(reinterpret_cast<unsigned long long*>(&plan.part[g + 1]), (unsigned long long)rows);
      }
    }
    count += w.items;
    size = max(size, w.items ? w.cut.blocks : 0);
    part += part_rows_of(a, w);
  }
  long long p = part;  // inclusive sum of the warp's partial rows
  if (a.part_o && kept)
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, p, o);
      if (lane >= o) p += y;
    }
  if (!kept)
    for (int o = 16; o > 0; o >>= 1) many += __shfl_xor_sync(~0u, many, o);
  count = __reduce_add_sync(~0u, count);
  size = __reduce_max_sync(~0u, size);
  if (lane == 31) {
    s_wsum[warp] = count;
    s_wsum[16 + warp] = size;
    s_wpart[warp] = kept ? p : many;
  }
  __syncthreads();
  {
    const bool has = lane < kThreads / 32;
    int all = __reduce_add_sync(~0u, has ? s_wsum[lane] : 0);
    if (!kept) {
      // Offsets that go back and forth give a row to several sequences, and of
      // thousands of sequences that can make more items than 32 bits count:
      // where the sequences have more queries than there are, nothing is done.
      long long queries = 0;
      for (int x = 0; x < kThreads / 32; ++x) queries += s_wpart[x];
      if (queries > a.total_q) {
        all = 0;
        if (tid == 0) report(a.status, MOE_ERR_INVALID);
        if (a.part_of)  // the join finds no rows
          for (long long i = (long long)blockIdx.x * kThreads + tid; i < (long long)a.total_q * a.heads_q;
               i += (long long)gridDim.x * kThreads)
            a.part_of[i] = make_int4(-1, 0, 0, 0);
      }
    }
    const int largest = __reduce_max_sync(~0u, has ? s_wsum[16 + lane] : 0);
    int shift = 0;
    while ((largest >> shift) >= kClasses) ++shift;
    if (kept && tid < kPlan) {
      p -= part;
      if (a.part_o)
        for (int x = 0; x < warp; ++x) p += s_wpart[x];
      plan.part[tid] = p;
    }
    const int classes = (largest >> shift) + 1;
    if (kept && a.n > 1)  // a warp counts a class
      for (int c = warp; c <= classes; c += kThreads / 32) {
        int items = 0;
        for (int i = lane; i < a.n; i += 32) items += items_from(a, plan.seq[i], c << shift, tpt);
        items = __reduce_add_sync(~0u, items);
        if (lane == 0) plan.from[c] = items;
      }
    if (tid == 0) {
      plan.total = all;
      plan.shift = shift;
      plan.classes = classes;
      plan.per = per;
      if (!kept) plan.group[0] = 0;
    }
  }
  __syncthreads();
  if (!kept) {
    if (warp == (maps.use ? 9 : 8)) {  // the warp that hands out: items and rows before each group
      int mine[kPlan / 32], sum = 0;
      long long rows[kPlan / 32], all = 0;
#pragma unroll
      for (int i = 0; i < kPlan / 32; ++i) {
        mine[i] = sum += plan.group[1 + lane * (kPlan / 32) + i];
        rows[i] = all += plan.part[lane * (kPlan / 32) + i];
      }
      int before = sum;
      long long rows_before = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, before, o);
        const long long z = __shfl_up_sync(~0u, rows_before, o);
        if (lane >= o) before += y, rows_before += z;
      }
#pragma unroll
      for (int i = 0; i < kPlan / 32; ++i) {
        plan.group[1 + lane * (kPlan / 32) + i] = mine[i] + before - sum;
        plan.part[lane * (kPlan / 32) + i] = rows[i] + rows_before - all;
      }
    }
    __syncwarp();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, a.status};

  // Every role takes the items from the ring in order.
  int seq_no = 0;
  Item it = {};
  auto next_item = [&]() -> bool {
    const int i = seq_no % kItems;
    if (!wait_bar(ifull_bar(i), (seq_no / kItems) & 1, ctl)) return false;
    it = s_item[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(iempty_bar(i));
    ++seq_no;
    return it.end == 0;
  };

  if (warp == 8 || warp == 9) {
    // ================================ loader ================================
    const int lw = warp - 8;
    int round = 0;  // of items: one for each CTA
    Place<kStages> ring = {0, 0};
    Place<2> qring = {0, 0};
    uint32_t landed = 0;  // parities of the land barriers, a bit each
    bool ok = true;
    // Decodes the next item and hands it out (after the last: ends).
    int handed = 0;
    auto hand_out = [&]() -> bool {
      const int i = handed % kItems;
      if (!wait_bar(iempty_bar(i), ((handed / kItems) & 1) ^ 1, ctl)) return false;
      ++handed;
      const Item x = item_of(a, plan, round, tpt);
      if (lane == 0) {
        s_item[i] = x;
        mbar_arrive(ifull_bar(i));
      }
      ++round;
      return true;
    };
    // Row of the packed keys or of the cache's planes that holds key `pos`, or kNoKey or kNoPage.
    auto row_of = [&](int pos) -> int {
      if (pos >= it.nk) return kNoKey;
      if (!a.paged) return it.k0 + pos;
      const int at = pos / a.page_size;
      const int p = ld_cg(a.table + (long long)it.k0 * a.max_pages + at);
      if (p < 0 || p >= a.n_pages) {
        report(a.status, MOE_ERR_INVALID);
        return kNoPage;
      }
      return p * a.page_size + (pos - at * a.page_size);
    };
    // Pages that none of the item's rows sees (a chain: its earlier rows do not
    // see the last pages). The piece that has the last key that the rows see
    // looks at the pages behind it before its first block, so that all rows of a
    // sequence agree on its pages.
    auto check_unseen_pages = [&]() {
      const int end = (it.b0 + it.blocks) * kTile;
      if (a.paged && !a.mask && end < it.nk && limit_of(a, it.nk, it.nq, it.i0 + it.tokens - 1) <= end &&
          any_bad(a.table + (long long)it.k0 * a.max_pages, end / a.page_size, (it.nk - 1) / a.page_size, a.n_pages)) {
        if (lane == 0) {
          report(a.status, MOE_ERR_INVALID);
          undone[(seq_no - 1) % kPoisoned] = seq_no;
        }
        __syncwarp();
      }
    };
    // 16-byte chunk c of row r of a tile.
    auto chunk_at = [](uint32_t tile, int r, int c) -> uint32_t {
      return tile + (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    };
    auto at_smem = [&](uint32_t at) { return reinterpret_cast<uint4*>(smem + (at - sQ)); };
    auto clean_chunk = [&](uint32_t at) -> bool {  // whether anything had to be cleared
      uint4 v = *at_smem(at);
      bool f = clear_nonfinite<kType>(v.x);
      f |= clear_nonfinite<kType>(v.y);
      f |= clear_nonfinite<kType>(v.z);
      f |= clear_nonfinite<kType>(v.w);
      if (f) *at_smem(at) = v;
      return f;
    };
    constexpr int kChunks = DP / 8;  // of a row
    if (maps.use && lw == 0) {
      // ----------------------------- TMA loads -----------------------------
      const int boxes = kTile / maps.box;
      const uint64_t normal = policy_normal(), once = policy_evict_first();
      const uint32_t box_bytes = (uint32_t)maps.box * 128u, q_bytes = (uint32_t)(tpt * group * 128);
      // per ring place: whether it was filled, by which barrier, in which parity
      uint32_t filled = 0, by_land = 0, parity = 0, qfilled = 0, qparity = 0;
      while (ok) {
        ok = next_item();
        if (!ok) break;
        const int n = __shfl_sync(~0u, it.blocks, 0), item_no = seq_no - 1;
        if (n == 0) continue;
        const int lim = limit_of(a, it.nk, it.nq, it.i0);  // the least that any row of the pair sees
        // keys that no other item of the sequence reads leave L2 first (to partial
        // results, for one): 4 trees over 24,000..40,000 keys 121 us so, 131
        // otherwise; 32 decode streams 83 and 86. Pages that forks share are not
        // told apart: 64 forks of 8000 keys 264 and 253, 16 forks 76 both ways
        const uint64_t policy = it.nq <= 2 * tpt ? once : normal;
        // lane i: row of box i of the block
        const int first = it.b0 * kTile + lane * maps.box;
        int row = lane < boxes ? row_of(first) : kNoKey;
        for (int q = 0; q < 1 + it.two && ok; ++q) {
          ok = wait_bar(qempty_bar(qring.slot), qring.parity ^ 1, ctl);
          if (ok && elect_one()) {
            mbar_expect_tx(qfull_bar(qring.slot), q_bytes * (DP / 64));
#pragma unroll
            for (int h = 0; h < DP / 64; ++h)
              tma_load(sQ + qring.slot * Sz::tile + h * kTile * 128, &maps.q, h * 64, it.kvh * group,
                       it.first + q * tpt, qfull_bar(qring.slot), normal);
          }
          __syncwarp();
          if (ok) {
            qfilled |= 1u << qring.slot;
            qparity = (qparity & ~(1u << qring.slot)) | (qring.parity << qring.slot);
          }
          qring.step(1);
        }
        check_unseen_pages();
        for (int b = 0; b < n && ok; ++b) {
          const int end = (it.b0 + b + 1) * kTile;
          const uint32_t there = __ballot_sync(~0u, row >= 0);
          if (__any_sync(~0u, row == kNoPage)) {
            if (lane == 0) undone[item_no % kPoisoned] = item_no + 1;
            __syncwarp();
          }
          const int nrow = lane < boxes && b + 1 < n ? row_of(first + (b + 1) * kTile) : kNoKey;
          const uint32_t bytes = (uint32_t)__popc(there) * box_bytes * (DP / 64);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (ok) ok = wait_bar(empty_bar(ring.slot), ring.parity ^ 1, ctl);
            if (!ok) break;
            const bool dirty = v == 1 && (end > it.nk || (end > lim && lim < it.nk));
            const uint32_t bar = dirty ? land_bar(ring.slot) : full_bar(ring.slot);
            const uint32_t dst = sKV + ring.slot * Sz::tile;
            const CUtensorMap* map = v ? &maps.v : &maps.k;
            const uint32_t bit = 1u << ring.slot;
            filled |= bit;
            if (dirty) landed ^= bit;  // parity of the next one to land
            by_land = dirty ? by_land | bit : by_land & ~bit;
            parity = ((dirty ? ~landed : ring.parity << ring.slot) & bit) | (parity & ~bit);
            if (elect_one()) mbar_expect_tx(bar, bytes);
            for (int i = 0; i < boxes; ++i) {
              const int z = __shfl_sync(~0u, row, i);
              if (z < 0) continue;
              if (elect_one()) {
#pragma unroll
                for (int h = 0; h < DP / 64; ++h)
                  tma_load(dst + h * kTile * 128 + i * box_bytes, map, h * 64, it.kvh, z, bar, policy);
              }
            }
            __syncwarp();
            ring.step(1);
          }
          row = nrow;
        }
      }
      if (*abort_flag) {
        // a role gave up: every load issued lands before the CTA exits
        const long long t0 = clock64();
        for (int i = 0; i < kStages; ++i)
          if ((filled >> i) & 1u)
            while (!mbar_try_wait((by_land >> i) & 1u ? land_bar(i) : full_bar(i), (parity >> i) & 1u) &&
                   clock64() - t0 < kWaitCycles) {
            }
        for (int i = 0; i < 2; ++i)
          if ((qfilled >> i) & 1u)
            while (!mbar_try_wait(qfull_bar(i), (qparity >> i) & 1u) && clock64() - t0 < kWaitCycles) {
            }
      }
    } else if (maps.use) {
      // -------------- values that some row does not see, and tails --------------
      // This warp also hands out the items, three ahead of the one that it
      // cleans (never more: the ring of items would wait for this warp itself),
      // the next one after the cleaning, which others wait for.
      for (int i = 0; i < 3 && ok; ++i) ok = hand_out();
      for (; ok; ok = ok && hand_out()) {
        ok = next_item();
        if (!ok) break;
        const int n = it.blocks;
        if (n == 0) continue;
        const int item_no = seq_no - 1;
        const int lim = limit_of(a, it.nk, it.nq, it.i0);
        Place<kStages> at = ring;
        for (int b = 0; b < n; ++b, at.step(2)) {
          const int end = (it.b0 + b + 1) * kTile;
          const bool edge = end > lim && lim < it.nk;
          if (end <= it.nk && !edge) continue;
          Place<kStages> v = at;
          v.step(1);
          if (!wait_bar(land_bar(v.slot), (landed >> v.slot) & 1, ctl)) { ok = false; break; }
          landed ^= 1u << v.slot;
          const uint32_t tile = sKV + v.slot * Sz::tile;
          const int rows = min(kTile, it.nk - (end - kTile));  // rows of this sequence
          // (the MMAs read whole steps of 16 rows)
          for (int i = rows * kChunks + lane; i < ((rows + 15) & ~15) * kChunks; i += 32)
            *at_smem(chunk_at(tile, i / kChunks, i % kChunks)) = make_uint4(0u, 0u, 0u, 0u);
          if (edge) {
            // carries out of the exponent tell whether anything is to be cleared
            constexpr uint32_t kExp = kType == MOE_BF16 ? 0x7F807F80u : 0x7C007C00u;
            constexpr uint32_t kOne = kType == MOE_BF16 ? 0x00800080u : 0x04000400u;
            uint32_t acc = 0;
#pragma unroll 8
            for (int i = lane; i < rows * kChunks; i += 32) {
              const uint4 x = *at_smem(tile + (uint32_t)i * 16 + (i * 16 >= rows * 128 ? (kTile - rows) * 128 : 0));
              acc |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
            }
            if (__any_sync(~0u, (acc & 0x80008000u) != 0)) {
              for (int i = lane; i < rows * kChunks; i += 32) clean_chunk(chunk_at(tile, i / kChunks, i % kChunks));
              if (lane == 0) poisoned[item_no % kPoisoned] = item_no + 1;
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(full_bar(v.slot));
        }
        ring.skip(2 * n);
      }
    } else {
      // --------------------------- cp.async copies ---------------------------
      // 32 rows (half h of this warp's 64) into a tile at `dst`: this lane's row
      // starts at element `at` of base, or is zero (at < 0); columns past the
      // head dimension are zero.
      constexpr int kRows = 32 / kChunks;  // rows of an instruction
      auto load_rows = [&](uint32_t dst, const uint16_t* base, int h, long long at) {
        const int c = lane % kChunks, sub = lane / kChunks;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kRows) {
          const int r = r0 + sub;
          const long long from = __shfl_sync(~0u, at, r);
          const bool there = from >= 0 && c * 8 < a.head_dim;
          cp_async16(chunk_at(dst, lw * 64 + h * 32 + r, c), base + (there ? from + c * 8 : 0), there);
        }
      };
      while (ok) {
        if (lw == 0) ok = hand_out();
        ok = ok && next_item();
        if (!ok) break;
        const int n = it.blocks, item_no = seq_no - 1;
        if (n == 0) continue;
        for (int q = 0; q < 1 + it.two && ok; ++q) {
          ok = wait_bar(qempty_bar(qring.slot), qring.parity ^ 1, ctl);
          if (!ok) break;
          for (int h = 0; h < 2; ++h) {
            const int r = lw * 64 + h * 32 + lane, token = r / group;
            long long at = -1;
            if (token < tpt && q * tpt + token < it.tokens)
              at = (long long)(it.first + q * tpt + token) * a.q.ts + (it.kvh * group + r % group) * a.q.hs;
            load_rows(sQ + qring.slot * Sz::tile, a.q.p, h, at);
          }
          cp_async_arrive(qfull_bar(qring.slot));
          qring.step(1);
        }
        const int lim = limit_of(a, it.nk, it.nq, it.i0);
        auto rows_of = [&](int block) {
          const int pos = (it.b0 + block) * kTile + lw * 64 + lane;
          return block < n ? make_int2(row_of(pos), row_of(pos + 32)) : make_int2(kNoKey, kNoKey);
        };
        int2 rows = rows_of(0);
        if (lw == 0) check_unseen_pages();
        for (int b = 0; b < n && ok; ++b) {
          const int2 later = rows_of(b + 1);
          if (rows.x == kNoPage || rows.y == kNoPage) {
            undone[item_no % kPoisoned] = item_no + 1;
            __threadfence_block();  // before this thread's arrival, which the copies make
          }
          const bool edge = (it.b0 + b + 1) * kTile > lim && lim < it.nk;
          for (int v = 0; v < 2; ++v) {
            const Heads& x = v ? a.v : a.k;
            ok = wait_bar(empty_bar(ring.slot), ring.parity ^ 1, ctl);
            if (!ok) break;
            const uint32_t dst = sKV + ring.slot * Sz::tile;
            load_rows(dst, x.p, 0, rows.x < 0 ? -1 : rows.x * x.ts + it.kvh * x.hs);
            load_rows(dst, x.p, 1, rows.y < 0 ? -1 : rows.y * x.ts + it.kvh * x.hs);
            if (v == 0 || !edge) {
              cp_async_arrive(full_bar(ring.slot));
            } else {  // each thread cleans what it copied
              cp_async_wait_all();
              bool found = false;
              for (int r0 = 0; r0 < 64; r0 += kRows)
                found |= clean_chunk(chunk_at(dst, lw * 64 + r0 + lane / kChunks, lane % kChunks));
              if (found) poisoned[item_no % kPoisoned] = item_no + 1;
              fence_proxy_async_shared();
              mbar_arrive(full_bar(ring.slot));
            }
            ring.step(1);
          }
          rows = later;
        }
      }
      if (*abort_flag) cp_async_wait_all();  // nothing of ours may be in flight at exit
    }
  } else if (warp >= 10) {
    // ============================== MMA issuer ==============================
    // Each of the two warps issues the MMAs of one S and O: S(0), then
    // O += P(j) V(j) and S(j + 1) in turn (S(j + 1) overwrites P(j), which the
    // order of one thread's MMAs allows). The whole warp keeps step and one
    // elected lane issues: in a branch of one lane the compiler moves every
    // operand to the uniform registers that these instructions take (8192 keys:
    // 856 us that way, 529 us this way, one issuing warp each time).
    const int w = warp - 10;
    const uint32_t id_s = idesc_f16(kType, kTile, false), id_o = idesc_f16(kType, DP, true);
    const uint32_t tS = tmem + kColS + w * 128, tO = tmem + kColO + w * 128;
    // Both warps go over every tile of the rings in order and let go of each,
    // its own ones by the completion of the MMAs that read them: a wait tells
    // two rounds of a barrier apart by parity alone, so a warp that skipped a
    // tile could take the round before last for the one that it waits for.
    const uint64_t qd0 = desc_kmajor(sQ), kd0 = desc_kmajor(sKV), vd0 = desc_mnmajor(sKV);
    Place<kStages> ring = {0, 0};
    Place<2> qring = {0, 0};
    uint32_t uses = 0, steps = 0;  // parities of O's items and of S's steps
    bool ok = true;
    auto pass = [&](uint32_t full, uint32_t parity, uint32_t empty) -> bool {  // a tile of the other warp's
      if (!wait_bar(full, parity, ctl)) return false;
      if (elect_one()) mbar_arrive(empty);
      return true;
    };
    while (ok && next_item()) {
      const int n = __shfl_sync(~0u, it.blocks, 0), two = __shfl_sync(~0u, it.two, 0);
      const int nk = __shfl_sync(~0u, it.nk, 0), b0 = __shfl_sync(~0u, it.b0, 0);
      if (n == 0) continue;
      const int last = two ? n - 1 : n - 1 - ((n - 1 - w) & 1);  // the last block of this S and O; below w: none
      Place<2> q = qring;
      if (two) {
        Place<2> o = qring;
        (w ? q : o).step(1);
        ok = pass(qfull_bar(o.slot), o.parity, qempty_bar(o.slot));
      }
      if (ok) ok = last < w && !two ? pass(qfull_bar(q.slot), q.parity, qempty_bar(q.slot))
                                    : wait_bar(qfull_bar(q.slot), q.parity, ctl);
      Place<kStages> at = ring, vat = ring;  // K of block b, V of the block whose P is awaited
      int pending = -1;
      bool first = true;
      for (int b = 0; b <= n && ok; ++b) {
        if (pending >= 0) {
          vat.step(1);
          if (first) ok = wait_bar(oempty_bar(w), uses ^ 1, ctl);
          if (!ok || !wait_bar(full_bar(vat.slot), vat.parity, ctl)) { ok = false; break; }
          fence_proxy_async_shared();
          const uint64_t vd = vd0 + (uint64_t)(vat.slot * (Sz::tile >> 4));
          // 16 keys a step; steps past the sequence's end are left out
          const int ksteps = min((nk - (b0 + pending) * kTile + 15) / 16, kTile / 16);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (ok) ok = wait_bar(pfull_bar(w, part), steps, ctl);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // keys 0..31 and 64..95, then the others: 8 columns of P, 2048 bytes of V
                const int k = 2 * part + (i & 1) + (i & 2) * 2;
                if (k < ksteps) tc_mma_ts(tO, tS + 8 * k, vd + (uint64_t)(k * (2048 >> 4)), id_o, !first || k != 0);
              }
              if (part) {
                tc_commit(empty_bar(vat.slot));
                if (pending == last) tc_commit(ofull_bar(w));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          steps ^= 1;
          first = false;
          pending = -1;
        }
        if (b == n) break;
        if (two || (b & 1) == w) {
          if (!wait_bar(full_bar(at.slot), at.parity, ctl)) { ok = false; break; }
          fence_proxy_async_shared();  // tiles may have been written by cp.async or cleaned
          tc_fence_after();
          const uint64_t qd = qd0 + (uint64_t)(q.slot * (Sz::tile >> 4));
          const uint64_t kd = kd0 + (uint64_t)(at.slot * (Sz::tile >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              const uint64_t off = (uint64_t)((k >> 2) * ((kTile * 128) >> 4) + (k & 3) * 2);
              tc_mma_ss(tS, qd + off, kd + off, id_s, k != 0);
            }
            tc_commit(sfull_bar(w));
            tc_commit(empty_bar(at.slot));
            if (b == last) tc_commit(qempty_bar(q.slot));
          }
          __syncwarp();
          vat = at;
          pending = b;
          at.step(2);
        } else {
          for (int i = 0; i < 2 && ok; ++i, at.step(1)) ok = pass(full_bar(at.slot), at.parity, empty_bar(at.slot));
        }
      }
      if (!first) uses ^= 1;
      ring.skip(2 * n);
      qring.skip(1 + two);
    }
    if (!ok || *abort_flag) {
      // wait for every MMA issued so far before tensor memory is freed
      const uint32_t bar = w ? drain2_bar : drain_bar;
      if (elect_one()) tc_commit(bar);
      const long long t0 = clock64();
      while (!mbar_try_wait(bar, 0) && clock64() - t0 < kWaitCycles) {
      }
    }
  } else {
    // =============================== softmax ===============================
    // Both warpgroups work on every step's S, a warpgroup on 64 of its 128 keys:
    // thread r of either has row r of the tile. The two threads of a row hold
    // the same maximum m; each has the sum l of its own keys and, of O, half of
    // the columns. They meet once a step (a barrier of the two warps that share
    // 32 rows, which tells whether any of these rows' maxima moves); only where
    // one moves do they exchange maxima. Splitting a row halves the time from S
    // to P, which with one warpgroup a tile was longer than the other tile's
    // MMAs.
    const int half = warp >> 2, quad = warp & 3;
    const int r = tid & 127;             // row of the tile = lane of tensor memory
    const int token = r / group, head_in = r - token * group;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const float c = a.scale * 1.4426950408889634f;
    uint32_t steps_done = 0, uses = 0;   // bit w: parities of S w's steps, of O w's items
    bool ok = true, agreed = false;      // agreed: the two warps of a row know from a step that they give up
    while (ok && next_item()) {
      const int n = it.blocks, two = it.two;
      const int steps = two ? 2 * n : n;
      const int rows0 = min(tpt, it.tokens) * group, rows1 = two ? (it.tokens - tpt) * group : rows0;
      // the least that any row of a tile sees
      const int lim0 = limit_of(a, it.nk, it.nq, it.i0), lim1 = two ? limit_of(a, it.nk, it.nq, it.i0 + tpt) : lim0;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // of the two S; m in units of the raw scores
      for (int t = 0; t < steps; ++t) {
        const int w = t & 1;
        const int tok0 = two && w ? tpt : 0;            // first token of the tile in the pair
        const int rows = w ? rows1 : rows0;
        const bool live = quad * 32 < rows;             // any row of this warp's
        const int pos = (it.b0 + (two ? t >> 1 : t)) * kTile;
        // some row of the tile does not see all of the block
        const bool edge = pos + kTile > (w ? lim1 : lim0);
        uint32_t bits[2] = {0u, 0u};
        if (edge && live && r < rows) {
          const int i = it.i0 + tok0 + token, limit = limit_of(a, it.nk, it.nq, i);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            bits[j] = seen_bits(a, it.first + tok0 + token, it.nk, it.nq, limit, pos + half * 64 + j * 32);
        }
        bool here = wait_bar(sfull_bar(w), (steps_done >> w) & 1, ctl);
        steps_done ^= 1u << w;
        if (live) {
          const uint32_t tS = lanes + kColS + w * 128, tO = lanes + kColO + w * 128 + half * (DP / 2);
          float m = w ? m1 : m0, l = w ? l1 : l0;
          tc_fence_after();
          uint32_t s[64];
          tc_ld32(tS + half * 64, s);
          tc_ld32(tS + half * 64 + 32, s + 32);
          tc_wait_ld();
          if (edge) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (!((bits[j / 32] >> (j % 32)) & 1u)) s[j] = 0xFF800000u;  // -inf
          }
          float mx[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mx[u] = max3(__uint_as_float(s[u]), __uint_as_float(s[u + 4]), __uint_as_float(s[u + 8]));
#pragma unroll
          for (int j = 12; j + 8 <= 64; j += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], __uint_as_float(s[j + u]), __uint_as_float(s[j + 4 + u]));
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], __uint_as_float(s[60 + u]));
          float top = max3(max3(m, mx[0], mx[1]), mx[2], mx[3]);
          // a warp whose wait gave up still meets the other one here, and tells
          if (!here) top = __int_as_float(0x7fffffff);
          if (pair_any(1 + quad, !here || (top > m && !((top - m) * c <= kLazy)))) {
            s_top[half * 128 + r] = top;
            pair_sync(1 + quad);
            const float theirs = s_top[(half ^ 1) * 128 + r];
            here = __all_sync(~0u, __float_as_int(top) != 0x7fffffff && __float_as_int(theirs) != 0x7fffffff);
            agreed = !here;
            top = fmaxf(top, theirs);
            const bool move = here && top > m && !((top - m) * c <= kLazy);
            if (here && t >= 2 && __any_sync(~0u, move)) {
              // S(t) is complete, so is every earlier MMA: O can be rescaled
              const float f = move ? ex2((m - top) * c) : 1.0f;
              l *= f;
              uint32_t o[32];
#pragma unroll 1
              for (int j = 0; j < DP / 2; j += 32) {
                tc_ld32(tO + j, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tc_st32(tO + j, o);
              }
            }
            if (move) m = top;
          }
          if (here) {
            const float base = m == -INFINITY ? 0.0f : fmaf(-m, c, kRaise<kType>);
            const uint64_t c2 = pair_of(c, c), base2 = pair_of(base, base);
            uint64_t sum[2] = {0, 0};
            // in two parts, so that the MMAs of the first run while the second is
            // made (8192 keys: 368 us, in one part 380); each waits for all eight
            // warps, whose rescaling of O must be over
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t p[16];
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const int e = part * 32 + j;
                const uint64_t x = fma2(pair_of(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, base2);
                float p0, p1;
                split_pair(x, p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], pair_of(p0, p1));
                p[j / 2] = pack2<kType>(p0, p1);
              }
              tc_st16(tS + half * 32 + part * 16, p);
              if (part == 0) {
                tc_wait_st();
                tc_fence_before();
                warp_arrive(pfull_bar(w, 0), lane);
              }
            }
            float a0, a1;
            split_pair(add2(sum[0], sum[1]), a0, a1);
            l += a0 + a1;
            tc_wait_st();
          }
          if (w) {
            m1 = m;
            l1 = l;
          } else {
            m0 = m;
            l0 = l;
          }
        }
        ok = here;
        if (!ok) break;
        if (!live) warp_arrive(pfull_bar(w, 0), lane);
        tc_fence_before();
        warp_arrive(pfull_bar(w, 1), lane);
      }
      if (!ok) break;
      // ------------------------------ epilogue ------------------------------
      // Of two tiles a warpgroup takes one each, of one tile half of the columns.
      const bool other = !two && n > 1;  // one tile: the second O holds the other half of its blocks
      const bool cut = it.pieces > 1;
      const int w = two ? half : 0, c0 = two ? 0 : half * (DP / 2), columns = two ? DP : DP / 2;
      const int rows = w ? rows1 : rows0;
      const bool live = quad * 32 < rows, valid = r < rows;
      float m = w ? m1 : m0, l = 0.0f, f0 = 1.0f, f1 = 1.0f;
      if (other) {
        m = fmaxf(m0, m1);
        f0 = m0 != -INFINITY ? ex2((m0 - m) * c) : 1.0f;
        f1 = m1 != -INFINITY ? ex2((m1 - m) * c) : 1.0f;
        l0 = l0 * f0 + l1 * f1;
      }
      if (n > 0 && quad * 32 < rows0) {  // the row's sum is that of its two threads
        agreed = pair_any(1 + quad, false);  // (the last exchange has been read) the other one gives up
        s_top[half * 128 + r] = two && half == 0 ? l1 : l0;
        pair_sync(1 + quad);
        l = (w ? l1 : l0) + s_top[(half ^ 1) * 128 + r];
      }
      ok = !agreed;
      if (!ok) break;
      if (n > 0) {
        // every warp sees every round of both O, its own or not
        if (two && half) {
          ok = wait_bar(ofull_bar(0), uses & 1, ctl);
          warp_arrive(oempty_bar(0), lane);
        }
        ok = ok && wait_bar(ofull_bar(w), (uses >> w) & 1, ctl);
        if (other) ok = ok && wait_bar(ofull_bar(1), (uses >> 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
      }
      // (O is complete, so every block has been through the loads and the cleaning)
      const bool gone = n > 0 && undone[(seq_no - 1) % kPoisoned] == seq_no;  // a page of the sequence's is bad
      const bool bad = n > 0 && !gone && poisoned[(seq_no - 1) % kPoisoned] == seq_no;
      if (gone) l = 0.0f;
      const int h = it.kvh * group + head_in;
      const int i = it.i0 + w * tpt + token, t_row = it.first + w * tpt + token;
      // rows of a cut sequence are kept a kv head after the other; eight of a
      // tile's together as [head_dim / 4][8][4], so that stores and the
      // join's reads are whole lines and what the join reads is in one place
      const int row0 = it.kvh * it.nq * group + (it.i0 + w * tpt) * group;
      const long long part = it.part + row0;
      const bool keep = cut && valid && part + rows <= a.part_rows;
      const int eight = min(8, rows - (r & ~7));  // rows of this row's eight
      float* part_o = a.part_o + part * a.head_dim + (r & ~7) * a.head_dim + (r & 7) * 4;
      // a row that sees no key gives 0; one whose scores are all -inf has no value
      float inv = 1.0f;
      if (!cut) {
        inv = rcp_approx(l);
        if (l == 0.0f) inv = valid && !gone && sees_any(a, t_row, it.nk, it.nq, limit_of(a, it.nk, it.nq, i)) ? NAN : 0.0f;
      }
      f0 *= inv;
      f1 *= inv;
      const long long at = valid && !cut ? (long long)t_row * a.out.ts + (long long)h * a.out.hs : -1;
      const uint32_t tO = lanes + kColO + w * 128 + c0;
#pragma unroll 1
      for (int j = 0; j < columns; j += 16) {
        uint32_t o[16];
        __syncwarp();
        if (n > 0 && live && !gone) {
          tc_ld16(tO + j, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          if (other) {
            uint32_t o1[16];
            tc_ld16(tO + 128 + j, o1);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0u;
        }
        const int column = c0 + j;
        if (column >= a.head_dim) continue;
        if (cut) {
          if (keep) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              if (column + e < a.head_dim)
                *reinterpret_cast<float4*>(part_o + (column + e) * eight) =
                    make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                __uint_as_float(o[e + 3]));
          }
        } else if (at >= 0) {
          // a thread has a row: 32 bytes at a time are whole sectors, and nothing
          // is waited for. 200 short prompts take 197 us so; with 32 columns of
          // the loop at a time (more code to fetch for every item) 205, by TMA
          // from shared memory about 210, and through shared memory, so that a
          // store writes whole lines, 208 to 214.
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = pack2<kType>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          uint16_t* to = a.out.p + at + column;
          if (maps.wide) {
            store32(to, v);
          } else {
            *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
            if (column + 8 < a.head_dim) *reinterpret_cast<uint4*>(to + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      if (n > 0) {  // O has been read
        tc_fence_before();
        warp_arrive(oempty_bar(w), lane);
        if (other) warp_arrive(oempty_bar(1), lane);
      }
      __syncwarp();
      if (n > 0) {
        if (two && !half) {
          ok = wait_bar(ofull_bar(1), (uses >> 1) & 1, ctl);
          warp_arrive(oempty_bar(1), lane);
        }
        uses ^= two || other ? 3u : 1u;
      }
      if (bad && valid && (keep || !cut)) {
        // add the values that are not finite of the keys that this row sees (a
        // rare path: kept small). The keys outside, 32 at a time, and the
        // columns inside: one infinity in a tree of 500 tokens takes 1.7 ms so,
        // 51 with a look at the mask and the table for every column (and tens
        // of thousands of tokens came near the other roles' limit on waits).
        const int from = max(it.b0, limit_of(a, it.nk, it.nq, it.i0) / kTile) * kTile;
        constexpr uint32_t kExp = kType == MOE_BF16 ? 0x7F807F80u : 0x7C007C00u;  // as in the cleaning
        constexpr uint32_t kOne = kType == MOE_BF16 ? 0x00800080u : 0x04000400u;
#pragma unroll 1
        for (int word = from; word < min((it.b0 + n) * kTile, it.nk); word += 32) {
#pragma unroll 1
          for (uint32_t seen = seen_bits(a, t_row, it.nk, it.nq, limit_of(a, it.nk, it.nq, i), word); seen; seen &= seen - 1) {
            const int pos = word + __ffs(seen) - 1;
            long long row = (long long)it.k0 + pos;
            if (a.paged) {
              const int p = ld_cg(a.table + (long long)it.k0 * a.max_pages + pos / a.page_size);
              if (p < 0 || p >= a.n_pages) continue;
              row = (long long)p * a.page_size + pos % a.page_size;
            }
            const uint16_t* values = a.v.p + row * a.v.ts + (long long)it.kvh * a.v.hs;
#pragma unroll 1
            for (int d0 = c0; d0 < min(c0 + columns, a.head_dim); d0 += 8) {
              const uint4 x = ld_cg(reinterpret_cast<const uint4*>(values + d0));
              if (!((((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne)) &
                    0x80008000u))
                continue;
#pragma unroll 1
              for (int d = d0; d < d0 + 8; ++d) {
                const float v = to_f32<kType>(values[d]);
                if (isfinite(v)) continue;
                if (cut) part_o[(d & ~3) * eight + (d & 3)] += v;
                else a.out.p[at + d] = (uint16_t)pack2<kType>(to_f32<kType>(a.out.p[at + d]) + v, 0.0f);
              }
            }
          }
        }
      }
      if (valid && (two || half == 0)) {
        const int row = t_row * a.heads_q + h;
        if (cut) {
          if (keep) a.part_ml[part + r] = make_float2(m * c, gone ? kUndone : l);
          else report(a.status, MOE_ERR_INVALID);
          if (it.piece == 0) {
            const bool any = sees_any(a, t_row, it.nk, it.nq, limit_of(a, it.nk, it.nq, i));
            a.part_of[(long long)(it.first - it.i0) * a.heads_q + row0 + r] =
                make_int4(keep ? (int)part : -1, rows | r << 8 | (any ? 1 << 16 : 0) | it.pieces << 17, it.rows, row);
          }
        } else {
          if (a.part_of) a.part_of[(long long)(it.first - it.i0) * a.heads_q + row0 + r] = make_int4(-1, 0, 0, 0);
          if (a.lse) a.lse[row] = l != 0.0f ? (m * c + (__log2f(l) - kRaise<kType>)) * 0.6931471805599453f : -INFINITY;
        }
      }
      __syncwarp();
    }
    // Every meeting of two warps begins with pair_any. If this one gave up
    // where the other one does not know (or the other way round), that one
    // will wait in its next meeting, or here: so they meet once more.
    if (!agreed && pair_any(1 + quad, !ok || *abort_flag != 0)) {
      s_top[half * 128 + r] = __int_as_float(0x7fffffff);
      pair_sync(1 + quad);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the pieces of cut sequences, in their order, with a running maximum: a
// CTA has eight rows of a tile (whose quads of columns lie together, 128
// bytes), a thread one quad of one row, the values of as many pieces in flight
// as middling sequences have. Bound by the latency of its reads where the
// pieces are few and small, so nothing is read before the values that could be
// read with them (16 trees over 300..5000 keys: 41 us in all; four pieces in
// flight 0.8 more).
constexpr int kJoinThreads = 256;
template <int kType>
__global__ void __launch_bounds__(kJoinThreads, 4) join_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int row = threadIdx.x & 7, q = threadIdx.x >> 3;
  const long long rows = (long long)a.total_q * a.heads_q, g = (long long)blockIdx.x * 8 + row;
  if (g >= rows) return;
  const int cu_first = ld_cg(a.cu_q), cu_end = ld_cg(a.cu_q + a.n);
  const int4 of = ld_cg(a.part_of + g);
  const int n = of.y & 0xFF, r = (of.y >> 8) & 0xFF, pieces = of.y >> 17;
  // (rows of no sequence hold anything)
  if (g < (long long)cu_first * a.heads_q || g >= (long long)cu_end * a.heads_q || of.x < 0 || pieces <= 1 || r >= n ||
      of.z <= 0 || of.w < 0 || of.w >= rows || of.x + (long long)(pieces - 1) * of.z + n > a.part_rows ||
      q * 4 >= a.head_dim)
    return;
  const int eight = min(8, n - (r & ~7));
  const float* from = a.part_o + ((long long)of.x + (r & ~7)) * a.head_dim + (r & 7) * 4 + q * 4 * eight;
  const float2* ml = a.part_ml + of.x + r;
  float top = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool undone = false;
#pragma unroll 1
  for (int i0 = 0; i0 < pieces; i0 += kSplitFew) {
    float4 v[kSplitFew];
    uint2 x[kSplitFew];
#pragma unroll
    for (int u = 0; u < kSplitFew; ++u) {  // past the last piece: the last one again, not used
      const long long at = (long long)min(i0 + u, pieces - 1) * of.z;
      x[u] = ld_cg(reinterpret_cast<const uint2*>(ml + at));
      v[u] = ld_cg(reinterpret_cast<const float4*>(from + at * a.head_dim));
    }
#pragma unroll
    for (int u = 0; u < kSplitFew; ++u) {
      const float m = __uint_as_float(x[u].x), sum = __uint_as_float(x[u].y);
      undone |= sum == kUndone;
      if (i0 + u < pieces && sum != 0.0f) {  // a sum of 0: the piece saw nothing
        const float now = fmaxf(top, m);
        const float keep = now == top ? 1.0f : ex2(top - now), f = now == m || m == -INFINITY ? 1.0f : ex2(m - now);
        l = l * keep + sum * f;
        o[0] = o[0] * keep + v[u].x * f;
        o[1] = o[1] * keep + v[u].y * f;
        o[2] = o[2] * keep + v[u].z * f;
        o[3] = o[3] * keep + v[u].w * f;
        top = now;
      }
    }
  }
  if (undone) l = o[0] = o[1] = o[2] = o[3] = 0.0f;
  const float inv = undone ? 0.0f : l != 0.0f ? rcp_approx(l) : ((of.y >> 16) & 1 ? NAN : 0.0f);
  const int t = of.w / a.heads_q, h = of.w - t * a.heads_q;
  *reinterpret_cast<uint2*>(a.out.p + (long long)t * a.out.ts + (long long)h * a.out.hs + q * 4) =
      make_uint2(pack2<kType>(o[0] * inv, o[1] * inv), pack2<kType>(o[2] * inv, o[3] * inv));
  if (a.lse && q == 0) a.lse[of.w] = l != 0.0f ? (top + (__log2f(l) - kRaise<kType>)) * 0.6931471805599453f : -INFINITY;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Boxes of 64 columns x box_heads x box_rows of [rows, heads, head_dim]. False
// where a tensor map cannot describe the tensor.
bool make_map(CUtensorMap* map, const Heads& h, int dtype, int head_dim, int heads, long long rows, int box_heads,
              int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode || !h.p || rows <= 0) return false;
  // a stride along one element says nothing
  const cuuint64_t hs = heads > 1 ? (cuuint64_t)h.hs * 2 : (cuuint64_t)head_dim * 2;
  const cuuint64_t ts = rows > 1 ? (cuuint64_t)h.ts * 2 : (cuuint64_t)head_dim * 2;
  if (hs == 0 || ts == 0 || hs >= (1ull << 40) || ts >= (1ull << 40)) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {hs, ts};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t steps[3] = {1, 1, 1};
  return encode(map, dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, h.p,
                dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kType, int DP>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t s) {
  cudaError_t err = cudaFuncSetAttribute(attention_kernel<kType, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Sizes<DP>::smem);
  if (err != cudaSuccess) return err;
  // no more CTAs than there can be items
  const int tpt = kTile / (a.heads_q / a.heads_kv);
  long long items = ((long long)a.total_q / (2 * tpt) + a.n) * a.heads_kv;
  if (a.part_o) items = items * kSplitItems;
  const int sms = num_sms();
  Maps maps = {};
  const int group = a.heads_q / a.heads_kv;
  auto whole = [](long long x) { return x % 16 == 0; };
  maps.wide = reinterpret_cast<uintptr_t>(a.out.p) % 32 == 0 && whole(a.head_dim) && whole(a.out.ts) && whole(a.out.hs);
  const long long rows = a.paged ? (long long)a.n_pages * a.page_size : a.total_k;
  maps.box = a.paged ? min(a.page_size & -a.page_size, kTile) : kTile;  // rows of a page that lie together
  maps.use = maps.box >= 8 && make_map(&maps.q, a.q, kType, a.head_dim, a.heads_q, a.total_q, group, tpt) &&
             make_map(&maps.k, a.k, kType, a.head_dim, a.heads_kv, rows, 1, maps.box) &&
             make_map(&maps.v, a.v, kType, a.head_dim, a.heads_kv, rows, 1, maps.box);
  err = launch_pdl(attention_kernel<kType, DP>, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads),
                   Sizes<DP>::smem, s, a, maps);
  if (err != cudaSuccess || !a.part_o) return err;
  const long long blocks = ((long long)a.total_q * a.heads_q + 7) / 8;
  return launch_pdl(join_kernel<kType>, dim3((unsigned)blocks), dim3(kJoinThreads), 0, s, a);
}

}  // namespace

AttnWs attention_ws(int n, int total_q, int heads_q, int heads_kv, int head_dim, long long max_keys) {
  AttnWs w = {};
  const long long blocks = (max_keys + kTile - 1) / kTile;
  const long long rows = (long long)total_q * heads_q;
  // one query tile pair: the most pieces
  const int most = blocks < 2 * kSplitMinBlocks || heads_kv >= kSplitItems ? 1 : pieces_within((int)blocks, heads_kv);
  if (most > 1 && rows > 0) {
    // a sequence of T pairs has at most 256 T heads_kv rows and, if it is cut,
    // T heads_kv < kSplitItems and at most kSplitItems / (T heads_kv) + 1 pieces
    const long long by_seq = (long long)n * 256 * 2 * kSplitItems;
    w.part_rows = rows * most;
    if (by_seq < w.part_rows) w.part_rows = by_seq;
    if (w.part_rows > 0x7fffffffLL) w.part_rows = 0;  // more than can be counted: nothing is cut
  }
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.o = 0;
  w.ml = up((size_t)w.part_rows * head_dim * sizeof(float));
  w.of = w.ml + up((size_t)w.part_rows * sizeof(float2));
  w.bytes = w.of + up(w.part_rows > 0 ? (size_t)rows * sizeof(int4) : 0);
  if (w.bytes < 256) w.bytes = 256;
  return w;
}

cudaError_t launch_attention(const AttnArgs& args, int dtype, cudaStream_t s) {
  AttnArgs a = args;
  a.group = a.heads_q / a.heads_kv;
  a.tile_tokens = kTile / a.group;
  if (dtype == MOE_BF16) return a.head_dim <= 64 ? launch_typed<MOE_BF16, 64>(a, s) : launch_typed<MOE_BF16, 128>(a, s);
  return a.head_dim <= 64 ? launch_typed<MOE_FP16, 64>(a, s) : launch_typed<MOE_FP16, 128>(a, s);
}

}  // namespace moe

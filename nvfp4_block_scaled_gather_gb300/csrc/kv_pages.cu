// Upkeep of a paged cache of keys and values: growing sequences (with copy of
// a shared open page), writing rows, forking, truncating, keeping drafted
// rows, copying and compacting pages.
//
// What bounds these: the tables are a few KB, so the planning is latency (one
// CTA, a handful of dependent reads), and the page data is a plain copy, bound
// by memory. So the planning kernels leave a list of page copies in the
// workspace and one copy kernel spreads the list's bytes over the whole GPU.
//
// Nothing read from device memory is followed as an index before it has been
// checked against its range.
#include <cstdint>

#include <cuda_runtime.h>

#include "attention_internal.h"
#include "internal.h"
#include "ldcg.cuh"
#include "mbar.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPiece = 16384;      // bytes of one unit of page copying
constexpr int kMovers = 4;         // warps that move units
constexpr int kSlots = 3;          // units that each holds in shared memory
constexpr int kAhead = 2;          // of them being read; the others are being written
constexpr int kCopyThreads = 256;  // the other warps go over the tables

struct Kv {
  uint8_t* pages;
  long long plane_bytes, page_bytes, row_bytes;
  int planes, n_pages, page_size;
  int *table, *length, *held, *refs;
  int max_seqs, max_pages;
};

Kv make_kv(const moe_kv_cache_t& c) {
  Kv k;
  k.pages = static_cast<uint8_t*>(c.pages);
  k.row_bytes = (long long)c.heads_kv * c.head_dim * 2;
  k.page_bytes = k.row_bytes * c.page_size;
  k.plane_bytes = k.page_bytes * c.n_pages;
  k.planes = c.planes;
  k.n_pages = c.n_pages;
  k.page_size = c.page_size;
  k.table = c.table;
  k.length = c.length;
  k.held = c.held;
  k.refs = c.refs;
  k.max_seqs = c.max_seqs;
  k.max_pages = c.max_pages;
  return k;
}

// The first thing found wrong stays until it is read.
__device__ __forceinline__ void report(int* status, int what) { atomicCAS(status, 0, what); }

// 16-byte aligned runs of bytes to shared memory (complete on the barrier) and
// back (one group each, of the thread that asks).
__device__ __forceinline__ void bulk_load(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(uint8_t* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// By a whole warp, the same answer in every lane; false after kWaitCycles.
__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity) {
  bool done = mbar_try_wait(bar, parity);
  for (const long long t0 = clock64(); !done && clock64() - t0 < kWaitCycles;) done = mbar_try_wait(bar, parity);
  return __all_sync(~0u, done);
}

__device__ __forceinline__ int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

// Exclusive sums over the CTA's threads (kPlanThreads of them) of N values at
// once, in place; total: the sums. Modulo 2^32.
template <int N>
__device__ void block_scan(int (&v)[N], int (&total)[N]) {
  __shared__ int part[N][kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kPlanThreads == 1024, "a lane for every warp's sum");
  int x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = v[e];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int y = __shfl_up_sync(~0u, x[e], o);
      if (lane >= o) x[e] = (int)((uint32_t)x[e] + (uint32_t)y);
    }
  if (lane == 31)
#pragma unroll
    for (int e = 0; e < N; ++e) part[e][warp] = x[e];
  __syncthreads();
  // every warp sums the warps' sums for itself
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const uint32_t mine = (uint32_t)part[e][lane];
    total[e] = (int)__reduce_add_sync(~0u, mine);
    v[e] = (int)((uint32_t)x[e] - (uint32_t)v[e] + __reduce_add_sync(~0u, lane < warp ? mine : 0u));
  }
  __syncthreads();
}

// A warp's share of the pool: a run of pages of its own, in groups of 32.
struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run run_of(int n_pages) {
  const int warps = kPlanThreads / 32, warp = threadIdx.x >> 5;
  const long long per = ((n_pages + kPlanThreads - 1) / kPlanThreads) * 32LL, lo = per * warp;
  static_assert(warps * 32 == kPlanThreads, "whole warps");
  return {(int)min(lo, (long long)n_pages), (int)min(lo + per, (long long)n_pages)};
}
// Bit l: page p + l of the run is in use. By a whole warp.
__device__ __forceinline__ uint32_t used_of(const int* refs, const Run& run, int p) {
  const int at = p + (threadIdx.x & 31);
  return __ballot_sync(~0u, at < run.hi && ld_cg(refs + at) != 0);
}

// Plans the growth of up to MOE_KV_MAX_CALL sequences in one CTA.
// want(i) = new pages of sequence i, its own copy of a shared open page first;
// off(i) = exclusive sum; the free page of rank r (ascending ids) goes to the
// sequence with off(i) <= r < off(i + 1). A sequence is the k-th of the call to
// share an open page: the refs it finds are those minus k (each before it has
// left for its own copy), so it copies while more than one remain.
//
// Latency bounds it, a chain of dependent reads of half a microsecond each. So
// a thread has one sequence of each 1024 (four in a row, one after the other,
// made it 14 us for 96 sequences; so it takes 6 us), and the pool is read
// before the sequences are compared. One CTA goes over the counts of the whole
// pool (twice if it is full) and compares the sequences pairwise: 6 us with a
// nearly full pool of 300 pages, 22 with 48,000 and 70 with 190,000 (32
// sequences); 16 us for 256 sequences, 38 for 1024 and 300 for 4096.
struct Growth {
  int seq[MOE_KV_MAX_CALL];
  int open[MOE_KV_MAX_CALL];     // the open page, or -1; then where its copy is in the list, or -1
  int off[MOE_KV_MAX_CALL + 1];
  int column[MOE_KV_MAX_CALL];   // of the table, where the first page wanted goes
};
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(Kv kv, const int* seqs, const int* add, int n,
                                                                   KvWs ws, int* status) {
  extern __shared__ int s_growth[];
  Growth& g = *reinterpret_cast<Growth*>(s_growth);
  constexpr int kPer = MOE_KV_MAX_CALL / kPlanThreads;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int need[kPer], refs[kPer], len[kPer], more[kPer], own[kPer];  // refs: of the open page
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * kPlanThreads + tid;
    need[u] = refs[u] = len[u] = more[u] = own[u] = 0;
    if (i >= n) continue;
    g.seq[i] = -1;
    g.open[i] = -1;
    const int s = ld_cg(seqs + i);
    const int a = ld_cg(add + i);
    if (s < 0 || s >= kv.max_seqs || a < 0) {
      bad = true;
      continue;
    }
    g.seq[i] = s;
    len[u] = ld_cg(kv.length + s);
    own[u] = ld_cg(kv.held + s);
    more[u] = a;
    const long long pages = ((long long)len[u] + a + kv.page_size - 1) / kv.page_size;
    if (len[u] < 0 || pages > kv.max_pages || own[u] != ceil_div(len[u], kv.page_size)) {
      bad = true;
      continue;
    }
    need[u] = (int)pages - own[u];
    if (a > 0 && len[u] % kv.page_size != 0) {
      const int p = ld_cg(kv.table + (long long)s * kv.max_pages + len[u] / kv.page_size);
      if (p < 0 || p >= kv.n_pages) {
        bad = true;
        continue;
      }
      g.open[i] = p;
      refs[u] = ld_cg(kv.refs + p);
    }
  }
  const Run run = run_of(kv.n_pages);
  int free_pages = 0;
#pragma unroll 4
  for (int p = run.lo; p < run.hi; p += 32) free_pages += min(32, run.hi - p) - __popc(used_of(kv.refs, run, p));
  __syncthreads();
  // a warp compares a sequence with those before it: listed twice? how many share its open page?
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    const int s = g.seq[i], p = g.open[i];
    int before = 0;
    for (int j = lane; j < i; j += 32) {
      bad |= g.seq[j] == s;
      before += g.open[j] == p ? 1 : 0;
    }
    before = __reduce_add_sync(~0u, before);
    if (lane == 0) g.off[i] = before;
  }
  if (tid == 0) *ws.count = 0;
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (tid == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  // The pages wanted can pass 32 bits (thousands of sequences of up to 2^30
  // each), so their multiples of 4096 are summed too: more of these than the
  // free pages have is more pages than there are, and with no more of them the
  // sum itself is below 2^30 + 2^24.
  int total = 0, copies = 0, high = 0, all_free = 0, first = 0;  // first: rank of the run's first free page
  int slot[kPer];                                      // in the list of copies, or -1
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * kPlanThreads + tid;
    slot[u] = -1;
    if (u * kPlanThreads >= n) continue;
    const bool copy = i < n && g.open[i] >= 0 && refs[u] - g.off[i] > 1;
    const int want = need[u] + (copy ? 1 : 0);
    int at[4] = {want, copy ? 1 : 0, u == 0 && lane == 0 ? free_pages : 0, want >> 12}, sums[4];
    block_scan(at, sums);
    if (i < n) {
      g.off[i] = (int)((uint32_t)total + (uint32_t)at[0]);
      g.column[i] = own[u] + need[u] - want;  // with a copy the open page's, before the new ones
    }
    if (copy) slot[u] = copies + at[1];
    if (u == 0) {
      first = __shfl_sync(~0u, at[2], 0);
      all_free = sums[2];
    }
    high += sums[3];
    if (high > all_free >> 12) break;  // (the same in every thread)
    total += sums[0];
    copies += sums[1];
  }
  if (high > all_free >> 12 || total > all_free) {
    if (tid == 0) report(status, MOE_ERR_PAGES);
    return;
  }
  // the lengths and the copies' sources; the sequences leave their shared open pages
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * kPlanThreads + tid;
    if (i >= n) continue;
    const int s = g.seq[i], open = g.open[i];
    kv.length[s] = len[u] + more[u];
    kv.held[s] = own[u] + need[u];
    g.open[i] = slot[u];
    if (slot[u] >= 0) {
      ws.src[slot[u]] = open;
      ws.rows[slot[u]] = len[u] % kv.page_size;
      atomicSub(kv.refs + open, 1);
    }
  }
  if (tid == 0) *ws.count = copies;
  __syncthreads();
  // every warp gives out the free pages of its run (a page's refs here only
  // fall from above 1 to at least 1, so a free page is still the same one)
  for (int p0 = run.lo; p0 < run.hi && first < total; p0 += 32) {
    const int p = p0 + lane;
    const uint32_t free = ~used_of(kv.refs, run, p0) & (run.hi - p0 < 32 ? (1u << (run.hi - p0)) - 1u : ~0u);
    const int rank = first + __popc(free & ((1u << lane) - 1u));
    first += __popc(free);
    if (!((free >> lane) & 1u) || rank >= total) continue;
    int lo = 0, hi = n;  // the last i with off(i) <= rank
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.off[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const int q = rank - g.off[lo];
    if (g.open[lo] >= 0 && q == 0) ws.dst[g.open[lo]] = p;
    kv.refs[p] = 1;
    kv.table[(long long)g.seq[lo] * kv.max_pages + g.column[lo] + q] = p;
  }
}

// Carries out a list of page copies in all planes. count: null (n entries) or
// their number on the device; rows: null for whole pages. check: the list is
// the caller's, its ids are checked here. With moved, the tables' page ids are
// replaced as well (compaction), by the other warps meanwhile.
//
// Memory bounds it: what it reads it writes once. A page goes in units of
// kPiece bytes through shared memory, by asynchronous copies; a warp looks up
// 32 units at a time, a lane each, so that the reads of the list do not stand
// between the units. 6.3 TB/s over 1300 MB of pages of 128 KB, 6.1 over pages
// of 4 KB (one moving warp with units of 32 KB: 6.3 and 3.4, its issuing lane
// is the limit; blocks of 256 threads that load and store 16 KB: 5.7 over
// large pages).
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(Kv kv, const int* src, const int* dst,
                                                                  const int* rows, const int* count, int n, int check,
                                                                  const int* moved, int* status) {
  extern __shared__ __align__(128) uint8_t s_units[];  // [kMovers][kSlots][kPiece]
  __shared__ uint64_t s_full[kMovers * kSlots];
  __shared__ unsigned long long s_to[kMovers * kSlots];
  __shared__ uint32_t s_bytes[kMovers * kSlots];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMovers * kSlots; ++i) mbar_init(smem_u32(s_full + i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int entries = count ? ld_cg(count) : n;
  if (warp >= kMovers) {
    if (!moved || entries <= 0) return;
    const long long cells = (long long)kv.max_seqs * kv.max_pages;
    constexpr int kOthers = kCopyThreads - 32 * kMovers;
    for (long long c = (long long)blockIdx.x * kOthers + threadIdx.x - 32 * kMovers; c < cells;
         c += (long long)gridDim.x * kOthers) {
      const int p = ld_cg(kv.table + c);
      if (p >= 0 && p < kv.n_pages) {
        const int q = ld_cg(moved + p);
        if (q != p) kv.table[c] = q;
      }
    }
    return;
  }
  const int pieces = (int)((kv.page_bytes + kPiece - 1) / kPiece);
  const long long all = (long long)entries * kv.planes * pieces;
  const uint32_t units = smem_u32(s_units) + warp * kSlots * kPiece, full = smem_u32(s_full + warp * kSlots);
  unsigned long long* const tos = s_to + warp * kSlots;
  uint32_t* const sizes = s_bytes + warp * kSlots;
  int begun = 0, ended = 0;  // units asked for, units given back
  bool ok = true;
  auto end_one = [&]() {
    const int i = ended % kSlots;
    ok = wait_full(full + 8 * i, (ended / kSlots) & 1);
    if (!ok) return;
    if (lane == 0) bulk_store(reinterpret_cast<uint8_t*>(tos[i]), units + i * kPiece, sizes[i]);
    ++ended;
  };
  const int movers = gridDim.x * kMovers;
  for (long long w0 = blockIdx.x * kMovers + warp; ok && w0 < all; w0 += 32LL * movers) {
    const long long w = w0 + (long long)lane * movers;
    unsigned long long from = 0, to = 0;
    uint32_t bytes = 0;
    if (w < all) {
      // all first pieces, then all second ones: of partly filled pages the later
      // ones are empty, and a grid that the pieces divide would give them all to
      // the same CTAs (96 forks: 52 us that way, 50 this way)
      const long long r = w / kv.planes;
      const int plane = (int)(w - r * kv.planes), piece = (int)(r / entries), i = (int)(r - (long long)piece * entries);
      const long long at = (long long)piece * kPiece;
      const int a = ld_cg(src + i), b = ld_cg(dst + i);
      const long long most = rows ? (long long)ld_cg(rows + i) * kv.row_bytes : kv.page_bytes;
      if (check && (a < 0 || a >= kv.n_pages || b < 0 || b >= kv.n_pages)) {
        report(status, MOE_ERR_INVALID);
      } else if (at < most && a != b) {
        const unsigned long long base = reinterpret_cast<unsigned long long>(kv.pages) + plane * kv.plane_bytes + at;
        from = base + a * kv.page_bytes;
        to = base + b * kv.page_bytes;
        bytes = (uint32_t)min((long long)kPiece, most - at);
      }
    }
    for (uint32_t left = __ballot_sync(~0u, bytes != 0); ok && left; left &= left - 1) {
      const int l = __ffs(left) - 1, i = begun % kSlots;
      const uint8_t* p = reinterpret_cast<const uint8_t*>(__shfl_sync(~0u, from, l));
      const unsigned long long q = __shfl_sync(~0u, to, l);
      const uint32_t size = __shfl_sync(~0u, bytes, l);
      if (lane == 0) {
        // of the begun - kAhead writes so far all but the last few have let go
        // of their slots: the one of unit begun - kSlots is among them
        asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kSlots - kAhead - 1) : "memory");
        tos[i] = q;
        sizes[i] = size;
        mbar_expect_tx(full + 8 * i, size);
        bulk_load(units + i * kPiece, p, size, full + 8 * i);
      }
      if (++begun > kAhead) end_one();
    }
  }
  while (ok && ended < begun) end_one();
  if (!ok) {
    // what is still on its way must land before the CTA may go
    if (lane == 0) report(status, MOE_ERR_TIMEOUT);
    for (; ended < begun; ++ended) wait_full(full + 8 * (ended % kSlots), (ended / kSlots) & 1);
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Compaction's plan in one CTA: U pages in use; the k-th used page from U on
// goes to the k-th free page before U (as many of the one as of the other). It
// goes over the pool's counts several times: with nothing to move the call takes 6
// us for 300 pages, 39 for 48,000 and 133 for 190,000.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Kv kv, KvWs ws) {
  pdl_wait();
  pdl_trigger();
  const Run run = run_of(kv.n_pages);
  const int lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  int used = 0;
#pragma unroll 4
  for (int p = run.lo; p < run.hi; p += 32) used += __popc(used_of(kv.refs, run, p));
  int count[1] = {lane == 0 ? used : 0}, all[1];
  block_scan(count, all);
  const int in_use = all[0];
  // bit l: page p + l of the run comes before page in_use
  auto front_of = [&](int p) {
    const int left = min(run.hi, in_use) - p;
    return left <= 0 ? 0u : left < 32 ? (1u << left) - 1u : ~0u;
  };
  int h = 0, m = 0;
#pragma unroll 4
  for (int p = run.lo; p < run.hi; p += 32) {
    const uint32_t busy = used_of(kv.refs, run, p), front = front_of(p);
    h += __popc(~busy & front);
    m += __popc(busy & ~front);
    if (p + lane < run.hi) ws.moved[p + lane] = p + lane;
  }
  int at[2] = {lane == 0 ? h : 0, lane == 0 ? m : 0}, sums[2];
  block_scan(at, sums);
  h = __shfl_sync(~0u, at[0], 0);
  m = __shfl_sync(~0u, at[1], 0);
  if (threadIdx.x == 0) *ws.count = sums[1];
  for (int p = run.lo; p < run.hi && p < in_use; p += 32) {
    const uint32_t hole = ~used_of(kv.refs, run, p) & front_of(p);
    if ((hole >> lane) & 1u) ws.dst[h + __popc(hole & below)] = p + lane;
    h += __popc(hole);
  }
  __syncthreads();
  for (int p = run.lo; p < run.hi; p += 32) {
    const uint32_t mover = used_of(kv.refs, run, p) & ~front_of(p);
    if ((mover >> lane) & 1u) {
      const int from = p + lane, k = m + __popc(mover & below);
      const int to = ld_cg(ws.dst + k), refs = ld_cg(kv.refs + from);
      ws.src[k] = from;
      ws.moved[from] = to;
      kv.refs[to] = refs;
      kv.refs[from] = 0;
    }
    m += __popc(mover);
  }
}

// One warp per row: both of its planes' rows, 16 bytes a lane. A row's place is
// found by a chain of dependent reads, so its values are asked for first, and
// its sequence is searched for with 32 probes at a time.
__global__ void __launch_bounds__(256) append_kernel(Kv kv, int layer, const int* seqs, const int* cu, int n, int total,
                                                     Heads k, Heads v, int heads, int head_dim, int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int per_head = head_dim / 8, chunks = heads * per_head;
  constexpr int kHeld = 4;  // chunks a lane that are asked for ahead
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < total; t += gridDim.x * 8) {
    uint4 a[kHeld], b[kHeld];
    auto load = [&](int c, uint4& x, uint4& y) {
      const int head = c / per_head, e = (c - head * per_head) * 8;
      x = ld_cg(reinterpret_cast<const uint4*>(k.p + t * k.ts + head * k.hs + e));
      y = ld_cg(reinterpret_cast<const uint4*>(v.p + t * v.ts + head * v.hs + e));
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (lane + 32 * j < chunks) load(lane + 32 * j, a[j], b[j]);
    const int last = ld_cg(cu + n);
    int lo = 0, hi = n;  // the last i with cu[i] <= t
    bool inside = n > 0 && t < last;
    while (hi > lo) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const uint32_t up_to = __ballot_sync(~0u, at < hi && ld_cg(cu + at) <= t);
      if (!up_to) inside = false;  // before the first
      const int i = up_to ? 31 - __clz(up_to) : 0;
      lo += i * step;
      hi = min(lo + step, hi);
      if (step == 1) break;
    }
    if (!inside) continue;
    const int s = ld_cg(seqs + lo), end = ld_cg(cu + lo + 1);
    bool ok = s >= 0 && s < kv.max_seqs && t < end;
    long long row = 0;
    if (ok) {
      const long long at = (long long)ld_cg(kv.length + s) - (end - t);
      ok = at >= 0 && at / kv.page_size < kv.max_pages;
      if (ok) {
        const int p = ld_cg(kv.table + (long long)s * kv.max_pages + at / kv.page_size);
        ok = p >= 0 && p < kv.n_pages && ld_cg(kv.refs + p) == 1;
        row = (long long)p * kv.page_size + at % kv.page_size;
      }
    }
    if (!ok) {
      if (lane == 0) report(status, MOE_ERR_INVALID);
      continue;
    }
    uint8_t* to = kv.pages + 2LL * layer * kv.plane_bytes + row * kv.row_bytes;
    auto store = [&](int c, const uint4& x, const uint4& y) {
      reinterpret_cast<uint4*>(to)[c] = x;
      reinterpret_cast<uint4*>(to + kv.plane_bytes)[c] = y;
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (lane + 32 * j < chunks) store(lane + 32 * j, a[j], b[j]);
    for (int c = lane + 32 * kHeld; c < chunks; c += 32) {
      uint4 x, y;
      load(c, x, y);
      store(c, x, y);
    }
  }
}

// One CTA per pair.
__global__ void __launch_bounds__(128) fork_kernel(Kv kv, const int* src, const int* dst, int n, int* status) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int a = ld_cg(src + i), b = ld_cg(dst + i);
  bool bad = a < 0 || a >= kv.max_seqs || b < 0 || b >= kv.max_seqs;
  if (!bad) {
    for (int j = threadIdx.x; j < n; j += 128) bad |= (j < i && ld_cg(dst + j) == b) || ld_cg(src + j) == b;
  }
  // (a repeated dst is taken by its first pair: the later ones stop here, and
  // only a dst that no other CTA writes is read below)
  if (!__syncthreads_or(bad ? 1 : 0)) bad = ld_cg(kv.held + b) != 0 || ld_cg(kv.length + b) != 0;
  else bad = true;
  int held = 0, length = 0;
  if (!bad) {
    held = ld_cg(kv.held + a);
    length = ld_cg(kv.length + a);
    bad = held < 0 || held > kv.max_pages;
  }
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (threadIdx.x == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  for (int c = threadIdx.x; c < kv.max_pages; c += 128) {
    const int p = c < held ? ld_cg(kv.table + (long long)a * kv.max_pages + c) : -1;
    kv.table[(long long)b * kv.max_pages + c] = p;
    if (p >= 0 && p < kv.n_pages) atomicAdd(kv.refs + p, 1);
  }
  if (threadIdx.x == 0) {
    kv.held[b] = held;
    kv.length[b] = length;
  }
}

// One CTA per sequence.
__global__ void __launch_bounds__(128) truncate_kernel(Kv kv, const int* seqs, const int* new_len, int n, int* status) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int s = ld_cg(seqs + i), to = ld_cg(new_len + i);
  bool bad = s < 0 || s >= kv.max_seqs || to < 0;
  for (int j = threadIdx.x; j < i; j += 128) bad |= ld_cg(seqs + j) == s;  // repeats: the first one counts
  int length = 0, held = 0;
  if (!bad) {
    length = min(ld_cg(kv.length + s), to);
    held = min(ld_cg(kv.held + s), kv.max_pages);
    bad = length < 0 || held < 0;  // of no sequence: its columns would lie before the table's row
  }
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (threadIdx.x == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  const int stay = min(ceil_div(length, kv.page_size), held);
  for (int c = stay + threadIdx.x; c < held; c += 128) {
    int* cell = kv.table + (long long)s * kv.max_pages + c;
    const int p = ld_cg(cell);
    if (p >= 0 && p < kv.n_pages) atomicSub(kv.refs + p, 1);
    *cell = -1;
  }
  __syncthreads();  // every thread has read length and held
  if (threadIdx.x == 0) {
    kv.length[s] = length;
    kv.held[s] = stay;
  }
}

// Moves the kept drafted rows together. One CTA per (sequence, plane, 2 KB of
// the row); a thread owns 16 bytes of every row. Destination j never comes
// after source keep[j], and sources ascend, so a thread that takes the rows in
// order reads every source before it is overwritten: rows j .. j + 3 are read
// before they are written, which keeps that.
constexpr int kKeepThreads = 128;
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(Kv kv, const int* seqs, const int* drafted, const int* keep,
                                                            int max_keep, const int* kept, int n, int* new_len,
                                                            int* status) {
  __shared__ long long s_src[kKeepThreads], s_dst[kKeepThreads];  // byte offsets in a plane
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int* row = keep + (long long)i * max_keep;
  const int mine = tid < max_keep ? ld_cg(row + tid) : 0;
  const int s = ld_cg(seqs + i), m = ld_cg(drafted + i), k = ld_cg(kept + i);
  bool bad = s < 0 || s >= kv.max_seqs || m < 0 || k < 0 || k > m || k > max_keep;
  for (int j = tid; j < i; j += kKeepThreads) bad |= ld_cg(seqs + j) == s;
  int length = 0, start = 0;
  auto offset = [&](int pos) -> long long {
    const int p = ld_cg(kv.table + (long long)s * kv.max_pages + pos / kv.page_size);
    return ((long long)p * kv.page_size + pos % kv.page_size) * kv.row_bytes;
  };
  if (!bad) {
    length = ld_cg(kv.length + s);
    bad = length < m || ceil_div(length, kv.page_size) > kv.max_pages;  // (m >= 0, so no length below 0 passes)
    start = bad ? 0 : length - m;
  }
  if (!bad) {
    for (int j = tid; j < k; j += kKeepThreads) {
      const int x = j == tid ? mine : ld_cg(row + j);
      const bool out = x < 0 || x >= m;
      if (j == tid && !out) {  // the first rows' places (of no use if a page turns out to be bad)
        s_src[tid] = offset(start + x);
        s_dst[tid] = offset(start + tid);
      }
      bad |= out || (j > 0 && ld_cg(row + j - 1) >= x);
    }
    if (k > 0)
      for (int c = start / kv.page_size + tid; c < ceil_div(length, kv.page_size); c += kKeepThreads) {
        const int p = ld_cg(kv.table + (long long)s * kv.max_pages + c);
        bad |= p < 0 || p >= kv.n_pages || ld_cg(kv.refs + p) != 1;
      }
  }
  bad = __syncthreads_or(bad ? 1 : 0) != 0;
  if (tid == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    new_len[i] = bad ? 0x7fffffff : start + k;  // nothing is cut off a sequence that is left alone
    if (bad) report(status, MOE_ERR_INVALID);
  }
  if (bad) return;
  uint8_t* plane = kv.pages + blockIdx.y * kv.plane_bytes;
  const long long byte = ((long long)blockIdx.z * kKeepThreads + tid) * 16;
  for (int j0 = 0; j0 < k; j0 += kKeepThreads) {
    const int count = min(kKeepThreads, k - j0);
    if (j0 > 0) {
      __syncthreads();
      if (tid < count) {
        s_src[tid] = offset(start + ld_cg(row + j0 + tid));
        s_dst[tid] = offset(start + j0 + tid);
      }
      __syncthreads();
    }
    if (byte >= kv.row_bytes) continue;
    for (int j = 0; j < count; j += 4) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j + u < count) v[u] = ld_cg(reinterpret_cast<const uint4*>(plane + s_src[j + u] + byte));
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j + u < count && s_src[j + u] != s_dst[j + u])
          *reinterpret_cast<uint4*>(plane + s_dst[j + u] + byte) = v[u];
    }
  }
}

// One CTA per sequence. A token's bits are its own and its parent's: all
// tokens at once take over the bits of the token that they point to and then
// point where that one points, so the line walked doubles each round (a walk
// up the parents one by one waits for a read each time: 12 us for trees of 64).
constexpr int kTreeThreads = 256;
constexpr int kTreeMost = 256, kTreeWords = kTreeMost / 32;  // larger trees are walked
__global__ void __launch_bounds__(kTreeThreads) tree_mask_kernel(const int* parents, const int* cu, int n, int total,
                                                                 int* mask, int words, int* status) {
  __shared__ uint32_t s_bits[2][kTreeMost * kTreeWords];
  __shared__ int s_up[2][kTreeMost];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int first = ld_cg(cu + blockIdx.x), end = min(ld_cg(cu + blockIdx.x + 1), total);
  if (first < 0 || end <= first) {
    if (first < 0 && tid == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  const int m = end - first;
  const int* from = parents + first;
  int* rows = mask + (long long)first * words;
  if (m > 32LL * words) {
    if (tid == 0) report(status, MOE_ERR_INVALID);
    for (long long x = tid; x < (long long)m * words; x += kTreeThreads) rows[x] = 0;
    return;
  }
  auto up_of = [&](int j) {  // an earlier token, or -1
    const int up = ld_cg(from + j);
    if (up >= -1 && up < j) return up;
    report(status, MOE_ERR_INVALID);
    return -1;
  };
  if (m <= kTreeMost) {
    const int used = (m + 31) / 32;
    if (tid < m) s_up[0][tid] = up_of(tid);
    for (int x = tid; x < m * used; x += kTreeThreads) {
      const int i = x / used, w = x - i * used;
      s_bits[0][x] = w == (i >> 5) ? 1u << (i & 31) : 0u;
    }
    __syncthreads();
    int now = 0;
    for (int reach = 1; reach < m; reach *= 2, now ^= 1) {
      for (int x = tid; x < m * used; x += kTreeThreads) {
        const int i = x / used, up = s_up[now][i];
        s_bits[now ^ 1][x] = s_bits[now][x] | (up >= 0 ? s_bits[now][x + (up - i) * used] : 0u);
      }
      if (tid < m) {
        const int up = s_up[now][tid];
        s_up[now ^ 1][tid] = up >= 0 ? s_up[now][up] : -1;
      }
      __syncthreads();
    }
    for (int x = tid; x < m * words; x += kTreeThreads) {
      const int i = x / words, w = x - i * words;
      rows[x] = w < used ? (int)s_bits[now][i * used + w] : 0;
    }
    return;
  }
  for (int i = tid; i < m; i += kTreeThreads) {
    int* row = rows + (long long)i * words;
    for (int w = 0; w < words; ++w) row[w] = 0;
    for (int j = i; j >= 0; j = up_of(j)) row[j >> 5] |= (int)(1u << (j & 31));
  }
}

cudaError_t launch_copy(const Kv& kv, long long entries, const int* src, const int* dst, const int* rows,
                        const int* count, int n, int check, const int* moved, int* status, cudaStream_t s) {
  const int smem = kMovers * kSlots * kPiece;
  const cudaError_t err = cudaFuncSetAttribute(copy_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const long long units = entries * kv.planes * ((kv.page_bytes + kPiece - 1) / kPiece), most = num_sms();
  // (few units: a CTA for each, so that they are in flight all over the GPU)
  const int grid = (int)(units < 1 ? 1 : units < most ? units : most);
  return launch_pdl(copy_pages_kernel, dim3(grid), dim3(kCopyThreads), smem, s, kv, src, dst, rows, count, n, check,
                    moved, status);
}

}  // namespace

KvWs kv_carve(void* base, const moe_kv_cache_t& c) {
  KvWs w;
  size_t off = 0;
  auto take = [&](size_t ints) {
    int* p = base ? reinterpret_cast<int*>(static_cast<uint8_t*>(base) + off) : nullptr;
    off += (ints * sizeof(int) + 255) & ~size_t(255);
    return p;
  };
  const size_t m = (size_t)kv_ws_entries(c);
  w.count = take(1);
  w.src = take(m);
  w.dst = take(m);
  w.rows = take(m);
  w.moved = take((size_t)c.n_pages);
  w.bytes = off;
  return w;
}

cudaError_t launch_kv_extend(const moe_kv_cache_t& c, const int* seqs, const int* add, int n, const KvWs& ws,
                             int* status, cudaStream_t s) {
  const Kv kv = make_kv(c);
  const size_t smem = sizeof(Growth);
  cudaError_t err = cudaFuncSetAttribute(extend_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  err = launch_pdl(extend_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, kv, seqs, add, n, ws, status);
  if (err != cudaSuccess) return err;
  return launch_copy(kv, n, ws.src, ws.dst, ws.rows, ws.count, 0, 0, nullptr, status, s);
}

cudaError_t launch_kv_append(const moe_kv_cache_t& c, int layer, const int* seqs, const int* cu, int n, int total,
                             const Heads& k, const Heads& v, int* status, cudaStream_t s) {
  const int blocks = (total + 7) / 8, most = num_sms() * 8;
  return launch_pdl(append_kernel, dim3(blocks < most ? blocks : most), dim3(256), 0, s, make_kv(c), layer, seqs, cu, n,
                    total, k, v, c.heads_kv, c.head_dim, status);
}

cudaError_t launch_kv_fork(const moe_kv_cache_t& c, const int* src, const int* dst, int n, int* status,
                           cudaStream_t s) {
  return launch_pdl(fork_kernel, dim3(n), dim3(128), 0, s, make_kv(c), src, dst, n, status);
}

cudaError_t launch_kv_truncate(const moe_kv_cache_t& c, const int* seqs, const int* new_len, int n, int* status,
                               cudaStream_t s) {
  return launch_pdl(truncate_kernel, dim3(n), dim3(128), 0, s, make_kv(c), seqs, new_len, n, status);
}

cudaError_t launch_kv_keep(const moe_kv_cache_t& c, const int* seqs, const int* drafted, const int* keep, int max_keep,
                           const int* kept, int n, const KvWs& ws, int* status, cudaStream_t s) {
  const Kv kv = make_kv(c);
  const dim3 grid(n, kv.planes, (unsigned)((kv.row_bytes / 16 + kKeepThreads - 1) / kKeepThreads));
  const cudaError_t err = launch_pdl(keep_kernel, grid, dim3(kKeepThreads), 0, s, kv, seqs, drafted, keep, max_keep,
                                     kept, n, ws.src, status);
  if (err != cudaSuccess) return err;
  // the bad ones' length is left as it is: what is wrong with them is reported already
  return launch_pdl(truncate_kernel, dim3(n), dim3(128), 0, s, kv, seqs, (const int*)ws.src, n, status);
}

cudaError_t launch_kv_copy_pages(const moe_kv_cache_t& c, const int* src, const int* dst, int n, int* status,
                                 cudaStream_t s) {
  return launch_copy(make_kv(c), n, src, dst, nullptr, nullptr, n, 1, nullptr, status, s);
}

cudaError_t launch_kv_compact(const moe_kv_cache_t& c, const KvWs& ws, int* status, cudaStream_t s) {
  const Kv kv = make_kv(c);
  const cudaError_t err = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, kv, ws);
  if (err != cudaSuccess) return err;
  return launch_copy(kv, c.n_pages, ws.src, ws.dst, nullptr, ws.count, 0, 0, ws.moved, status, s);
}

cudaError_t launch_tree_mask(const int* parents, const int* cu, int n, int total, int* mask, int words, int* status,
                             cudaStream_t s) {
  return launch_pdl(tree_mask_kernel, dim3(n), dim3(kTreeThreads), 0, s, parents, cu, n, total, mask, words,
                    status);
}

}  // namespace moe

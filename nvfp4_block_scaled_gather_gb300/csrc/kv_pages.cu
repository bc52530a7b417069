// Upkeep of a paged cache of keys and values: growing sequences (with copy of
// a shared open page), writing rows, forking, truncating, keeping drafted
// rows, copying and compacting pages.
//
// What bounds these: the tables are a few KB, so the planning is latency (one
// CTA, a handful of dependent reads), and the page data is a plain copy. So
// the planning kernels leave a list of page copies in the workspace and one
// copy kernel spreads the list's bytes over the whole GPU.
//
// Nothing read from device memory is followed as an index before it has been
// checked against its range.
#include <cstdint>

#include <cuda_runtime.h>

#include "attention_internal.h"
#include "internal.h"
#include "ldcg.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPiece = 16384;      // bytes of one unit of page copying
constexpr int kCopyThreads = 256;  // 64 bytes a thread and unit: four 16-byte loads in flight

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

__device__ __forceinline__ int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

// Exclusive sum over the CTA's threads (kPlanThreads of them); total: the sum.
__device__ int block_scan(int v, int& total) {
  __shared__ int part[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int p = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  const int before = warp ? part[warp - 1] : 0;
  total = part[kPlanThreads / 32 - 1];
  __syncthreads();
  return before + x - v;
}

// A thread's share of the pool: a run of pages of its own.
struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run run_of(int n_pages) {
  const int per = (n_pages + kPlanThreads - 1) / kPlanThreads;
  const long long lo = (long long)per * threadIdx.x;
  return {(int)min(lo, (long long)n_pages), (int)min(lo + per, (long long)n_pages)};
}

// Plans the growth of up to MOE_KV_MAX_CALL sequences in one CTA.
// want(i) = new pages of sequence i, its own copy of a shared open page first;
// off(i) = exclusive sum; the free page of rank r (ascending ids) goes to the
// sequence with off(i) <= r < off(i + 1). A sequence is the k-th of the call to
// share an open page: the refs it finds are those minus k (each before it has
// left for its own copy), so it copies while more than one remain.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(Kv kv, const int* seqs, const int* add, int n,
                                                                   KvWs ws, int* status) {
  __shared__ int s_seq[MOE_KV_MAX_CALL];
  __shared__ int s_page[MOE_KV_MAX_CALL];     // the open page, or -1
  extern __shared__ int s_off[];              // [MOE_KV_MAX_CALL + 1]
  constexpr int kPer = MOE_KV_MAX_CALL / kPlanThreads;
  static_assert(kPer == 4, "the sum of cow[] below");
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // thread tid plans sequences kPer * tid .. (so that the scan keeps their order)
  int need[kPer], cow[kPer], len[kPer], more[kPer], own[kPer];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid * kPer + u;
    need[u] = cow[u] = len[u] = more[u] = own[u] = 0;
    if (i >= n) continue;
    s_seq[i] = -1;
    s_page[i] = -1;
    const int s = ld_cg(seqs + i);
    const int a = ld_cg(add + i);
    if (s < 0 || s >= kv.max_seqs || a < 0) {
      bad = true;
      continue;
    }
    s_seq[i] = s;
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
      s_page[i] = p;
    }
  }
  __syncthreads();
  int want = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid * kPer + u;
    if (i >= n || bad) continue;
    const int s = s_seq[i], p = s_page[i];
    int before = 0;
    for (int j = 0; j < i; ++j) {
      bad |= s_seq[j] == s;
      before += (p >= 0 && s_page[j] == p) ? 1 : 0;
    }
    cow[u] = p >= 0 && ld_cg(kv.refs + p) - before > 1 ? 1 : 0;
    want += need[u] + cow[u];
  }
  if (tid == 0) *ws.count = 0;
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (tid == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  int total, copies;
  int off = block_scan(want, total);
  int slot = block_scan(cow[0] + cow[1] + cow[2] + cow[3], copies);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    s_off[tid * kPer + u] = off;
    off += need[u] + cow[u];
  }
  if (tid == kPlanThreads - 1) s_off[MOE_KV_MAX_CALL] = off;
  const Run run = run_of(kv.n_pages);
  int mine = 0, all_free;
  for (int p = run.lo; p < run.hi; ++p) mine += ld_cg(kv.refs + p) == 0 ? 1 : 0;
  int rank = block_scan(mine, all_free);
  if (total > all_free) {
    if (tid == 0) report(status, MOE_ERR_PAGES);
    return;
  }
  // the lengths and the copies' sources; the sequences leave their shared open pages
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid * kPer + u;
    if (i >= n) continue;
    const int s = s_seq[i];
    kv.length[s] = len[u] + more[u];
    kv.held[s] = own[u] + need[u];
    const int open = s_page[i];
    s_page[i] = -1;  // from here on: where sequence i's copy is in the list, or -1
    if (cow[u]) {
      ws.src[slot] = open;
      ws.rows[slot] = len[u] % kv.page_size;
      s_page[i] = slot++;
      atomicSub(kv.refs + open, 1);
    }
  }
  if (tid == 0) *ws.count = copies;
  __syncthreads();
  // every thread gives out the free pages of its run (a page's refs here only
  // fall from above 1 to at least 1, so a free page is still the same one)
  for (int p = run.lo; p < run.hi && rank < total; ++p) {
    if (ld_cg(kv.refs + p) != 0) continue;
    int lo = 0, hi = n;  // the last i with off(i) <= rank
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid] <= rank) lo = mid;
      else hi = mid;
    }
    const int s = s_seq[lo], q = rank - s_off[lo], wanted = s_off[lo + 1] - s_off[lo];
    // the last columns of the grown sequence; with a copy the first page is
    // the open one's column, which is the one before the new ones
    const int column = ld_cg(kv.held + s) - wanted + q;
    if (s_page[lo] >= 0 && q == 0) ws.dst[s_page[lo]] = p;
    kv.refs[p] = 1;
    kv.table[(long long)s * kv.max_pages + column] = p;
    ++rank;
  }
}

// One unit of page copying: kPiece bytes (or the rest) of `bytes` at src and dst.
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, long long at, long long bytes) {
  const long long left = min((long long)kPiece, bytes - at);
  const uint4* from = reinterpret_cast<const uint4*>(src + at);
  uint4* to = reinterpret_cast<uint4*>(dst + at);
  const int count = (int)(left / 16);
  uint4 v[kPiece / 16 / kCopyThreads];
#pragma unroll
  for (int j = 0; j < kPiece / 16 / kCopyThreads; ++j) {
    const int c = threadIdx.x + j * kCopyThreads;
    if (c < count) v[j] = ld_cg(from + c);
  }
#pragma unroll
  for (int j = 0; j < kPiece / 16 / kCopyThreads; ++j) {
    const int c = threadIdx.x + j * kCopyThreads;
    if (c < count) to[c] = v[j];
  }
}

// Carries out a list of page copies in all planes. count: null (n entries) or
// their number on the device; rows: null for whole pages. check: the list is
// the caller's, its ids are checked here. With moved, the tables' page ids are
// replaced as well (compaction).
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(Kv kv, const int* src, const int* dst,
                                                                  const int* rows, const int* count, int n, int check,
                                                                  const int* moved, int* status) {
  pdl_wait();
  pdl_trigger();
  const int entries = count ? ld_cg(count) : n;
  const int pieces = (int)((kv.page_bytes + kPiece - 1) / kPiece);
  const long long per = (long long)kv.planes * pieces;
  for (long long w = blockIdx.x; w < entries * per; w += gridDim.x) {
    const int i = (int)(w / per);
    const int r = (int)(w - i * per);
    const int plane = r / pieces, piece = r - plane * pieces;
    const int a = ld_cg(src + i);
    const int b = ld_cg(dst + i);
    if (check && (a < 0 || a >= kv.n_pages || b < 0 || b >= kv.n_pages)) {
      if (threadIdx.x == 0) report(status, MOE_ERR_INVALID);
      continue;
    }
    const long long bytes = rows ? (long long)ld_cg(rows + i) * kv.row_bytes : kv.page_bytes;
    const long long at = (long long)piece * kPiece;
    if (at >= bytes || a == b) continue;
    uint8_t* plane_at = kv.pages + plane * kv.plane_bytes;
    copy_piece(plane_at + a * kv.page_bytes, plane_at + b * kv.page_bytes, at, bytes);
  }
  if (moved && entries > 0) {
    const long long cells = (long long)kv.max_seqs * kv.max_pages;
    for (long long c = (long long)blockIdx.x * kCopyThreads + threadIdx.x; c < cells;
         c += (long long)gridDim.x * kCopyThreads) {
      const int p = ld_cg(kv.table + c);
      if (p >= 0 && p < kv.n_pages) {
        const int q = ld_cg(moved + p);
        if (q != p) kv.table[c] = q;
      }
    }
  }
}

// Compaction's plan in one CTA: U pages in use; the k-th used page from U on
// goes to the k-th free page before U (as many of the one as of the other).
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Kv kv, KvWs ws) {
  pdl_wait();
  pdl_trigger();
  const Run run = run_of(kv.n_pages);
  int used = 0, in_use, holes, movers;
  for (int p = run.lo; p < run.hi; ++p) used += ld_cg(kv.refs + p) != 0 ? 1 : 0;
  block_scan(used, in_use);
  int h = 0, m = 0;
  for (int p = run.lo; p < run.hi; ++p) {
    const bool busy = ld_cg(kv.refs + p) != 0;
    h += !busy && p < in_use ? 1 : 0;
    m += busy && p >= in_use ? 1 : 0;
    ws.moved[p] = p;
  }
  h = block_scan(h, holes);
  m = block_scan(m, movers);
  if (threadIdx.x == 0) *ws.count = movers;
  for (int p = run.lo; p < run.hi && p < in_use; ++p)
    if (ld_cg(kv.refs + p) == 0) ws.dst[h++] = p;
  __syncthreads();
  for (int p = max(run.lo, in_use); p < run.hi; ++p) {
    const int refs = ld_cg(kv.refs + p);
    if (refs == 0) continue;
    const int to = ld_cg(ws.dst + m);
    ws.src[m++] = p;
    ws.moved[p] = to;
    kv.refs[to] = refs;
    kv.refs[p] = 0;
  }
}

// One warp per row: both of its planes' rows, 16 bytes a lane.
__global__ void __launch_bounds__(256) append_kernel(Kv kv, int layer, const int* seqs, const int* cu, int n, int total,
                                                     Heads k, Heads v, int heads, int head_dim, int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int per_head = head_dim / 8, chunks = heads * per_head;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < total; t += gridDim.x * 8) {
    if (t < ld_cg(cu) || t >= ld_cg(cu + n)) continue;
    int lo = 0, hi = n;  // the last i with cu[i] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ld_cg(cu + mid) <= t) lo = mid;
      else hi = mid;
    }
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
    for (int c = lane; c < chunks; c += 32) {
      const int head = c / per_head, e = (c - head * per_head) * 8;
      const uint4 a = ld_cg(reinterpret_cast<const uint4*>(k.p + t * k.ts + head * k.hs + e));
      const uint4 b = ld_cg(reinterpret_cast<const uint4*>(v.p + t * v.ts + head * v.hs + e));
      reinterpret_cast<uint4*>(to)[c] = a;
      reinterpret_cast<uint4*>(to + kv.plane_bytes)[c] = b;
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
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (threadIdx.x == 0) report(status, MOE_ERR_INVALID);
    return;
  }
  const int length = min(ld_cg(kv.length + s), to);
  const int held = min(ld_cg(kv.held + s), kv.max_pages);
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
  const int s = ld_cg(seqs + i), m = ld_cg(drafted + i), k = ld_cg(kept + i);
  bool bad = s < 0 || s >= kv.max_seqs || m < 0 || k < 0 || k > m || k > max_keep;
  for (int j = tid; j < i; j += kKeepThreads) bad |= ld_cg(seqs + j) == s;
  int length = 0, start = 0;
  const int* row = keep + (long long)i * max_keep;
  if (!bad) {
    length = ld_cg(kv.length + s);
    start = length - m;
    bad = start < 0 || ceil_div(length, kv.page_size) > kv.max_pages;
  }
  if (!bad) {
    for (int j = tid; j < k; j += kKeepThreads) {
      const int x = ld_cg(row + j);
      bad |= x < 0 || x >= m || (j > 0 && ld_cg(row + j - 1) >= x);
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
  auto offset = [&](int pos) -> long long {
    const int p = ld_cg(kv.table + (long long)s * kv.max_pages + pos / kv.page_size);
    return ((long long)p * kv.page_size + pos % kv.page_size) * kv.row_bytes;
  };
  for (int j0 = 0; j0 < k; j0 += kKeepThreads) {
    const int count = min(kKeepThreads, k - j0);
    __syncthreads();
    if (tid < count) {
      s_src[tid] = offset(start + ld_cg(row + j0 + tid));
      s_dst[tid] = offset(start + j0 + tid);
    }
    __syncthreads();
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
  const int first = ld_cg(cu + blockIdx.x), end = min(ld_cg(cu + blockIdx.x + 1), total), m = end - first;
  if (first < 0 || m <= 0) {
    if (first < 0 && tid == 0) report(status, MOE_ERR_INVALID);
    return;
  }
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

int copy_grid(const Kv& kv, long long entries) {
  const long long units = entries * kv.planes * ((kv.page_bytes + kPiece - 1) / kPiece);
  const long long most = (long long)num_sms() * 8;
  return (int)(units < 1 ? 1 : units < most ? units : most);
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
  const size_t smem = (MOE_KV_MAX_CALL + 1) * sizeof(int);
  cudaError_t err = cudaFuncSetAttribute(extend_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  err = launch_pdl(extend_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, kv, seqs, add, n, ws, status);
  if (err != cudaSuccess) return err;
  return launch_pdl(copy_pages_kernel, dim3(copy_grid(kv, n)), dim3(kCopyThreads), 0, s, kv, (const int*)ws.src,
                    (const int*)ws.dst, (const int*)ws.rows, (const int*)ws.count, 0, 0, (const int*)nullptr, status);
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
  const Kv kv = make_kv(c);
  return launch_pdl(copy_pages_kernel, dim3(copy_grid(kv, n)), dim3(kCopyThreads), 0, s, kv, src, dst,
                    (const int*)nullptr, (const int*)nullptr, n, 1, (const int*)nullptr, status);
}

cudaError_t launch_kv_compact(const moe_kv_cache_t& c, const KvWs& ws, cudaStream_t s) {
  const Kv kv = make_kv(c);
  const cudaError_t err = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, kv, ws);
  if (err != cudaSuccess) return err;
  return launch_pdl(copy_pages_kernel, dim3(copy_grid(kv, c.n_pages)), dim3(kCopyThreads), 0, s, kv,
                    (const int*)ws.src, (const int*)ws.dst, (const int*)nullptr, (const int*)ws.count, 0, 0,
                    (const int*)ws.moved, (int*)nullptr);
}

cudaError_t launch_tree_mask(const int* parents, const int* cu, int n, int total, int* mask, int words, int* status,
                             cudaStream_t s) {
  return launch_pdl(tree_mask_kernel, dim3(n), dim3(kTreeThreads), 0, s, parents, cu, n, total, mask, words,
                    status);
}

}  // namespace moe

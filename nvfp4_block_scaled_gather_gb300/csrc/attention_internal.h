// Host-side launchers of the attention operators; arguments are validated by
// attention_api.cu before these are called.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "moe_attention.h"

namespace moe {

// Device address of the status word on the current device (moe_api.cu; looked
// up once per device), where kernels report what only they can see; null on a
// CUDA error.
int* status_ptr();

constexpr int kMaxGroup = 128;   // query heads per kv head
constexpr int kMaxHeadDim = 128;
constexpr int kMaxKeys = 0x7fffffff - 127;  // a place in the last block of 128 keys is still counted in 31 bits

// Rows of heads, 16-bit elements.
struct Heads {
  uint16_t* p;
  long long ts, hs;  // token and head strides, elements
};

// ------------------------------ pages (kv_pages.cu) ------------------------------
// Scratch of the upkeep calls, carved from the caller's workspace: a list of
// page copies, its count, and for compaction the new id of
// every page. keep uses new_len in the same place as src.
struct KvWs {
  int* count;   // copies in the list
  int* src;     // [entries]
  int* dst;     // [entries]
  int* rows;    // [entries] rows to copy
  int* moved;   // [n_pages]
  size_t bytes;
};
inline int kv_ws_entries(const moe_kv_cache_t& c) { return c.n_pages > c.max_seqs ? c.n_pages : c.max_seqs; }
KvWs kv_carve(void* base, const moe_kv_cache_t& c);

cudaError_t launch_kv_extend(const moe_kv_cache_t& c, const int* seqs, const int* add, int n, const KvWs& ws,
                             int* status, cudaStream_t s);
cudaError_t launch_kv_append(const moe_kv_cache_t& c, int layer, const int* seqs, const int* cu, int n, int total,
                             const Heads& k, const Heads& v, int* status, cudaStream_t s);
cudaError_t launch_kv_fork(const moe_kv_cache_t& c, const int* src, const int* dst, int n, int* status,
                           cudaStream_t s);
cudaError_t launch_kv_truncate(const moe_kv_cache_t& c, const int* seqs, const int* new_len, int n, int* status,
                               cudaStream_t s);
cudaError_t launch_kv_keep(const moe_kv_cache_t& c, const int* seqs, const int* drafted, const int* keep, int max_keep,
                           const int* kept, int n, const KvWs& ws, int* status, cudaStream_t s);
cudaError_t launch_kv_copy_pages(const moe_kv_cache_t& c, const int* src, const int* dst, int n, int* status,
                                 cudaStream_t s);
cudaError_t launch_kv_compact(const moe_kv_cache_t& c, const KvWs& ws, int* status, cudaStream_t s);
cudaError_t launch_tree_mask(const int* parents, const int* cu, int n, int total, int* mask, int words, int* status,
                             cudaStream_t s);

// ---------------------------- attention (attention.cu) ----------------------------
// How a sequence's keys are cut into pieces that are worked on by themselves
// (128 keys are a block). The cut goes by the sequence alone, so that its
// results do not depend on the call's other sequences. Many short pieces serve
// a lone sequence, few long ones a batch: against pieces of at least 4 blocks
// throughout, this rule takes 16.8 instead of 15.3 us for one stream over 4000
// keys and 83 instead of 88 for 32 streams over 500..6000, 42 instead of 51 for
// trees of 16 streams over 300..5000 (at least 8 blocks throughout: 17.7, 81, 42).
// pieces x heads x query tiles that one sequence is cut for: one a SM (the quotient is rounded up: fewer than twice as many)
constexpr int kSplitItems = 152;
constexpr int kSplitMinBlocks = 4;   // blocks of a piece at least ...
constexpr int kSplitFew = 6;         // ... of up to this many pieces; of more, twice as many blocks
struct Cut {
  int pieces, blocks;                // pieces of `blocks` blocks, the last one what is left
};
// The most pieces (a limit that only rises with the blocks).
__host__ __device__ inline int pieces_within(int blocks, int tiles_and_heads) {
  int most = blocks / kSplitMinBlocks;
  const int want = (kSplitItems + tiles_and_heads - 1) / tiles_and_heads;
  const int few = blocks / (2 * kSplitMinBlocks) > kSplitFew ? blocks / (2 * kSplitMinBlocks) : kSplitFew;
  if (few < most) most = few;
  return want < most ? want : most;
}
__host__ __device__ inline Cut cut_of(int blocks, int tiles_and_heads) {
  if (blocks < 2 * kSplitMinBlocks || tiles_and_heads >= kSplitItems) return {1, blocks};
  const int most = pieces_within(blocks, tiles_and_heads);
  const int per = (blocks + most - 1) / most;
  return {(blocks + per - 1) / per, per};
}

// One call: keys and values either packed rows (paged == 0: cu_k) or the
// planes of a paged cache.
struct AttnArgs {
  Heads q, k, v, out;
  float* lse;               // may be null
  const int* cu_q;          // [n + 1]
  const int* cu_k;          // [n + 1], packed rows
  int n, total_q, total_k;
  int heads_q, heads_kv, head_dim;
  float scale;
  // paged cache
  const int* seqs;          // [n]
  const int* table;
  const int* length;
  int paged, max_seqs, max_pages, n_pages, page_size;
  const int* mask;          // tree bits, or null (chain)
  int mask_words;
  int* status;
  int group, tile_tokens;   // filled in by the launch: query heads of a kv head, tokens of a tile of 128 rows
  // partial results of cut sequences (null: no sequence of the call is cut)
  float* part_o;            // [part_rows, head_dim], not divided by the sum
  float2* part_ml;          // [part_rows] maximum (in powers of two) and sum
  // [total_q * heads_q], a sequence's rows a kv head after the other: first partial row of the row's tile (or -1), the tile's
  // rows | the row in it << 8 | whether it sees any key << 16 | pieces << 17, rows between pieces, token * heads_q + head
  int4* part_of;
  long long part_rows;
};
// The partial rows that any call with these bounds can need, and their bytes.
struct AttnWs {
  long long part_rows;
  size_t o, ml, of, bytes;  // offsets and the total
};
AttnWs attention_ws(int n, int total_q, int heads_q, int heads_kv, int head_dim, long long max_keys);
cudaError_t launch_attention(const AttnArgs& a, int dtype, cudaStream_t s);

}  // namespace moe

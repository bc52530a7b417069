// C ABI of the attention operators (moe_attention.h): argument checks and
// launches. The kernels live in attention.cu and kv_pages.cu.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "attention_internal.h"
#include "internal.h"

namespace moe {
namespace {

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }
bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16; }

// A cache whose arrays and sizes can be used at all: MOE_OK, MOE_ERR_INVALID or MOE_ERR_SHAPE.
int cache_status(const moe_kv_cache_t* c) {
  if (!c || !c->pages || !c->table || !c->length || !c->held || !c->refs) return MOE_ERR_INVALID;
  if (misaligned(c->pages) || misaligned(c->table) || misaligned(c->length) || misaligned(c->held) ||
      misaligned(c->refs))
    return MOE_ERR_INVALID;
  if (c->planes <= 0 || c->n_pages <= 0 || c->page_size <= 0 || c->heads_kv <= 0 || c->head_dim <= 0 ||
      c->max_seqs <= 0 || c->max_pages <= 0 || !dtype_ok(c->dtype))
    return MOE_ERR_INVALID;
  if (c->planes % 2 || c->planes > 65534 || c->head_dim % 8) return MOE_ERR_SHAPE;
  // rows of a plane and tokens of a sequence are counted in 32 bits, a row in 1 GB
  if ((long long)c->n_pages * c->page_size > (1LL << 30) || (long long)c->max_pages * c->page_size > (1LL << 30) ||
      (long long)c->heads_kv * c->head_dim > (1LL << 29) || (long long)c->page_size * c->heads_kv * c->head_dim > (1LL << 30))
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

bool heads_ok(const moe_heads_t* h) {
  return h && h->data && !misaligned(h->data) && h->token_stride >= 0 && h->head_stride >= 0 &&
         h->token_stride % 8 == 0 && h->head_stride % 8 == 0;
}

Heads make_heads(const moe_heads_t& h) { return {static_cast<uint16_t*>(h.data), h.token_stride, h.head_stride}; }

// What both attention calls ask of their shapes.
int attention_status(int n, int total_q, int heads_q, int heads_kv, int head_dim, float scale) {
  if (n < 0 || total_q < 0 || heads_q <= 0 || heads_kv <= 0 || head_dim <= 0) return MOE_ERR_INVALID;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return MOE_ERR_INVALID;
  if (head_dim % 8 || head_dim > kMaxHeadDim || heads_q % heads_kv || heads_q / heads_kv > kMaxGroup)
    return MOE_ERR_SHAPE;
  if ((long long)total_q * heads_q > (1LL << 30)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int upkeep_status(const moe_kv_cache_t* c, int n) {
  const int st = cache_status(c);
  if (st != MOE_OK) return st;
  return n < 0 || n > MOE_KV_MAX_CALL ? MOE_ERR_INVALID : MOE_OK;
}

int workspace_status(const void* ws, size_t have, size_t need) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return MOE_ERR_INVALID;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_workspace_size(const moe_kv_cache_t* cache) {
  return cache_status(cache) == MOE_OK ? kv_carve(nullptr, *cache).bytes : 0;
}

int moe_kv_extend(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* add, int n, void* workspace,
                  size_t ws_bytes, cudaStream_t stream) {
  int st = upkeep_status(cache, n);
  if (st != MOE_OK || n == 0) return st;
  if (!seqs || !add) return MOE_ERR_INVALID;
  const KvWs ws = kv_carve(workspace, *cache);
  if ((st = workspace_status(workspace, ws_bytes, ws.bytes)) != MOE_OK) return st;
  if (n > cache->max_seqs) return MOE_ERR_INVALID;  // they are distinct
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_extend(*cache, seqs, add, n, ws, word, stream));
}

int moe_kv_append(const moe_kv_cache_t* cache, int layer, const int32_t* seqs, const int32_t* cu, int n, int total,
                  const moe_heads_t* k, const moe_heads_t* v, cudaStream_t stream) {
  const int st = upkeep_status(cache, n);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= cache->planes / 2 || total < 0) return MOE_ERR_INVALID;
  if (n == 0 || total == 0) return MOE_OK;
  if (!seqs || !cu || !heads_ok(k) || !heads_ok(v)) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(
      launch_kv_append(*cache, layer, seqs, cu, n, total, make_heads(*k), make_heads(*v), word, stream));
}

int moe_kv_fork(const moe_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
  const int st = upkeep_status(cache, n);
  if (st != MOE_OK || n == 0) return st;
  if (!src || !dst) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_fork(*cache, src, dst, n, word, stream));
}

int moe_kv_truncate(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* new_len, int n,
                    cudaStream_t stream) {
  const int st = upkeep_status(cache, n);
  if (st != MOE_OK || n == 0) return st;
  if (!seqs || !new_len) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_truncate(*cache, seqs, new_len, n, word, stream));
}

int moe_kv_keep(const moe_kv_cache_t* cache, const int32_t* seqs, const int32_t* drafted, const int32_t* keep,
                int max_keep, const int32_t* kept, int n, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int st = upkeep_status(cache, n);
  if (st != MOE_OK) return st;
  if (max_keep < 0) return MOE_ERR_INVALID;
  if (n == 0) return MOE_OK;
  if (!seqs || !drafted || (max_keep > 0 && !keep) || !kept) return MOE_ERR_INVALID;
  const KvWs ws = kv_carve(workspace, *cache);
  if ((st = workspace_status(workspace, ws_bytes, ws.bytes)) != MOE_OK) return st;
  if (n > cache->max_seqs) return MOE_ERR_INVALID;  // they are distinct
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_keep(*cache, seqs, drafted, keep, max_keep, kept, n, ws, word, stream));
}

int moe_kv_copy_pages(const moe_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t stream) {
  const int st = cache_status(cache);
  if (st != MOE_OK) return st;
  if (n < 0) return MOE_ERR_INVALID;  // (pages, not sequences: MOE_KV_MAX_CALL does not bound them)
  if (n == 0) return MOE_OK;
  if (!src || !dst) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_copy_pages(*cache, src, dst, n, word, stream));
}

int moe_kv_compact(const moe_kv_cache_t* cache, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int st = cache_status(cache);
  if (st != MOE_OK) return st;
  const KvWs ws = kv_carve(workspace, *cache);
  if ((st = workspace_status(workspace, ws_bytes, ws.bytes)) != MOE_OK) return st;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_kv_compact(*cache, ws, word, stream));
}

int moe_tree_mask(const int32_t* parents, const int32_t* cu, int n, int total, int32_t* mask, int mask_words,
                  cudaStream_t stream) {
  if (n < 0 || total < 0 || mask_words <= 0) return MOE_ERR_INVALID;
  if (n == 0 || total == 0) return MOE_OK;
  if (!parents || !cu || !mask) return MOE_ERR_INVALID;
  int* word = status_ptr();
  if (!word) return MOE_ERR_CUDA;
  return status_of(launch_tree_mask(parents, cu, n, total, mask, mask_words, word, stream));
}

int moe_attention_prompt(const moe_heads_t* q, const moe_heads_t* k, const moe_heads_t* v, const int32_t* cu_q,
                         const int32_t* cu_k, int n, int total_q, int total_k, int heads_q, int heads_kv, int head_dim,
                         int dtype, float scale, const moe_heads_t* out, float* lse, cudaStream_t stream) {
  const int st = attention_status(n, total_q, heads_q, heads_kv, head_dim, scale);
  if (st != MOE_OK) return st;
  if (total_k < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID;
  if (total_k > kMaxKeys) return MOE_ERR_SHAPE;
  if (n == 0 || total_q == 0) return MOE_OK;
  if (!heads_ok(q) || !heads_ok(out) || !cu_q || !cu_k) return MOE_ERR_INVALID;
  if (total_k > 0 && (!heads_ok(k) || !heads_ok(v))) return MOE_ERR_INVALID;
  AttnArgs a = {};
  a.q = make_heads(*q);
  if (total_k > 0) {
    a.k = make_heads(*k);
    a.v = make_heads(*v);
  }
  a.out = make_heads(*out);
  a.lse = lse;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.n = n;
  a.total_q = total_q;
  a.total_k = total_k;
  a.heads_q = heads_q;
  a.heads_kv = heads_kv;
  a.head_dim = head_dim;
  a.scale = scale;
  a.status = status_ptr();
  if (!a.status) return MOE_ERR_CUDA;
  return status_of(launch_attention(a, dtype, stream));
}

size_t moe_attention_cached_workspace_size(const moe_kv_cache_t* cache, int n, int total_q, int heads_q) {
  if (cache_status(cache) != MOE_OK || n < 0 || total_q < 0 || heads_q <= 0) return 0;
  if ((long long)total_q * heads_q > (1LL << 30)) return 0;
  return attention_ws(n, total_q, heads_q, cache->heads_kv, cache->head_dim,
                      (long long)cache->max_pages * cache->page_size)
      .bytes;
}

int moe_attention_cached(const moe_heads_t* q, const moe_kv_cache_t* cache, int layer, const int32_t* seqs,
                         const int32_t* cu_q, int n, int total_q, int heads_q, const int32_t* mask, int mask_words,
                         float scale, const moe_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                         cudaStream_t stream) {
  int st = cache_status(cache);
  if (st == MOE_OK) st = attention_status(n, total_q, heads_q, cache->heads_kv, cache->head_dim, scale);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= cache->planes / 2 || mask_words < 0 || (mask && mask_words == 0)) return MOE_ERR_INVALID;
  if (n == 0 || total_q == 0) return MOE_OK;
  if (!heads_ok(q) || !heads_ok(out) || !seqs || !cu_q) return MOE_ERR_INVALID;
  st = workspace_status(workspace, ws_bytes, moe_attention_cached_workspace_size(cache, n, total_q, heads_q));
  if (st != MOE_OK) return st;
  AttnArgs a = {};
  const long long hs = cache->head_dim, ts = hs * cache->heads_kv;
  const long long plane = ts * cache->page_size * cache->n_pages;
  uint16_t* pages = static_cast<uint16_t*>(cache->pages) + 2LL * layer * plane;
  a.q = make_heads(*q);
  a.k = {pages, ts, hs};
  a.v = {pages + plane, ts, hs};
  a.out = make_heads(*out);
  a.lse = lse;
  a.cu_q = cu_q;
  a.n = n;
  a.total_q = total_q;
  a.heads_q = heads_q;
  a.heads_kv = cache->heads_kv;
  a.head_dim = cache->head_dim;
  a.scale = scale;
  a.seqs = seqs;
  a.table = cache->table;
  a.length = cache->length;
  a.paged = 1;
  a.max_seqs = cache->max_seqs;
  a.max_pages = cache->max_pages;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.mask = mask;
  a.mask_words = mask_words;
  const AttnWs ws = attention_ws(n, total_q, heads_q, cache->heads_kv, cache->head_dim,
                                 (long long)cache->max_pages * cache->page_size);
  if (ws.part_rows > 0) {
    uint8_t* base = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(base + ws.o);
    a.part_ml = reinterpret_cast<float2*>(base + ws.ml);
    a.part_of = reinterpret_cast<int4*>(base + ws.of);
    a.part_rows = ws.part_rows;
  }
  a.status = status_ptr();
  if (!a.status) return MOE_ERR_CUDA;
  return status_of(launch_attention(a, cache->dtype, stream));
}

}  // extern "C"

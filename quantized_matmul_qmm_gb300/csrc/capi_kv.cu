// C-ABI entry points of the paged key/value cache: argument validation, then
// the launch.  Every check runs on the host before anything is queued.
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "kv_cache.h"

using namespace qmm;

namespace {

qmm_status kv_status(cudaError_t e) {
  if (e == cudaSuccess) return QMM_OK;
  if (std::getenv("QMM_LOG")) std::fprintf(stderr, "qmm: CUDA error %s\n", cudaGetErrorString(e));
  return QMM_ERR_CUDA;
}

// A stride (elements of `size` bytes) of a dimension of `count` rows: whole 16
// bytes and at least `least`; what a single row's stride holds is not used.
bool stride_ok(int64_t stride, int64_t count, int64_t least, int64_t size) {
  return count <= 1 || (stride >= least && stride <= (INT64_MAX >> 8) / size && stride * size % 16 == 0);
}
int64_t used(int64_t stride, int64_t count) { return count > 1 ? stride : 0; }

qmm_status cache_view(const qmm_kv_cache* c, KvView& v) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return QMM_ERR_INVALID_ARG;
  if (c->type != QMM_BF16 && c->type != QMM_S8) return QMM_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1) return QMM_ERR_INVALID_ARG;
  if (c->type == QMM_S8 &&
      (c->k_scale == nullptr || c->v_scale == nullptr || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return QMM_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return QMM_ERR_UNSUPPORTED;
  if (c->page_size >= (int64_t)1 << 30 || c->n_heads > 65535 || c->n_pages > INT32_MAX) return QMM_ERR_UNSUPPORTED;
  const int64_t size = c->type == QMM_BF16 ? 2 : 1;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QMM_ERR_INVALID_ARG;
  if (!stride_ok(c->stride_page, c->n_pages, c->head_dim, size) ||
      !stride_ok(c->stride_token, c->page_size, c->head_dim, size) ||
      !stride_ok(c->stride_head, c->n_heads, c->head_dim, size))
    return QMM_ERR_INVALID_ARG;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->type == QMM_S8 ? c->k_scale : nullptr;
  v.v_scale = c->type == QMM_S8 ? c->v_scale : nullptr;
  v.st_page = used(c->stride_page, c->n_pages) * size;
  v.st_token = used(c->stride_token, c->page_size) * size;
  v.st_head = used(c->stride_head, c->n_heads) * size;
  v.n_pages = c->n_pages;
  v.page_size = (uint32_t)c->page_size;
  v.n_heads = (int)c->n_heads;
  return QMM_OK;
}

qmm_status attn_rows_of(int64_t n_q_heads, int64_t n_kv_heads, int64_t max_new, int64_t* rows) {
  if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0 || max_new < 1) return QMM_ERR_INVALID_ARG;
  const int64_t group = n_q_heads / n_kv_heads;
  if (n_q_heads > 65535 || max_new >= ((int64_t)1 << 30) / group) return QMM_ERR_UNSUPPORTED;
  *rows = max_new * group;
  return QMM_OK;
}

}  // namespace

extern "C" {

qmm_status qmm_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t R, const int32_t* free_pages,
                       int64_t n_free, int32_t* block_table, int64_t ld_table, int64_t max_blocks,
                       int64_t page_size, const int32_t* parents, uint32_t* mask, int64_t ld_mask,
                       int64_t mask_words, int64_t max_tokens, int32_t* cu_new, int64_t* slots,
                       int32_t* positions, int32_t* pages_taken, int32_t* dev_status, cudaStream_t stream) {
  if (ctx_lens == nullptr || new_lens == nullptr || block_table == nullptr || cu_new == nullptr ||
      pages_taken == nullptr)
    return QMM_ERR_INVALID_ARG;
  if (R < 1 || n_free < 0 || max_blocks < 1 || ld_table < max_blocks || page_size < 1 || max_tokens < 0 ||
      mask_words < 0)
    return QMM_ERR_INVALID_ARG;
  if ((n_free > 0 && free_pages == nullptr) || (max_tokens > 0 && (slots == nullptr || positions == nullptr)))
    return QMM_ERR_INVALID_ARG;
  if (max_tokens > 0 && (parents != nullptr) != (mask != nullptr)) return QMM_ERR_INVALID_ARG;
  if ((mask != nullptr) != (mask_words > 0) && max_tokens > 0) return QMM_ERR_INVALID_ARG;
  if (mask != nullptr && ld_mask < mask_words) return QMM_ERR_INVALID_ARG;
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(cu_new, 4) ||
      !aligned(pages_taken, 4) || !aligned(free_pages, 4) || !aligned(parents, 4) || !aligned(mask, 4) ||
      !aligned(positions, 4) || !aligned(slots, 8))
    return QMM_ERR_INVALID_ARG;
  if (R > kPlanMaxRequests || page_size > INT32_MAX || max_tokens >= INT32_MAX || mask_words > (1 << 20))
    return QMM_ERR_UNSUPPORTED;
  KvPlanArgs a{};
  a.ctx = ctx_lens;
  a.fresh = new_lens;
  a.R = (int)R;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.table = block_table;
  a.ld_table = ld_table;
  a.max_blocks = max_blocks;
  a.page_size = (uint32_t)page_size;
  a.parents = parents;
  a.max_tokens = (int)max_tokens;
  a.cu = cu_new;
  a.slots = slots;
  a.positions = positions;
  a.mask = mask;
  a.ld_mask = ld_mask;
  a.mask_words = (int)mask_words;
  a.taken = pages_taken;
  a.dev_status = dev_status;
  return kv_status(launch_kv_plan(a, stream));
}

qmm_status qmm_kv_append(const void* K, int64_t k_stride_token, int64_t k_stride_head, const void* V,
                         int64_t v_stride_token, int64_t v_stride_head, qmm_dtype type, int64_t T,
                         const int64_t* slots, const qmm_kv_cache* cache, int32_t* dev_status,
                         cudaStream_t stream) {
  KvAppendArgs a{};
  const qmm_status st = cache_view(cache, a.cache);
  if (st != QMM_OK) return st;
  if (T < 0 || (type != QMM_F32 && type != QMM_BF16)) return QMM_ERR_INVALID_ARG;
  const int64_t size = type == QMM_F32 ? 4 : 2;
  if (!stride_ok(k_stride_token, T, 0, size) || !stride_ok(k_stride_head, cache->n_heads, 0, size) ||
      !stride_ok(v_stride_token, T, 0, size) || !stride_ok(v_stride_head, cache->n_heads, 0, size))
    return QMM_ERR_INVALID_ARG;
  if (T == 0) return QMM_OK;
  if (K == nullptr || V == nullptr || slots == nullptr) return QMM_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8)) return QMM_ERR_INVALID_ARG;
  if (T > INT32_MAX || T * cache->n_heads / 8 >= INT32_MAX) return QMM_ERR_UNSUPPORTED;
  a.k = static_cast<const uint8_t*>(K);
  a.v = static_cast<const uint8_t*>(V);
  a.k_st = used(k_stride_token, T) * size;
  a.k_sh = used(k_stride_head, cache->n_heads) * size;
  a.v_st = used(v_stride_token, T) * size;
  a.v_sh = used(v_stride_head, cache->n_heads) * size;
  a.T = (int)T;
  a.slots = slots;
  a.dev_status = dev_status;
  return kv_status(launch_kv_append(a, type == QMM_BF16, cache->type == QMM_S8, (int)cache->head_dim, stream));
}

qmm_status qmm_tree_attention_workspace_size(int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                                             int64_t max_new, size_t* ws_bytes) {
  int64_t rows = 0;
  if (ws_bytes == nullptr) return QMM_ERR_INVALID_ARG;
  const qmm_status st = attn_rows_of(n_q_heads, n_kv_heads, max_new, &rows);
  if (st != QMM_OK) return st;
  if (head_dim != 64 && head_dim != 128) return QMM_ERR_UNSUPPORTED;
  *ws_bytes = attn_workspace_bytes(rows, (int)head_dim);
  return QMM_OK;
}

qmm_status qmm_tree_attention(const void* q, qmm_dtype q_type, int64_t q_stride_token, int64_t q_stride_head,
                              int64_t n_q_heads, const qmm_kv_cache* cache, const int32_t* block_table,
                              int64_t ld_table, int64_t max_blocks, const int32_t* ctx_lens,
                              const int32_t* cu_new, int64_t R, int64_t T, int64_t max_new,
                              const uint32_t* mask, int64_t ld_mask, float scale, void* out,
                              int64_t out_stride_token, int64_t out_stride_head, void* workspace,
                              size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  AttnArgs a{};
  qmm_status st = cache_view(cache, a.cache);
  if (st != QMM_OK) return st;
  int64_t rows = 0;
  if ((st = attn_rows_of(n_q_heads, cache->n_heads, max_new, &rows)) != QMM_OK) return st;
  if (q_type != QMM_F32 && q_type != QMM_BF16) return QMM_ERR_INVALID_ARG;
  if (R < 1 || T < 0 || max_blocks < 1 || ld_table < max_blocks || !(scale > 0.f) || !std::isfinite(scale))
    return QMM_ERR_INVALID_ARG;
  const int64_t q_size = q_type == QMM_F32 ? 4 : 2;
  if (!stride_ok(q_stride_token, T, 0, q_size) || !stride_ok(q_stride_head, n_q_heads, 0, q_size) ||
      !stride_ok(out_stride_token, T, cache->head_dim, 2) ||
      !stride_ok(out_stride_head, n_q_heads, cache->head_dim, 2))
    return QMM_ERR_INVALID_ARG;
  if (mask != nullptr && (ld_mask < 1 || ld_mask * 32 < max_new)) return QMM_ERR_INVALID_ARG;
  if (R >= (int64_t)1 << 30 || T >= (int64_t)1 << 30) return QMM_ERR_UNSUPPORTED;
  if (T == 0) return QMM_OK;
  if (q == nullptr || out == nullptr || block_table == nullptr || ctx_lens == nullptr || cu_new == nullptr)
    return QMM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(ctx_lens, 4) ||
      !aligned(cu_new, 4) || !aligned(mask, 4))
    return QMM_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < attn_workspace_bytes(rows, (int)cache->head_dim))
    return QMM_ERR_WORKSPACE;
  a.q = q;
  a.q_st = used(q_stride_token, T);
  a.q_sh = used(q_stride_head, n_q_heads);
  a.table = block_table;
  a.ld_table = ld_table;
  a.max_len = max_blocks > INT32_MAX / cache->page_size ? INT32_MAX : max_blocks * cache->page_size;
  a.ctx = ctx_lens;
  a.cu = cu_new;
  a.R = (int)R;
  a.T = (int)T;
  a.max_new = (int)max_new;
  a.n_q_heads = (int)n_q_heads;
  a.group = (int)(n_q_heads / cache->n_heads);
  a.mask = mask;
  a.ld_mask = ld_mask;
  a.scale_log2 = scale * 1.4426950408889634f;   // log2(e): the softmax runs in base 2
  a.out = static_cast<__nv_bfloat16*>(out);
  a.o_st = used(out_stride_token, T);
  a.o_sh = used(out_stride_head, n_q_heads);
  a.dev_status = dev_status;
  return kv_status(launch_attn(a, q_type == QMM_F32, cache->type == QMM_S8, (int)cache->head_dim, workspace, stream));
}

}  // extern "C"

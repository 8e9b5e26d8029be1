// Host-side declarations of the paged key/value cache: the plan of a step, the
// append of its rows and the attention that reads them.
#pragma once

#include <atomic>

#include "qmm_internal.h"

namespace qmm {

// A kernel's attribute, set once per process and device: the runtime call costs
// about as much as an argument check of the whole entry point.
inline cudaError_t set_once(std::atomic<uint64_t>& done, const void* kernel, cudaFuncAttribute attr, int value) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, attr, value);
  if (err == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// ---- plan (kv_plan.cu) ----
constexpr int64_t kPlanMaxRequests = 16384;   // three int32 per request fit one block's shared memory
struct KvPlanArgs {
  const int32_t* ctx;        // [R]
  const int32_t* fresh;      // [R] new tokens of each request
  int R;
  const int32_t* free_pages; // [n_free]
  int64_t n_free;
  int32_t* table;            // [R][ld_table]
  int64_t ld_table;
  int64_t max_blocks;
  uint32_t page_size;
  const int32_t* parents;    // [max_tokens] or null
  int max_tokens;
  int32_t* cu;               // [R + 1]
  int64_t* slots;            // [max_tokens]
  int32_t* positions;        // [max_tokens]
  uint32_t* mask;            // [max_tokens][ld_mask], with parents
  int64_t ld_mask;
  int mask_words;
  int32_t* taken;            // [1]
  int32_t* dev_status;
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream);

// ---- the cache as the kernels see it (strides in bytes) ----
struct KvView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;            // int8 cache: [n_pages][n_heads][page_size]
  float* v_scale;
  int64_t st_page, st_token, st_head;
  int64_t n_pages;
  uint32_t page_size;
  int n_heads;
};

// ---- append (kv_append.cu) ----
struct KvAppendArgs {
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_st, k_sh, v_st, v_sh;   // bytes
  int T;
  const int64_t* slots;
  KvView cache;
  int32_t* dev_status;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, bool rows_bf16, bool cache_s8, int head_dim,
                             cudaStream_t stream);

// ---- tree attention (attn_rows.cu) ----
struct AttnArgs {
  const void* q;
  int64_t q_st, q_sh;        // elements
  KvView cache;
  const int32_t* table;      // [R][ld_table]
  int64_t ld_table;
  int64_t max_len;           // tokens that a table row has pages for
  const int32_t* ctx;        // [R]
  const int32_t* cu;         // [R + 1]
  int R, T, max_new;
  int n_q_heads, group;      // query heads, and query heads per key head
  const uint32_t* mask;      // [T][ld_mask] or null (causal)
  int64_t ld_mask;
  float scale_log2;          // softmax scale * log2(e)
  __nv_bfloat16* out;
  int64_t o_st, o_sh;        // elements
  float* part_o;             // workspace: [2 * grid][rows][head_dim]
  float2* part_ml;           // workspace: [2 * grid][rows]: running maximum (log2 domain) and sum
  int4* owned;               // workspace: [grid]: items that a block begins and another ends
  int* owned_rows;           // workspace: [grid]: their rows, 0 for none
  int grid;
  int32_t* dev_status;
};
// A cache side as a 4-D tensor {head_dim, place, head, page} for TMA: boxes of
// box_tokens places x 64 bf16 dimensions (128-byte swizzle) or x all int8 codes
// of a row (no swizzle).
bool make_tmap_kv(CUtensorMap* map, const void* base, bool s8, int head_dim, uint32_t page_size, uint64_t n_heads,
                  uint64_t n_pages, int64_t st_token, int64_t st_head, int64_t st_page, uint32_t box_tokens);

// What a call needs of the device, and how its workspace is laid out.
struct AttnPlan {
  bool tiles;          // attn_tiles.cu (tcgen05), else attn_rows.cu
  int rows_per_tile;   // query rows of an item
  int grid;            // blocks
};
int attn_sm_count();
// `pages_tile`: the cache's pages and scales allow TMA boxes (attn_pages_tile).
AttnPlan attn_plan(int64_t rows, bool pages_tile, bool s8);
bool attn_pages_tile(const KvView& c, bool s8);
size_t attn_workspace_bytes(int64_t rows, int head_dim);   // for any cache
cudaError_t launch_attn(AttnArgs& a, bool q_f32, bool cache_s8, int head_dim, void* workspace, cudaStream_t stream);
// one of the two kernels, and the joining of items that blocks share (attn_rows.cu)
cudaError_t launch_attn_rows(const AttnArgs& a, int rows_per_tile, bool q_f32, bool cache_s8, int head_dim,
                             cudaStream_t stream);
cudaError_t launch_attn_tiles(const AttnArgs& a, int rows_per_tile, bool q_f32, bool cache_s8, int head_dim,
                              cudaStream_t stream);
cudaError_t launch_attn_combine(const AttnArgs& a, int rows_per_tile, int head_dim, cudaStream_t stream);

}  // namespace qmm

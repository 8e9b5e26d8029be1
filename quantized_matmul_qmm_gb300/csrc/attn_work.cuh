// How the attention kernels split their work, shared by the kernels.
//
// An item is one (request, key head, tile of query rows); the query rows of a
// key head are row = i * group + e for new token i and query head e of the
// head's group.  An item's unit is one tile of `tile_tokens` cached tokens.
// Units are numbered request by request, then head, row tile and cached tile;
// block b of G gets units [b U / G, (b + 1) U / G), whatever the lengths, so
// the load is even without the host knowing them.  An item cut by a block
// boundary leaves partial results, which the combine kernel joins.
#pragma once

#include "kv_cache.h"

namespace qmm {

struct AttnReq {
  int L, n, first;   // cached tokens, new tokens, row of the first new token in q
  int row_tiles, kv_tiles;
  int64_t units;     // 0: nothing to do
};

// Lengths that do not fit the call's buffers give no units, and the status.
QMM_DEV AttnReq attn_req(const AttnArgs& a, int r, int rows_per_tile, int tile_tokens) {
  AttnReq q{};
  const int L = a.ctx[r], c0 = a.cu[r], c1 = a.cu[r + 1];
  const int64_t n = (int64_t)c1 - c0, len = (int64_t)L + n;
  if (L < 0 || c0 < 0 || n < 0 || c1 > a.T || n > a.max_new || len > INT32_MAX - 256 ||
      len > a.max_blocks * (int64_t)a.cache.page_size) {
    set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    return q;
  }
  q.L = L;
  q.n = (int)n;
  q.first = c0;
  q.row_tiles = ((int)n * a.group + rows_per_tile - 1) / rows_per_tile;
  q.kv_tiles = ((int)len + tile_tokens - 1) / tile_tokens;
  q.units = (int64_t)a.cache.n_heads * q.row_tiles * q.kv_tiles;
  return q;
}

struct AttnWork {
  int64_t total;     // units of the call
  int64_t blocks;    // blocks that share them
  int64_t u0, u1;    // this block's
  int r;             // request of u0
  int64_t off;       // u0's place among the request's units
};

struct AttnFindScratch {
  int64_t warp_sum[32];
  int64_t off;
  int r;
};

// All kThreads threads of the block; false (for all) when the block has none.
template <int kThreads>
QMM_DEV bool attn_find_work(const AttnArgs& a, int rows_per_tile, int tile_tokens, AttnFindScratch* s, AttnWork& w) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += attn_req(a, r, rows_per_tile, tile_tokens).units;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s->warp_sum[wid] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int64_t v = s->warp_sum[i];
    if (i < wid) before += v;
    total += v;
  }
  w.total = total;
  w.blocks = min((int64_t)a.grid, total);
  const int64_t b = blockIdx.x;
  if (b >= w.blocks) return false;
  w.u0 = b * total / w.blocks;
  w.u1 = (b + 1) * total / w.blocks;
  int64_t start = before + incl - mine;
  if (w.u0 >= start && w.u0 < start + mine) {   // one thread's requests hold u0
    for (int r = r0; r < r1; ++r) {
      const int64_t u = attn_req(a, r, rows_per_tile, tile_tokens).units;
      if (w.u0 < start + u) {
        s->r = r;
        s->off = w.u0 - start;
        break;
      }
      start += u;
    }
  }
  __syncthreads();
  w.r = s->r;
  w.off = s->off;
  return true;
}

// The block that has unit e.
QMM_DEV int64_t attn_block_of(const AttnWork& w, int64_t e) {
  return ((e + 1) * w.blocks + w.total - 1) / w.total - 1;
}

// Whether new token i (of the request whose first new token is row `first`)
// sees new token j; without a mask the tokens are a chain.
QMM_DEV bool attn_sees(const AttnArgs& a, int first, int i, int j) {
  if (a.mask == nullptr) return j <= i;
  return (a.mask[(int64_t)(first + i) * a.ld_mask + (j >> 5)] >> (j & 31)) & 1u;
}

// Byte offset of a cached token's row inside a head (page * st_page + place *
// st_token), or -1 where the block table holds no page of the cache.
QMM_DEV int64_t attn_row_offset(const AttnArgs& a, int32_t page, uint32_t tok) {
  if (page < 0 || page >= a.cache.n_pages) return -1;
  return page * a.cache.st_page + (int64_t)(tok % a.cache.page_size) * a.cache.st_token;
}

}  // namespace qmm

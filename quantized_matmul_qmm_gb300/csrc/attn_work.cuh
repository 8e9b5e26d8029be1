// How the attention kernels split their work, shared by the kernels.
//
// An item is one (request, key head, tile of query rows); the query rows of a
// key head are row = i * group + e for new token i and query head e of the
// head's group.  An item's unit is one tile of `tile_tokens` cached tokens;
// without a mask (causal chunks) an item has no units past its last row's own
// token, which halves a prompt that begins at an empty cache.
// Units are numbered request by request, then head, row tile and cached tile;
// each block gets the same number of consecutive units (to one), whatever the
// lengths, so the load is even without the host knowing them.  An item's first
// `setup` units stand for what it costs besides its tiles (queries in, the
// pipeline's first and last steps, outputs): a block with many short items
// would else be the last to end (chunks of 300 to 512 tokens at contexts of 0 to
// 6000: 118 -> 65 us).  With no more tiles than blocks, every block has one tile
// of one item, and they count for nothing (4 x 64 tokens at 1000: 18.7 us, with
// them 21.3).  An item cut by
// a block boundary leaves partial results, which the combine kernel joins.
// Unit numbers are 32-bit, so that the few divisions on a block's way to its
// first load are short.
#pragma once

#include "kv_cache.h"

namespace qmm {

// A kernel's items: query rows, cached tokens of a unit, units for the setup (at most).
struct AttnShape {
  int rows, tokens, setup;
};

struct AttnReq {
  int L, n, first;   // cached tokens, new tokens, row of the first new token in q
  int row_tiles, kv_tiles;   // 0 row tiles: nothing to do
};

// Token numbers are 32-bit and step past a request's end: the tile kernel looks
// pages up for the 32 boxes of up to 128 tokens from a tile's first, five tiles
// ahead of the last (4863 tokens), the row kernel eight steps of 64.
constexpr int kAttnMaxLen = INT32_MAX - 8192;

// Lengths that do not fit the call's buffers give no work, and the status.
QMM_DEV AttnReq attn_req(const AttnArgs& a, int r, AttnShape sh) {
  AttnReq q{};
  const int L = a.ctx[r], c0 = a.cu[r], c1 = a.cu[r + 1];
  const int64_t n = (int64_t)c1 - c0, len = (int64_t)L + n;
  if (L < 0 || c0 < 0 || n < 0 || c1 > a.T || n > a.max_new || len > kAttnMaxLen || len > a.max_len) {
    set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    return q;
  }
  q.L = L;
  q.n = (int)n;
  q.first = c0;
  q.row_tiles = ((int)n * a.group + sh.rows - 1) / sh.rows;
  q.kv_tiles = ((int)len + sh.tokens - 1) / sh.tokens;
  return q;
}

// Cached tiles of the items of row tile t: up to its last row's own token, or
// with a mask (any pattern) all.
QMM_DEV int attn_item_tiles(const AttnArgs& a, const AttnReq& q, int t, AttnShape sh) {
  if (a.mask != nullptr || t >= q.row_tiles - 1) return q.kv_tiles;
  return (q.L + ((t + 1) * sh.rows - 1) / a.group) / sh.tokens + 1;
}

// sum of (s * i + b) / m over i = 0 .. n - 1, in as many steps as Euclid's
// algorithm takes for s and m: the whole parts are sums of i, and the rest
// counts points below a line, which is the same sum with the axes exchanged.
QMM_DEV int64_t attn_floor_sum(uint32_t n, uint32_t m, uint32_t s, uint32_t b) {
  int64_t sum = 0;
#pragma unroll 1
  while (n > 0) {
    sum += (int64_t)n * (n - 1) / 2 * (s / m) + (int64_t)n * (b / m);
    s %= m;
    b %= m;
    const uint32_t top = s * n + b;              // below 2^31: at most the request's rows and m
    n = top / m;
    b = top - n * m;
    const uint32_t old = m;
    m = s;
    s = old;
  }
  return sum;
}

// Tiles of a head's first t < row_tiles row tiles.
QMM_DEV int64_t attn_tiles_before(const AttnArgs& a, const AttnReq& q, int t, AttnShape sh) {
  if (t <= 0) return 0;
  if (a.mask != nullptr) return (int64_t)t * q.kv_tiles;
  // attn_item_tiles with the whole tiles of L set apart
  return (int64_t)t * (q.L / sh.tokens + 1) +
         attn_floor_sum(t, sh.tokens * a.group, sh.rows, sh.rows - 1 + q.L % sh.tokens * a.group);
}
QMM_DEV int64_t attn_head_tiles(const AttnArgs& a, const AttnReq& q, AttnShape sh) {
  return q.row_tiles == 0 ? 0 : attn_tiles_before(a, q, q.row_tiles - 1, sh) + q.kv_tiles;
}

struct AttnWork {
  int total, blocks;     // units of the call, and the blocks that share them
  int setup;             // units that an item's setup counts for
  int per, extra;        // each block has `per` units, the first `extra` blocks one more
  int u0, u1;            // this block's
  int r;                 // request of u0
  AttnReq q;
  int h, t, pos;         // u0's key head, row tile and place among the item's units
  QMM_DEV int block_of(int e) const {
    const int head = extra * (per + 1);
    return e < head ? e / (per + 1) : extra + (e - head) / per;
  }
};

struct AttnFindScratch {
  int64_t warp_tiles[32], warp_items[32];
  AttnReq q;
  int r, off, head_units;
};

QMM_DEV bool attn_share(const AttnArgs& a, int64_t tiles, int64_t items, AttnShape sh, AttnWork& w) {
  w.setup = tiles > a.grid ? sh.setup : 0;
  const int64_t total = tiles + w.setup * items;
  if (total > INT32_MAX) {
    set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    return false;
  }
  w.total = (int)total;
  w.blocks = min(a.grid, w.total);
  const int b = blockIdx.x;
  if (b >= w.blocks) return false;
  w.per = w.total / w.blocks;
  w.extra = w.total - w.per * w.blocks;
  w.u0 = b * w.per + min(b, w.extra);
  w.u1 = w.u0 + w.per + (b < w.extra ? 1 : 0);
  return true;
}

// u0 is unit `off` of request w.q, whose heads have head_units units each.
QMM_DEV void attn_place(const AttnArgs& a, int off, int head_units, AttnShape sh, AttnWork& w) {
  w.h = off / head_units;
  off -= w.h * head_units;
  int lo = 0, hi = w.q.row_tiles - 1;            // the last row tile that begins at or before `off`
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (attn_tiles_before(a, w.q, mid, sh) + (int64_t)w.setup * mid <= off) lo = mid; else hi = mid - 1;
  }
  w.t = lo;
  w.pos = off - (int)attn_tiles_before(a, w.q, lo, sh) - w.setup * lo;
}

// All kThreads threads of the block; false (for all) when the block has none.
template <int kThreads>
QMM_DEV bool attn_find_work(const AttnArgs& a, AttnShape sh, AttnFindScratch* s, AttnWork& w) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (a.R <= 32) {   // every warp for itself: one request per lane, no barrier
    AttnReq q{};
    if (lane < a.R) q = attn_req(a, lane, sh);
    const int64_t head_tiles = attn_head_tiles(a, q, sh), tiles = a.cache.n_heads * head_tiles;
    const int64_t items = (int64_t)a.cache.n_heads * q.row_tiles;
    int64_t incl = tiles, incl_items = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o), up_items = __shfl_up_sync(0xffffffffu, incl_items, o);
      if (lane >= o) incl += up, incl_items += up_items;
    }
    if (!attn_share(a, __shfl_sync(0xffffffffu, incl, 31), __shfl_sync(0xffffffffu, incl_items, 31), sh, w))
      return false;
    const int stop = (int)(incl + w.setup * incl_items);   // all fit 32 bits now
    const int start = stop - (int)(tiles + w.setup * items), head_units = (int)head_tiles + w.setup * q.row_tiles;
    const int at = __ffs(__ballot_sync(0xffffffffu, w.u0 >= start && w.u0 < stop)) - 1;
    w.r = at;
    w.q.L = __shfl_sync(0xffffffffu, q.L, at);
    w.q.n = __shfl_sync(0xffffffffu, q.n, at);
    w.q.first = __shfl_sync(0xffffffffu, q.first, at);
    w.q.row_tiles = __shfl_sync(0xffffffffu, q.row_tiles, at);
    w.q.kv_tiles = __shfl_sync(0xffffffffu, q.kv_tiles, at);
    attn_place(a, w.u0 - __shfl_sync(0xffffffffu, start, at), __shfl_sync(0xffffffffu, head_units, at),
               sh, w);
    return true;
  }
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  int64_t tiles = 0, items = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const AttnReq q = attn_req(a, r, sh);
    tiles += a.cache.n_heads * attn_head_tiles(a, q, sh);
    items += (int64_t)a.cache.n_heads * q.row_tiles;
  }
  int64_t incl = tiles, incl_items = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o), up_items = __shfl_up_sync(0xffffffffu, incl_items, o);
    if (lane >= o) incl += up, incl_items += up_items;
  }
  if (lane == 31) s->warp_tiles[wid] = incl, s->warp_items[wid] = incl_items;
  __syncthreads();
  int64_t before = incl - tiles, before_items = incl_items - items, total = 0, total_items = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < wid) before += s->warp_tiles[i], before_items += s->warp_items[i];
    total += s->warp_tiles[i];
    total_items += s->warp_items[i];
  }
  if (!attn_share(a, total, total_items, sh, w)) return false;
  int64_t start = before + w.setup * before_items;
  if (w.u0 >= start && w.u0 < start + tiles + w.setup * items) {   // one thread's requests hold u0
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const AttnReq q = attn_req(a, r, sh);
      const int64_t head_units = attn_head_tiles(a, q, sh) + (int64_t)w.setup * q.row_tiles;
      if (w.u0 < start + a.cache.n_heads * head_units) {
        s->q = q;
        s->r = r;
        s->off = (int)(w.u0 - start);
        s->head_units = (int)head_units;
        break;
      }
      start += a.cache.n_heads * head_units;
    }
  }
  __syncthreads();
  w.r = s->r;
  w.q = s->q;
  attn_place(a, s->off, s->head_units, sh, w);
  return true;
}

// A block's part of one item: cached tiles [kv0, kv0 + seg).
struct AttnItem {
  AttnReq q;
  int r;              // request
  int h, row0, n_rows;
  int kv0, seg, len;
  int seen;           // every row sees the tokens before this one; the step's first rows' own count as not seen
  bool whole;
  int pieces;         // of an item that this block begins and another ends; else 0
};

// Walks a block's units item by item.
struct AttnWalk {
  AttnReq q;
  int r, h, t, pos, u;   // the next unit
  QMM_DEV void start(const AttnWork& w) {
    q = w.q;
    r = w.r;
    h = w.h;
    t = w.t;
    pos = w.pos;
    u = w.u0;
  }
  QMM_DEV bool next(const AttnArgs& a, const AttnWork& w, AttnShape sh, AttnItem& it) {
    while (u < w.u1) {
      if (t >= q.row_tiles) t = 0, ++h;
      while (h >= a.cache.n_heads || q.row_tiles == 0) {   // to the next request that has work
        q = attn_req(a, ++r, sh);
        h = 0;
      }
      const int tiles = attn_item_tiles(a, q, t, sh), units = w.setup + tiles;
      const int take = min(units - pos, w.u1 - u), end = pos + take - w.setup;
      it.kv0 = max(pos - w.setup, 0);
      it.seg = end - it.kv0;
      it.h = h;
      it.row0 = t * sh.rows;
      it.whole = it.seg == tiles;
      it.pieces = 0;           // up to the block that has the item's last unit
      if (!it.whole && it.kv0 == 0) it.pieces = w.block_of(u - pos + units - 1) - (int)blockIdx.x + 1;
      u += take;
      pos += take;
      if (pos == units) pos = 0, ++t;
      if (it.seg <= 0) continue;   // only of the setup: the next block's item
      it.q = q;
      it.r = r;
      it.n_rows = min(sh.rows, q.n * a.group - it.row0);
      it.len = q.L + q.n;
      it.seen = q.L + (a.mask != nullptr || it.row0 == 0 ? 0 : it.row0 / a.group + 1);
      return true;
    }
    return false;
  }
};

// What the combine kernel is told of an item that a block begins and another
// ends (pieces 0: nothing).  The workspace's descriptors are the numbers of
// rows of all blocks' items, then the rest.
struct AttnOwned {
  int h, row0, pieces, first;
  int n_rows;
};
QMM_DEV AttnOwned attn_owned(const AttnItem& it) {
  return AttnOwned{it.h, it.row0, it.pieces, it.q.first, it.n_rows};
}
QMM_DEV void attn_post_owned(const AttnArgs& a, const AttnOwned& o) {
  a.owned_rows[blockIdx.x] = o.n_rows;
  if (o.n_rows > 0) a.owned[blockIdx.x] = make_int4(o.h, o.row0, o.pieces, o.first);
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

// Which of the 32 tokens from tok0 on new token i sees: bit b for tok0 + b.
QMM_DEV uint32_t attn_sees32(const AttnArgs& a, const AttnReq& q, int i, int tok0) {
  const int j0 = tok0 - q.L;
  if (j0 + 32 <= 0) return ~0u;
  auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; };
  if (a.mask == nullptr) return below(i + 1 - j0);
  const uint32_t* row = a.mask + (int64_t)(q.first + i) * a.ld_mask;
  const int words = (q.n + 31) >> 5;
  uint32_t w;
  if (j0 >= 0) {
    const int k = j0 >> 5;
    w = __funnelshift_r(k < words ? row[k] : 0u, k + 1 < words ? row[k + 1] : 0u, j0 & 31);
  } else {
    w = (row[0] << -j0) | below(-j0);
  }
  return w & below(q.n - j0);
}

QMM_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

QMM_DEV uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two int8 codes in the low bytes of 16-bit lanes (the high bytes may hold
// anything) -> bf16x2, exactly: the low seven bits on top of 128, and -128 or
// (sign bit) -256 added.
QMM_DEV uint32_t s8_lanes_to_bf16(uint32_t x) {
  uint32_t lo, hi, r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(lo) : "r"(x), "r"(0x007F007Fu), "r"(0x43004300u));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(hi) : "r"(x), "r"(0x00800080u), "r"(0xC300C300u));
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(lo), "r"(hi));
  return r;
}

// Zeros in place of the non-finite ones of eight bf16 values; whether there were any.
QMM_DEV bool bf16_drop_nonfinite(uint4& v) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
  bool hit = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((x[e] & 0x7F80u) == 0x7F80u) x[e] &= 0xFFFF0000u, hit = true;
    if ((x[e] & 0x7F800000u) == 0x7F800000u) x[e] &= 0x0000FFFFu, hit = true;
  }
  v = make_uint4(x[0], x[1], x[2], x[3]);
  return hit;
}

// One element of the cache's value rows.
QMM_DEV float attn_cached_v(const AttnArgs& a, int r, int h, int tok, int d) {
  const int32_t page = a.table[(int64_t)r * a.ld_table + tok / a.cache.page_size];
  const int64_t off = attn_row_offset(a, page, tok);
  if (off < 0) return 0.f;
  if (a.cache.v_scale != nullptr) {
    const float s =
        a.cache.v_scale[((int64_t)page * a.cache.n_heads + h) * a.cache.page_size + (uint32_t)tok % a.cache.page_size];
    return s * (float)*reinterpret_cast<const int8_t*>(a.cache.v + h * a.cache.st_head + off + d);
  }
  const uint8_t* p = a.cache.v + h * a.cache.st_head + off + 2 * d;
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

// The non-finite value elements of an item's new tokens (which the products
// leave out) in the outputs d0 .. d0 + n - 1 of new token i: bit e of the
// results for +inf, -inf and NaN.  Rare: kept out of line.
struct AttnNonfinite {
  uint32_t pos, neg, nan;
};
static __device__ __noinline__ AttnNonfinite attn_nonfinite(const AttnArgs& a, int r, int h, int L, int first, int j0, int j1,
                                                     int i, int d0, int n) {
  AttnNonfinite f{0, 0, 0};
  for (int j = j0; j < j1; ++j) {
    if (!attn_sees(a, first, i, j)) continue;
    for (int e = 0; e < n; ++e) {
      const float v = attn_cached_v(a, r, h, L + j, d0 + e);
      if (v == INFINITY) f.pos |= 1u << e;
      if (v == -INFINITY) f.neg |= 1u << e;
      if (v != v) f.nan |= 1u << e;
    }
  }
  return f;
}
template <int N>
QMM_DEV void attn_add_nonfinite(const AttnArgs& a, const AttnItem& it, int tile_tokens, int i, int d0, float (&x)[N]) {
  const int j0 = max(0, it.kv0 * tile_tokens - it.q.L), j1 = min(it.len, (it.kv0 + it.seg) * tile_tokens) - it.q.L;
  const AttnNonfinite f = attn_nonfinite(a, it.r, it.h, it.q.L, it.q.first, j0, j1, i, d0, N);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if ((f.pos >> e) & 1) x[e] += INFINITY;
    if ((f.neg >> e) & 1) x[e] -= INFINITY;
    if ((f.nan >> e) & 1) x[e] = NAN;
  }
}

QMM_DEV __nv_bfloat16* attn_out_row(const AttnArgs& a, int first, int h, int row) {
  return a.out + (int64_t)(first + row / a.group) * a.o_st + (int64_t)(h * a.group + row % a.group) * a.o_sh;
}
QMM_DEV int64_t attn_q_row(const AttnArgs& a, const AttnReq& q, int h, int row) {
  return (int64_t)(q.first + row / a.group) * a.q_st + (int64_t)(h * a.group + row % a.group) * a.q_sh;
}

}  // namespace qmm

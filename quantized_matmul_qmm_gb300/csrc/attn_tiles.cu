// Tree attention for many query rows per key head, on the tcgen05 tensor cores.
//
// An item is up to 128 (kRT = 1) or 256 (kRT = 2) query rows of one key head;
// cached tokens come in tiles of 128.  Per tile of 128 rows x 128 tokens:
//   S = Q K^T   into TMEM (128 columns of fp32), Q and K in shared memory;
//   p = exp2(c s - c m) by four warps, one row per thread, m a running
//       reference that follows the row's maximum;
//   O += P V    with P (bf16) over S's columns in TMEM as the A operand and V
//       as it lies in memory (MN-major B operand).
// Two streams, so that one's exponentials run under the other's products: with
// kRT = 1 they take the even and the odd cached tiles of the same rows (joined
// when the item ends), with kRT = 2 the two halves of 256 rows, and each
// cached tile is fetched once for both.
//
// TMEM has 512 columns, and the two O take 256.  A bf16 cache: one S of 128
// columns for both streams and a P of 64 for each.  A row's scores go to
// registers at once, the other stream's scores follow into the same columns,
// and a stream finds its next scores ready when it has stored its weights.
// With S and P of a stream in the same columns the
// next scores could only follow the product with the weights, which left the
// tensor pipe idle for a third of a tile.  An int8 cache (with the scales there
// are no registers for a row of scores): S of 128 columns for each stream, P
// over it, PV(q) before S(q + 2).
//
// Up to 64 rows the tile's other 64 lanes hold the same rows again, and their P
// the part of each weight that the first bf16 rounding left over: the padded
// products then give the weights 16 bits for nothing (see attn_rows.cu).
// With more rows no lane is free and a second term would be a product of its own:
// half as many operations again where the tensor pipe is 60 % busy, and another
// 64 columns of TMEM that the two streams do not leave.  There the weights are
// rounded to bf16 once, and the outputs' error against 64 bits is 0.0020 (chunks)
// to 0.0023 (512 rows) of their size, 0.0016 of it the outputs' own rounding.
//
// The reference m moves only when a tile's maximum passes it by 2^8 in the
// weights, so that O is rarely rescaled (it is in TMEM, not in registers).
//
// Warps: 0 loads (TMA boxes of page_size's power of two; the pages of a tile
// looked up by one lane each), 1 and 2 issue the products, 3 cleans the value
// tiles that hold tokens which a row may not see (zeros past the request's end
// and for non-finite values, see attn_rows.cu), 4..11 are the two streams' rows.  With
// an int8 cache, 1 issues all products, tiles arrive as codes, eight more warps write them out as
// bf16 in the products' layout, and 2 and 3 bring the scales; a token's key
// scale multiplies its column of s, its value scale the weight.
//
// What bounds it: 4 * 128 operations per row and token against 512 (bf16) or
// 264 (int8) bytes per token: the cache's bytes up to about 128 rows, the
// tensor pipe and the exponentials above.  Measured, heads of 128:
//   bf16, 400k tokens, 8 key heads, pages of 64: 128 rows 254 us (0.95 of a copy's
//   rate); pages of 16: 32 to 128 rows 324 to 336 us (0.74: 64 TMA boxes per tile);
//   bf16, 400k tokens, 512 rows: 0.76 of a library product's rate; 16 trees of 64
//   nodes (512 rows) at 6k to 16k tokens 167 to 170 us (0.60; 16 us of it the joining),
//   fp32 queries 178, heads of 64 127 us (0.40: the exponentials are as many);
//   a prompt of 8192 tokens, 32 heads: 508 us (0.57);
//   int8, 32 rows at 200k tokens 163 us (0.38 of a copy's rate), 128 rows at 400k 290
//   (0.43), 512 rows at 6k to 16k 258 (0.39 of a library product's rate), a prompt of
//   8192 tokens 738 us (0.39).  It is bound by the converters' and rows' shared-memory
//   passes and their issue slots, about 9300 warp instructions per tile;
//   chunks of 300 to 512 tokens at 0 to 6000: 64 us (int8 86, heads of 64 50, fp32
//   queries 69), of which a block spends about 9 us per item on queries, the first
//   and last steps and fp32 partial outputs.
// The call's max_new chooses the kernel for all of its requests: 63 requests of one
// token at 3 to 8191 beside a chunk of 512 take 263 us, apart 164 and 44.
#include <algorithm>
#include <type_traits>

#include "attn_umma.cuh"
#include "attn_work.cuh"

namespace qmm {
namespace {

using namespace umma;

constexpr int kTok = 128;                        // cached tokens per tile
constexpr int kHalf = 128 * 128;                 // bytes of 128 rows x 64 bf16
constexpr int kScaleRing = 8;
// Items' flags, by number.  One is raised for an item whose tile has been fetched,
// which is at most 8 items ahead of the rows (a tile each in the rings), so no item
// that still needs its place; nothing is cleared.
constexpr int kBadRing = 32;

template <int D, bool kS8, int kRT>
struct Tg {
  static constexpr int kNH = D / 64;             // 64-column halves of a row
  static constexpr int kTile = kNH * kHalf;      // bytes of a bf16 tile
  static constexpr int kRaw = kTok * D;          // bytes of a tile of codes
  static constexpr int kSlots = D == 64 ? (kS8 ? 6 : 8) : kS8 ? 3 : (kRT == 1 ? 6 : 5);
  static constexpr int kKeySlots = kS8 ? kSlots : kSlots / 2;   // bf16: the first ones for keys, the others for values
  static constexpr int kRawSlots = !kS8 ? 0 : D == 64 ? 8 : (kRT == 1 ? 5 : 3);
  static constexpr int kConvWarps = kS8 ? 8 : 0;
  static constexpr int kThreads = 384 + 32 * kConvWarps;
  static constexpr int kOffSlots = kRT * kTile;
  static constexpr int kOffRaw = kOffSlots + kSlots * kTile;
  static constexpr int kOffScale = kOffRaw + kRawSlots * kRaw;
  static constexpr int kBytes = kOffScale + (kS8 ? kScaleRing * 2 * kTok * 4 : 0);
  // An item's setup takes about 9 us, a tile 1 to 2 (bf16) or 2 (int8).  In us with
  // 0, 3, 6 and 10 units (bf16), 0, 3, 4 and 10 (int8):
  //   chunks of 300 to 512 tokens   123  75.5 63.8 65.2     136  84.6 86.0 97.8
  //   trees of 9 to 25 nodes        37.8 35.7 33.4 34.8     36.8 33.3 31.6 36.0
  //   512 rows at 6k to 16k         175  171  167  166      265  258  258  275
  //   a prompt of 8192 tokens       648  523  508  527      872  731  739  790
  //   128 rows at 400k              259  257  253  251      296  291  290  290
  static constexpr AttnShape kShape{128 * kRT, kTok, kS8 ? 4 : 6};
  static constexpr bool kShared = !kS8;          // one S for both streams (see the top)
  static constexpr int kAhead = (kRT == 1 ? 2 : 1) + (kShared ? 1 : 0);   // key tiles fetched ahead of value tiles
};

struct TBars {
  uint64_t full[8], empty[8];        // bf16 tiles
  uint64_t tail_full[8];             // value tiles that warp 3 hands on
  uint64_t raw_full[8], raw_empty[8];
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing];
  uint64_t s_full[2], s_free, p_ready[2], o_done[2];
  uint64_t q_full, o_free, sync;
  uint64_t done;
};

struct RowItem {
  AttnWalk walk;
  AttnItem it;
  int more;
};

struct TShared {
  TBars bar;
  AttnWork work;                                 // out of the roles' registers
  union {
    struct {
      float m[2][128], l[2][128];                // kRT == 1
    };
    RowItem item[8];                             // of the row warps (see row_warps)
    AttnFindScratch find;                        // before the roles begin
  };
  uint32_t bad[kBadRing];            // [i % kBadRing] = i + 1: a non-finite value was taken out of item i
  uint32_t tmem;
  int abort;
};

// TMEM columns (the block allocates all 512, which begin at column 0); stream st: + 128 * st
constexpr int kColS = 0, kColP = 128, kColO = 256;   // kColP (+ 64 * st): with a shared S

struct Ctx {
  const AttnArgs& a;
  TShared* sh;
  uint8_t* smem;
  uint32_t box;                                  // tokens of a TMA box
  // The first tries suspend the thread until the phase completes; only then
  // does the wait read the clock for its limit (the read itself takes long).
  QMM_DEV bool wait(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait_suspend(bar, parity, kSuspendHintNs)) return true;
    return mbar_wait(bar, parity, &sh->abort, a.dev_status);
  }
  QMM_DEV bool wait_all(uint64_t* bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait(bar, parity)); }
};

// The order in which an item's tiles are fetched and used: kAhead key tiles,
// then value tile i and key tile i + kAhead in turn.  Every role walks it in
// one loop with one body: a block runs most of its code for a few tiles only,
// and code seen for the first time costs more to fetch than to run.
template <int kAhead>
struct TileOrder {
  int seg, keys = 0, values = 0;
  QMM_DEV bool next(bool& value, int& i) {
    if (values >= seg) return false;
    value = keys >= seg || keys - values >= kAhead;
    i = value ? values++ : keys++;
    return true;
  }
};

// A ring of n slots from `base` on: the next slot, and its barriers' phase.
struct Ring {
  uint32_t base, n, slot, phase;
  QMM_DEV Ring(uint32_t b, uint32_t count, uint32_t ph) : base(b), n(count), slot(b), phase(ph) {}
  QMM_DEV void next() {
    if (++slot == base + n) slot = base, phase ^= 1;
  }
};

// ---- warp 0: tiles into shared memory ----
// One warp's chain of instructions per tile has to stay well under the tile's
// time at HBM rate (0.8 to 1.5 us): places of a tile follow from the last
// tile's by an addition (no division), and the page table is read two tiles
// ahead.
template <int D, bool kS8, int kRT>
QMM_DEV void load_warp(const Ctx& x, const CUtensorMap& mk, const CUtensorMap& mv) {
  using G = Tg<D, kS8, kRT>;
  const AttnArgs& a = x.a;
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kN = kS8 ? G::kRawSlots : G::kSlots, kStage = kS8 ? G::kRaw : G::kTile;
  constexpr uint32_t kRow = kS8 ? D : 128;       // bytes of a row of a box
  constexpr int kWin = G::kAhead + 2;            // tiles looked up and not yet fetched
  uint64_t* full = kS8 ? x.sh->bar.raw_full : x.sh->bar.full;
  uint64_t* empty = kS8 ? x.sh->bar.raw_empty : x.sh->bar.empty;
  const uint32_t box = x.box, P = a.cache.page_size, lane_off = lane * box * kRow;
  const uint32_t base = smem_u32(x.smem) + (kS8 ? G::kOffRaw : G::kOffSlots) + lane_off;
  const uint32_t box_bytes = box * D * (kS8 ? 1 : 2);
  const int lane_tok = lane * (int)box;
  const uint32_t step_blk = kTok / P, step_place = kTok % P;
  Ring keys(0, kS8 ? kN : G::kKeySlots, 1), vals(G::kKeySlots, kN - G::kKeySlots, 1);
  if (lane == 0) {
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  AttnWalk walk;
  walk.start(x.sh->work);
  AttnItem it;
  while (walk.next(a, x.sh->work, G::kShape, it)) {
    const int32_t* trow = a.table + (int64_t)it.r * a.ld_table;
    // lane b's box of each tile: block and place of the next tile to look up
    int tok = it.kv0 * kTok + lane_tok;
    uint32_t blk = (uint32_t)tok / P, place = (uint32_t)tok % P;
    const int tok_end = lane_tok < kTok ? min(it.len, (it.kv0 + it.seg) * kTok) : 0;
    int32_t page[kWin];                          // page[j]: of tile (value tiles fetched) + j
    uint32_t places[kWin];
    auto look_up = [&](int32_t& pg, uint32_t& pl) {
      pg = tok < tok_end ? trow[blk] : -1;
      pl = place;
      tok += kTok;
      blk += step_blk;
      place += step_place;
      if (place >= P) place -= P, ++blk;
    };
#pragma unroll
    for (int j = 0; j < kWin; ++j) look_up(page[j], places[j]);
    TileOrder<G::kAhead> order{it.seg};
    bool value;
    int i;
#pragma unroll 1
    while (order.next(value, i)) {
      // value tile i: page[0]; key tile i: page[i - value tiles]
      int32_t pg = page[0];
      uint32_t pl = places[0];
#pragma unroll
      for (int j = 1; j < G::kAhead; ++j)
        if (!value && i - order.values == j) pg = page[j], pl = places[j];
      Ring& ring = !kS8 && value ? vals : keys;
      const uint32_t slot = ring.slot;
      if (!x.wait_all(&empty[slot], ring.phase)) return;
      const int tok0 = (it.kv0 + i) * kTok, left = it.len - tok0;
      const uint32_t boxes = ((uint32_t)min(left, kTok) + box - 1) / box;
      uint64_t* landed = !kS8 && value && tok0 + kTok > it.seen ? &x.sh->bar.tail_full[slot] : &full[slot];
      if (lane == 0) mbar_arrive_expect_tx(landed, boxes * box_bytes);
      __syncwarp();
      if (lane < boxes) {
        if ((uint32_t)pg >= (uint64_t)a.cache.n_pages) {   // reported; page 0 stands in
          set_status(a.dev_status, QMM_ERR_INVALID_ARG);
          pg = 0;
        }
        const CUtensorMap* map = value ? &mv : &mk;
        const uint32_t dst = base + slot * kStage;
        if constexpr (kS8) {
          tma_load_4d(dst, map, landed, 0, pl, it.h, pg);
        } else {
#pragma unroll
          for (int hf = 0; hf < G::kNH; ++hf) tma_load_4d(dst + hf * kHalf, map, landed, 64 * hf, pl, it.h, pg);
        }
      }
      ring.next();
      if (value) {
#pragma unroll
        for (int j = 0; j < kWin - 1; ++j) page[j] = page[j + 1], places[j] = places[j + 1];
        look_up(page[kWin - 1], places[kWin - 1]);
      }
    }
  }
}

// Zeros for the non-finite ones of four scales from number `from` on.
QMM_DEV bool drop_nonfinite(float4& f, int from) {
  bool hit = false;
  if (from <= 0 && !isfinite(f.x)) f.x = 0.f, hit = true;
  if (from <= 1 && !isfinite(f.y)) f.y = 0.f, hit = true;
  if (from <= 2 && !isfinite(f.z)) f.z = 0.f, hit = true;
  if (from <= 3 && !isfinite(f.w)) f.w = 0.f, hit = true;
  return hit;
}

// ---- int8: warps 2 and 3 bring the tiles' key and value scales ----
// Four tokens per lane.  Bulk copies of a page's few scales each would cost the
// copy engine as much as the pages' rows.  Value scales that are not finite, of
// tokens that a row may not see, count as 0 and raise the item's flag: the rows that see them get
// theirs at the end, as for a bf16 cache.
template <int D, int kRT>
QMM_DEV void scale_warps(const Ctx& x) {
  using G = Tg<D, true, kRT>;
  const AttnArgs& a = x.a;
  const int lane = threadIdx.x & 31, side = (threadIdx.x >> 5) & 1;
  const float* src = side ? a.cache.v_scale : a.cache.k_scale;
  float4* ring = reinterpret_cast<float4*>(x.smem + G::kOffScale) + side * (kTok / 4) + lane;
  const uint32_t P = a.cache.page_size, step_blk = kTok / P, step_place = kTok % P;
  uint32_t sc = 0, phase = 1, seq = 0;
  AttnWalk walk;
  walk.start(x.sh->work);
  AttnItem it;
  for (; walk.next(a, x.sh->work, G::kShape, it); ++seq) {
    const int32_t* trow = a.table + (int64_t)it.r * a.ld_table;
    const int tok_end = min(it.len, (it.kv0 + it.seg) * kTok);
    int tok = it.kv0 * kTok + 4 * lane;
    uint32_t blk = (uint32_t)tok / P, place = (uint32_t)tok % P;
    // a tile's page entries are read two tiles ahead, its scales one
    auto page_of = [&](uint32_t& pl) -> int32_t {
      const int32_t pg = tok < tok_end ? trow[blk] : -1;
      pl = place;
      tok += kTok;
      blk += step_blk;
      place += step_place;
      if (place >= P) place -= P, ++blk;
      return pg;
    };
    auto scales = [&](int32_t pg, uint32_t pl) {
      if ((uint32_t)pg >= (uint64_t)a.cache.n_pages) return make_float4(0.f, 0.f, 0.f, 0.f);
      return *reinterpret_cast<const float4*>(src + ((int64_t)pg * a.cache.n_heads + it.h) * P + pl);
    };
    uint32_t pl = 0, pl_next = 0;
    int32_t pg = page_of(pl), pg_next = page_of(pl_next);
    float4 v = scales(pg, pl);
#pragma unroll 1
    for (int i = 0; i < it.seg; ++i) {
      const float4 v_next = scales(pg_next, pl_next);
      pg_next = page_of(pl_next);
      if (!x.wait_all(&x.sh->bar.sc_empty[sc], phase)) return;
      const int from = it.seen - (it.kv0 + i) * kTok - 4 * lane;   // of the lane's four, the first that a row may not see
      if (side && from < 4 && drop_nonfinite(v, from)) x.sh->bad[seq % kBadRing] = seq + 1;
      ring[sc * (2 * kTok / 4)] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.sh->bar.sc_full[sc]);
      v = v_next;
      if (++sc == kScaleRing) sc = 0, phase ^= 1;
    }
  }
}

// ---- int8: eight warps write codes out as bf16 ----
// Four codes of a word leave in the order 0, 2, 1, 3, which costs no byte
// permutes: the query tile has its dimensions in the same order, and the
// outputs' columns are put right at the end.  About 30 instructions per 16
// codes; four warps took 1.6 us per tile of keys and values, twice what the
// codes take from HBM.
QMM_DEV uint4 s8x8_to_bf16(uint32_t w0, uint32_t w1) {
  return make_uint4(s8_lanes_to_bf16(w0), s8_lanes_to_bf16(w0 >> 8), s8_lanes_to_bf16(w1), s8_lanes_to_bf16(w1 >> 8));
}

template <int D, int kRT>
QMM_DEV void convert_warps(const Ctx& x) {
  using G = Tg<D, true, kRT>;
  const AttnArgs& a = x.a;
  constexpr int kThr = 32 * G::kConvWarps, kPieces = D / 16;   // 16-code pieces of a row
  constexpr int kRows = kThr / kPieces;          // rows of a pass: a multiple of 8, so one swizzle for all
  const int lane = threadIdx.x & 31, tid = threadIdx.x - 384, row = tid / kPieces, p = tid % kPieces;
  // the second half's lanes store their odd 16 bytes first: no two lanes of a phase on one bank
  const uint32_t line = (p >> 2) * kHalf + row * 128, u = (p & 3) * 2, odd = p >> 2 & 1;
  const uint32_t src = smem_u32(x.smem) + G::kOffRaw + tid * 16;
  const uint32_t dst1 = smem_u32(x.smem) + G::kOffSlots + line + (((u + odd) ^ (row & 7)) << 4);
  const uint32_t dst2 = smem_u32(x.smem) + G::kOffSlots + line + (((u + 1 - odd) ^ (row & 7)) << 4);
  uint32_t rs = 0, r_phase = 0, cs = 0, c_phase = 1;
  AttnWalk walk;
  walk.start(x.sh->work);
  AttnItem it;
  while (walk.next(a, x.sh->work, G::kShape, it)) {
#pragma unroll 1
    for (int i = 0; i < 2 * it.seg; ++i) {
      if (!x.wait_all(&x.sh->bar.raw_full[rs], r_phase)) return;
      if (!x.wait_all(&x.sh->bar.empty[cs], c_phase)) return;
#pragma unroll
      for (int k = 0; k < kTok / kRows; ++k) {
        const uint4 c = lds128(src + rs * G::kRaw + k * kThr * 16);
        const uint4 lo = s8x8_to_bf16(c.x, c.y), hi = s8x8_to_bf16(c.z, c.w);
        const uint32_t at = cs * G::kTile + k * kRows * 128;
        sts128(dst1 + at, odd ? hi : lo);
        sts128(dst2 + at, odd ? lo : hi);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&x.sh->bar.full[cs]);
        mbar_arrive(&x.sh->bar.raw_empty[rs]);
      }
      if (++rs == G::kRawSlots) rs = 0, r_phase ^= 1;
      if (++cs == G::kSlots) cs = 0, c_phase ^= 1;
    }
  }
}

// ---- bf16: warp 3 cleans the value tiles that hold tokens which a row may not
// see, and hands them on ----
// Eight 16-byte pieces per lane are tested together: exponents of all ones
// carry into the sign bit.
template <int D, int kRT>
QMM_DEV void clean_warp(const Ctx& x) {
  using G = Tg<D, false, kRT>;
  const AttnArgs& a = x.a;
  constexpr int kP = D / 8;                      // pieces of a row
  constexpr int kBatch = 32 * 8 / kP;            // rows of a batch
  const int lane = threadIdx.x & 31, t_lane = lane / kP, p = lane % kP;
  uint32_t seq = 0, phases = 0;                  // phases: a bit per slot
  Ring vals(G::kKeySlots, G::kSlots - G::kKeySlots, 0);
  AttnWalk walk;
  walk.start(x.sh->work);
  AttnItem it;
  for (; walk.next(a, x.sh->work, G::kShape, it); ++seq) {
#pragma unroll 1
    for (int i = 0; i < it.seg; ++i) {
      const uint32_t slot = vals.slot;
      vals.next();
      const int tok0 = (it.kv0 + i) * kTok;
      if (tok0 + kTok <= it.seen) continue;
      const uint32_t parity = (phases >> slot) & 1;
      phases ^= 1u << slot;
      if (!x.wait_all(&x.sh->bar.tail_full[slot], parity)) return;
      const uint32_t base = smem_u32(x.smem) + G::kOffSlots + slot * G::kTile + (p >> 3) * kHalf;
      bool bad = false;
#pragma unroll 1
      for (int t0 = 0; t0 < kTok; t0 += kBatch) {
        if (tok0 + t0 + kBatch <= it.seen) continue;
        auto at = [&](int k) {
          const int t = t0 + k * (32 / kP) + t_lane;
          return base + t * 128 + (((p & 7) ^ (t & 7)) << 4);
        };
        uint4 v[8];
        uint32_t hit = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = lds128(at(k));
#pragma unroll
          for (int e = 0; e < 4; ++e) hit |= (u4_get(v[k], e) & 0x7F807F80u) + 0x00800080u;
        }
        if (!__any_sync(0xffffffffu, hit & 0x80008000u) && tok0 + t0 + kBatch <= it.len) continue;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          const int tok = tok0 + t0 + k * (32 / kP) + t_lane;
          if (tok < it.seen) continue;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (tok < it.len) {
            w = lds128(at(k));
            if (!bf16_drop_nonfinite(w)) continue;
            bad = true;
          }
          sts128(at(k), w);
        }
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) x.sh->bad[seq % kBadRing] = seq + 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x.sh->bar.full[slot]);
    }
  }
}

// ---- warp 1 (bf16: 1 and 2): the products ----
// A bf16 cache has a warp for the scores and one for the products with the
// values: nothing orders the two but the barriers, so neither waits while the
// other could issue.  With int8 (P over S) one warp issues both, in order.
// A warp runs in step and one lane issues: operands that only the issuing
// lane held would each be moved to a uniform register first, and 16 or 32
// products per tile (64 to 80 cycles each) leave no time for that.
template <int D, bool kS8, int kRT>
QMM_DEV void mma_warp(const Ctx& x, bool do_scores, bool do_values) {
  using G = Tg<D, kS8, kRT>;
  const AttnArgs& a = x.a;
  TBars& b = x.sh->bar;
  constexpr uint32_t kIdS = idesc_f16(128, kTok, true), kIdO = idesc_f16(128, D, true) | kIdescBMnMajor;
  const uint32_t q_s = smem_u32(x.smem), slots = q_s + G::kOffSlots;
  const uint32_t one = elect_one();
  uint32_t seq = 0, s_phase = 1, p_phase[2] = {0, 0};
  Ring keys(0, G::kKeySlots, 0), vals(G::kKeySlots, G::kSlots - G::kKeySlots, 0);   // int8: `keys` for both
  AttnWalk walk;
  walk.start(x.sh->work);
  AttnItem it;
  for (; walk.next(a, x.sh->work, G::kShape, it); ++seq) {
    if (do_scores && !x.wait_all(&b.q_full, seq & 1)) return;
    // Steps: (tile, stream) pairs, with kRT == 1 a tile each, streams in turn.
    const int streams = kRT == 2 && it.n_rows > 128 ? 2 : 1;   // on every tile (kRT == 2)
    const int steps = it.seg * streams, lead = kRT == 1 ? 2 : streams;
    uint32_t k_slot = 0, v_slot = 0;
    auto take = [&](Ring& ring, uint32_t& held) {
      held = ring.slot;
      if (!x.wait_all(&b.full[held], ring.phase)) return false;
      ring.next();
      return true;
    };
    auto scores = [&](int q) {
      const int st = kRT == 1 || streams == 2 ? q & 1 : 0;
      const bool opens = kRT == 1 || st == 0, closes = kRT == 1 || st == streams - 1;
      if (opens && !take(keys, k_slot)) return false;
      if constexpr (G::kShared) {                // the step before has been read
        if (!x.wait_all(&b.s_free, s_phase)) return false;
        s_phase ^= 1;
      }
      tc_fence_after();
      // the address fields do not carry past their 14 bits: shared memory ends below 2^18
      const uint64_t q_desc = desc_kmajor_sw128(q_s + (kRT == 2 ? st * G::kTile : 0));
      const uint64_t k_desc = desc_kmajor_sw128(slots + k_slot * G::kTile);
      const uint32_t d = G::kShared ? kColS : kColS + 128 * st;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
        umma_f16_one(one, d, q_desc + at, k_desc + at, kIdS, k > 0);
      }
      umma_commit_one(one, &b.s_full[st]);
      if (closes) umma_commit_one(one, &b.empty[k_slot]);
      return true;
    };
    auto values = [&](int q) {
      const int st = kRT == 1 || streams == 2 ? q & 1 : 0;
      const bool opens = kRT == 1 || st == 0, closes = kRT == 1 || st == streams - 1;
      if (!x.wait_all(&b.p_ready[st], p_phase[st])) return false;
      p_phase[st] ^= 1;
      if (q == 0 && !x.wait_all(&b.o_free, (seq & 1) ^ 1)) return false;
      if (opens && !take(kS8 ? keys : vals, v_slot)) return false;
      tc_fence_after();
      const uint64_t v_desc = desc_mnmajor_sw128(slots + v_slot * G::kTile, kHalf);
      const uint32_t d = kColO + 128 * st, p = G::kShared ? kColP + 64 * st : kColS + 128 * st;
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k)
        umma_f16_ta_one(one, d, p + 8 * k, v_desc + k * (2048 >> 4), kIdO, k > 0 || q >= (kRT == 1 ? 2 : streams));
      if (G::kShared || q + (kRT == 1 ? 2 : streams) >= steps) umma_commit_one(one, &b.o_done[st]);
      if (closes) umma_commit_one(one, &b.empty[v_slot]);
      return true;
    };
#pragma unroll 1
    for (int q = -lead; q < steps; ++q) {
      if (do_values && q >= 0 && !values(q)) return;
      if (do_scores && q + lead < steps && !scores(q + lead)) return;
    }
  }
}

// ---- warps 4..11: the rows ----
// The exponentials of one tile of 128 rows x 128 tokens, by four warps of 32
// rows: scores of the warp's rows in TMEM at t_s become weights (bf16, in half
// the columns).
//
// bf16: one row per lane, all of its scores in registers at once, so that the
// columns are free for the other stream's scores as soon as they are read.
struct RowsBf16 {
  float m = -INFINITY;                           // the row's reference, before the scale c
  uint64_t l = 0;                                // the weights' sum, in two halves
  QMM_DEV void own(float& om, float& ol) const {
    float lo, hi;
    f2_unpack(l, lo, hi);
    om = m;
    ol = lo + hi;
  }
  // loaded(): the scores have been read.  pv_done(): waits until the products
  // with the weights before have run (has_o: there were some).
  template <typename Seen, typename Loaded, typename PvDone, typename Rescale>
  QMM_DEV bool tile(uint32_t t_s, uint32_t t_p, float c, float slack, bool masked, Seen seen, bool low, bool has_o,
                    Loaded loaded, PvDone pv_done, Rescale rescale) {
    float s[kTok];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t r[32];
      tmem_ld32(t_s + 32 * q, r);
#pragma unroll
      for (int e = 0; e < 32; ++e) s[32 * q + e] = __uint_as_float(r[e]);
    }
    tmem_wait_ld();
    loaded();
    if (masked) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = seen(32 * q);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!((w >> e) & 1)) s[32 * q + e] = -INFINITY;
      }
    }
    float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int e = 4; e < kTok; e += 2) t4[(e >> 1) & 3] = fmaxf(fmaxf(t4[(e >> 1) & 3], s[e]), s[e + 1]);
    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
    const bool move = top > m + slack || (m == -INFINITY && top > -INFINITY);
    bool wait = has_o;
    if (__any_sync(0xffffffffu, move)) {
      const float next = move ? top : m;
      const float f = move ? exp2_approx((m - next) * c) : 1.f;   // m = -infinity: 0
      l = f2_mul(l, f2_pack(f, f));
      if (has_o) {
        if (!pv_done()) return false;
        wait = false;
        rescale(f);
      }
      m = next;
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    const uint64_t c2 = f2_pack(c, c), mc2 = f2_pack(-mc, -mc);
    uint64_t l2 = 0;
    uint32_t p[kTok / 2];
    auto weights = [&](auto low_parts) {
#pragma unroll
      for (int e = 0; e < kTok; e += 2) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), c2, mc2), x0, x1);
        x0 = exp2_approx(x0);
        x1 = exp2_approx(x1);
        if (e & 2) l2 = f2_add(l2, f2_pack(x0, x1));
        else l = f2_add(l, f2_pack(x0, x1));
        uint32_t w = bf16_pair(x0, x1);
        if constexpr (decltype(low_parts)::value) w = bf16_pair(x0 - bf16lo_to_f32(w), x1 - bf16hi_to_f32(w));
        p[e >> 1] = w;
      }
    };
    if (low) weights(std::true_type{});
    else weights(std::false_type{});
    l = f2_add(l, l2);
    if (wait && !pv_done()) return false;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t w[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) w[e] = p[32 * q + e];
      tmem_st32(t_p + 32 * q, w);
    }
    return true;
  }
};

// int8: two blocks of 16 rows in the layout of mma.sync accumulators, columns
// 2c, 2c + 1 of every eight of rows g and g + 8 per thread, so that a token's
// scales serve two rows of each lane.  Shared memory is what an int8 tile
// runs out of (codes in and out of the converters, three operands, scales):
// with a row per lane each scale is a broadcast of its own and the tile took
// 1.2 times as long.
struct RowsS8 {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // rows g, g + 8, g + 16, g + 24
  uint64_t l[4] = {0, 0, 0, 0};
  // this lane's own row: its reference and sum
  QMM_DEV void own(float& om, float& ol) const {
    const int lane = threadIdx.x & 31;
    om = ol = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      f2_unpack(l[k], lo, hi);
      lo += hi;
      lo += __shfl_xor_sync(0xffffffffu, lo, 1);
      lo += __shfl_xor_sync(0xffffffffu, lo, 2);
      const float mk = __shfl_sync(0xffffffffu, m[k], 4 * (lane & 7)), lk = __shfl_sync(0xffffffffu, lo, 4 * (lane & 7));
      if ((lane >> 3) == k) om = mk, ol = lk;
    }
  }
  // scales: the tile's 128 key scales, then its value scales.
  template <typename Seen, typename Rescale>
  QMM_DEV void tile(uint32_t t_s, const float* scales, float c, float slack, bool masked, Seen seen_at, bool low,
                    bool has_o, Rescale rescale) {
    const float2* sc = reinterpret_cast<const float2*>(scales);
    uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};     // of this lane's row
    if (masked) {
#pragma unroll
      for (int q = 0; q < 4; ++q) seen[q] = seen_at(32 * q);
    }
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = lane & 3;
    bool moved = false;
    float f_other[2] = {1.f, 1.f};               // block 0's factors, in block 1's turn
#pragma unroll 1
    for (int blk = 0; blk < 2; ++blk) {
      float s[64];
      float2 ks[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) ks[i] = sc[4 * i + c2];
      {
        uint32_t r[64];
        tmem_ld_16x256b_x16(t_s + ((uint32_t)(16 * blk) << 16), r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 64; ++e) s[e] = __uint_as_float(r[e]);
      }
#pragma unroll
      for (int e = 0; e < 64; e += 2)
        f2_unpack(f2_mul(f2_pack(s[e], s[e + 1]), f2_pack(ks[e >> 2].x, ks[e >> 2].y)), s[e], s[e + 1]);
      if (masked) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t w = __shfl_sync(0xffffffffu, seen[q], 16 * blk + 8 * hf + g) >> (2 * c2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!((w >> (8 * j + e)) & 1)) s[16 * q + 4 * j + 2 * hf + e] = -INFINITY;
          }
      }
      float f[2], mc[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float t0 = s[2 * hf], t1 = s[2 * hf + 1];
#pragma unroll
        for (int e = 4; e < 64; e += 8) {
          t0 = fmaxf(fmaxf(t0, s[e + 2 * hf]), s[e + 2 * hf + 1]);
          if (e + 4 < 64) t1 = fmaxf(fmaxf(t1, s[e + 4 + 2 * hf]), s[e + 5 + 2 * hf]);
        }
        float top = fmaxf(t0, t1);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float was = m[hf];
        const bool move = top > was + slack || (was == -INFINITY && top > -INFINITY);
        m[hf] = move ? top : was;
        moved |= move;
        f[hf] = move ? exp2_approx((was - top) * c) : 1.f;   // was -infinity: 0
        l[hf] = f2_mul(l[hf], f2_pack(f[hf], f[hf]));
        mc[hf] = m[hf] == -INFINITY ? 0.f : -m[hf] * c;
      }
      if (blk == 1 && has_o && __any_sync(0xffffffffu, moved)) {
        const int from = 4 * (lane & 7);         // each lane its own row's factor
        const float f0 = __shfl_sync(0xffffffffu, f_other[0], from), f1 = __shfl_sync(0xffffffffu, f_other[1], from);
        const float f2 = __shfl_sync(0xffffffffu, f[0], from), f3 = __shfl_sync(0xffffffffu, f[1], from);
        rescale(lane < 16 ? (lane < 8 ? f0 : f1) : (lane < 24 ? f2 : f3));
      }
      f_other[0] = f[0];
      f_other[1] = f[1];
      const uint64_t cc = f2_pack(c, c), mc2[2] = {f2_pack(mc[0], mc[0]), f2_pack(mc[1], mc[1])};
#pragma unroll
      for (int h = 0; h < 2; ++h) {              // 64 tokens at a time, over columns that have been read
        float2 vs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) vs[i] = sc[kTok / 2 + 32 * h + 4 * i + c2];
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int hf = j & 1, e = 32 * h + 2 * j;
          f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), cc, mc2[hf]), s[e], s[e + 1]);
          s[e] = exp2_approx(s[e]);
          s[e + 1] = exp2_approx(s[e + 1]);
          l[hf] = f2_add(l[hf], f2_pack(s[e], s[e + 1]));
          f2_unpack(f2_mul(f2_pack(s[e], s[e + 1]), f2_pack(vs[j >> 1].x, vs[j >> 1].y)), s[e], s[e + 1]);
          p[j] = bf16_pair(s[e], s[e + 1]);
        }
        if (low) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int e = 32 * h + 2 * j;
            p[j] = bf16_pair(s[e] - bf16lo_to_f32(p[j]), s[e + 1] - bf16hi_to_f32(p[j]));
          }
        }
        tmem_st_16x128b_x8(t_s + ((uint32_t)(16 * blk) << 16) + 32 * h, p);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {           // the blocks take turns in m[0..1], l[0..1]
        const float t = m[hf];
        m[hf] = m[2 + hf];
        m[2 + hf] = t;
        const uint64_t u = l[hf];
        l[hf] = l[2 + hf];
        l[2 + hf] = u;
      }
    }
  }
};

template <bool kS8> struct RowsOf { using type = RowsBf16; };
template <> struct RowsOf<true> { using type = RowsS8; };

template <int kRegs>
QMM_DEV void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
QMM_DEV void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

template <int D, bool kS8, bool kQF32, int kRT>
QMM_DEV AttnOwned row_warps(const Ctx& x) {
  using G = Tg<D, kS8, kRT>;
  const AttnArgs& a = x.a;
  TBars& b = x.sh->bar;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int st = (wid - 4) >> 2, quarter = wid & 3;
  const int trow = 32 * quarter + lane;          // lane of TMEM, row of the tile
  const uint32_t tlane = (uint32_t)(32 * quarter) << 16;
  const uint32_t t_s = tlane + kColS + (G::kShared ? 0 : 128 * st);
  const float c = a.scale_log2, slack = 8.f / c;
  AttnOwned owned{};
  uint32_t seq = 0, s_count = 0, o_count = 0, tiles = 0, syncs = 0;
  auto sync8 = [&]() {                           // the eight warps
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.sync);
    return x.wait_all(&b.sync, syncs++ & 1);
  };
  // A bf16 row's scores fill the registers.  With 256 rows, where the products
  // leave the least slack, the walk and its item are kept in shared memory (16
  // trees of 64 nodes over 11k tokens 174 -> 166 us, 4 chunks of 400 over 3k 77
  // -> 75.5; with 128 rows or int8 the registers last and it would cost 1 to 2 %).
  constexpr bool kItemOut = kRT == 2 && !kS8;
  RowItem local;
  auto now = [&]() -> RowItem& { return kItemOut ? x.sh->item[wid - 4] : local; };
  auto next = [&](bool first) {
    RowItem& to = now();
    if (kItemOut) __syncwarp();
    if (!kItemOut || lane == 0) {
      if (first) to.walk.start(x.sh->work);
      to.more = to.walk.next(a, x.sh->work, G::kShape, to.it);
    }
    if (kItemOut) __syncwarp();
  };
  next(true);
  for (;; ++seq) {
    if (!now().more) break;
    const AttnItem& it = now().it;
    const int seg = it.seg;
    if (it.pieces > 0) owned = attn_owned(it);
    const bool split = kRT == 1 && it.n_rows <= 64;   // lanes 64..127: the same rows, the weights' low parts
    const bool low = split && trow >= 64;
    const int rr = kRT == 2 ? 128 * st + trow : split ? trow & 63 : trow;
    const bool live = rr < it.n_rows, active = __any_sync(0xffffffffu, live);
    const int row = it.row0 + rr, node = row / a.group;
    // the query rows, whole rows at a time (with kRT == 1 each stream's warp
    // takes 16 of its quarter's 32)
    {
      constexpr int kCh = D / 8;                 // 16-byte pieces of a bf16 row
      constexpr int kAt = 32 / kCh;              // rows of a load
      constexpr int kLoads = (kRT == 1 ? 16 : 32) / kAt;
      const int ch = lane % kCh, r_first = kRT == 1 ? 16 * st : 0;
      const int64_t qo = live ? attn_q_row(a, it.q, it.h, row) : -1;
      const uint32_t base = smem_u32(x.smem) + (kRT == 2 ? st * G::kTile : 0) + (ch >> 3) * kHalf;
#pragma unroll (kS8 ? 8 : 16)
      for (int j = 0; j < kLoads; ++j) {
        const int rl = r_first + j * kAt + lane / kCh, tr = 32 * quarter + rl;
        const int64_t at = __shfl_sync(0xffffffffu, qo, rl);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (at >= 0) {
          if constexpr (kQF32) {
            const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + 8 * ch);
            const float4 f0 = f[0], f1 = f[1];
            v = make_uint4(bf16_pair(f0.x, f0.y), bf16_pair(f0.z, f0.w), bf16_pair(f1.x, f1.y), bf16_pair(f1.z, f1.w));
          } else {
            v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at + 8 * ch);
          }
        }
        if constexpr (kS8)                       // the converters' order: 0, 2, 1, 3 of each four
          v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                         __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        sts128(base + tr * 128 + (((ch & 7) ^ (tr & 7)) << 4), v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.q_full);
      // a stream without rows must not get an item ahead of the other
      if (kRT == 2 && !x.wait_all(&b.q_full, seq & 1)) return owned;
    }

    typename RowsOf<kS8>::type rows;             // references and sums
    const bool has = kRT == 1 || it.n_rows > 128 * st;   // this stream has products
    const int step = kRT == 1 ? 2 : 1, first_tok = it.kv0 * kTok, seen_tok = it.seen;
    for (int i = kRT == 1 ? st : 0; i < seg; i += step) {
      const uint32_t sc = (tiles + i) % kScaleRing;
      const float* ksc = nullptr;                // the tile's 128 key scales, then its value scales
      if constexpr (kS8) {
        if (!x.wait_all(&b.sc_full[sc], ((tiles + i) / kScaleRing) & 1)) return owned;
        ksc = reinterpret_cast<const float*>(x.smem + G::kOffScale + sc * (2 * kTok * 4));
      }
      if (has) {
        if (!x.wait_all(&b.s_full[st], s_count++ & 1)) return owned;
        tc_fence_after();
        auto loaded = [&]() {
          if constexpr (G::kShared) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.s_free);
          }
        };
        auto pv_done = [&]() {
          if (!x.wait_all(&b.o_done[st], o_count++ & 1)) return false;
          tc_fence_after();
          return true;
        };
        if (!active) {
          loaded();
          if (G::kShared && i >= step && !pv_done()) return owned;
        } else {
          const int tok0 = first_tok + i * kTok;
          const bool masked = tok0 + kTok > seen_tok;
          // O (of this lane's row) to a new reference
          auto rescale = [&](float f) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t r[16];
              tmem_ld16(tlane + kColO + 128 * st + 16 * q, r);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st16(tlane + kColO + 128 * st + 16 * q, r);
            }
          };
          auto seen = [&](int at) { return live ? attn_sees32(a, it.q, node, tok0 + at) : 0u; };
          if constexpr (kS8) {
            rows.tile(t_s, ksc, c, slack, masked, seen, low, i >= step, rescale);
          } else if (!rows.tile(t_s, tlane + kColP + 64 * st, c, slack, masked, seen, low, i >= step, loaded, pv_done,
                                rescale)) {
            return owned;
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.p_ready[st]);
      }
      if (kS8) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.sc_empty[sc]);
      }
    }
    tiles += seg;

    // ---- the item's end ----
    const bool own_tiles = has && (kRT == 2 || seg > st);
    if (own_tiles) {
      if (!x.wait_all(&b.o_done[st], o_count++ & 1)) return owned;
    }
    float own_m, sum;                            // of this lane's row
    rows.own(own_m, sum);
    float f[2] = {1.f, 1.f}, top = own_m;        // each stream's factor; maximum of the row
    if constexpr (kRT == 1) {
      x.sh->m[st][trow] = own_m;
      x.sh->l[st][trow] = sum;
      if (!sync8()) return owned;                // both streams' O and sums are there
      top = fmaxf(x.sh->m[0][rr], x.sh->m[1][rr]);
      sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // the row's own reference, for the lanes of its low parts another one;
        // without a maximum there is no weight, unless the scores were not numbers
        const float mk = x.sh->m[k][trow], ms = x.sh->m[k][rr], ls = x.sh->l[k][rr];
        f[k] = mk == -INFINITY ? (x.sh->l[k][trow] == 0.f ? 0.f : 1.f) : exp2_approx((mk - top) * c);
        sum += ls * (ms == -INFINITY ? (ls == 0.f ? 0.f : 1.f) : exp2_approx((ms - top) * c));
      }
    }
    tc_fence_after();
    const bool bad = x.sh->bad[seq % kBadRing] == seq + 1;
    // 16 columns of O at a time, of both streams with kRT == 1 (each takes half
    // of the columns).  Loops, not straight code: it runs once per item, and
    // fetching instructions would cost more than running them.
    constexpr int kCols = kRT == 1 ? D / 2 : D;
    const int d_first = kRT == 1 ? st * kCols : 0;
    // [64][D]: the low rows' part, over the query tile; 16-byte piece p of row t at p ^ (t & 7)
    float4* lows = reinterpret_cast<float4*>(x.smem) + (trow & 63) * (D / 4);
    auto load_o = [&](int d, float (&o)[16]) {
      uint32_t r[16];
      if constexpr (kRT == 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k >= seg) continue;             // stream 1 had no tile
          tmem_ld16(tlane + kColO + 128 * k + d, r);
          tmem_wait_ld();
          // a factor of 0 counts as well: 0 times a visible infinity or NaN
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(r[e]), f[k], o[e]);
        }
      } else {
        tmem_ld16(tlane + kColO + 128 * st + d, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(r[e]);
      }
      if constexpr (kS8) {                       // columns in order again
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float t = o[e + 1];
          o[e + 1] = o[e + 2];
          o[e + 2] = t;
        }
      }
    };
    if (split) {
      if (quarter >= 2 && active) {
#pragma unroll 1
        for (int d = d_first; d < d_first + kCols; d += 16) {
          float o[16];
          load_o(d, o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            lows[(d / 4 + e) ^ (trow & 7)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (!sync8()) return owned;
    }
    if (active && has && !(split && quarter >= 2)) {
      const float inv = !it.whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;   // no visible token: 0
      const int64_t slot = (2 * (int64_t)blockIdx.x + (it.kv0 > 0 ? 0 : 1)) * (128 * kRT) + rr;
      // Rows go out through shared memory, four lanes a row (a store of one
      // 16-byte piece of 32 rows takes eight times as long): over the warp's
      // own rows of the query tile, or (split) in place of the low parts.
      float4* stage = reinterpret_cast<float4*>(x.smem + (kRT == 2 ? st * G::kTile : st * 2048) + quarter * 4096);
      auto piece = [&](int r, int d, int e) -> float4& {
        return split ? reinterpret_cast<float4*>(x.smem)[(32 * quarter + r) * (D / 4) + ((d / 4 + e) ^ (r & 7))]
                     : stage[r * 4 + (e ^ ((r >> 1) & 3))];
      };
      const int64_t own = !live ? -1 : it.whole ? attn_out_row(a, it.q.first, it.h, row) - a.out : slot * D;
      int64_t to[4];                             // of the rows that this lane stores a piece of
#pragma unroll
      for (int j = 0; j < 4; ++j) to[j] = __shfl_sync(0xffffffffu, own, 8 * j + (lane >> 2));
#pragma unroll 1
      for (int d = d_first; d < d_first + kCols; d += 16) {
        float o[16];
        load_o(d, o);
        if (split) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = piece(lane, d, e);
            o[4 * e] += v.x, o[4 * e + 1] += v.y, o[4 * e + 2] += v.z, o[4 * e + 3] += v.w;
          }
        }
        if (bad && live) attn_add_nonfinite(a, it, kTok, node, d, o);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          piece(lane, d, e) = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 8 * j + (lane >> 2), e = lane & 3;
          const float4 v = piece(r, d, e);
          if (to[j] >= 0) {
            if (it.whole)
              *reinterpret_cast<uint2*>(a.out + to[j] + d + 4 * e) =
                  make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
            else
              *reinterpret_cast<float4*>(a.part_o + to[j] + d + 4 * e) = v;
          }
        }
      }
      if (live && !it.whole && d_first == 0) a.part_ml[slot] = make_float2(top == -INFINITY ? top : top * c, sum);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.o_free);
    // the query tile, the sums and (split) the low parts are written again for the next item
    if (kRT == 1 && !sync8()) return owned;
    next(false);
  }
  return owned;
}

template <int D, bool kS8, bool kQF32, int kRT>
__global__ void __launch_bounds__(Tg<D, kS8, kRT>::kThreads, 1)
attn_tiles_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, uint32_t box) {
  using G = Tg<D, kS8, kRT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  TShared& sh = *reinterpret_cast<TShared*>(smem + G::kBytes);
  if (smem_u32(smem) & 1023u) {                  // the swizzled tiles need it; no static shared memory precedes
    set_status(a.dev_status, QMM_ERR_UNSUPPORTED);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TBars& b = sh.bar;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(&b.full[i], kS8 ? G::kConvWarps : 1);   // converters, or the loads or the cleaner
      mbar_init(&b.empty[i], 1);
      mbar_init(&b.tail_full[i], 1);
    }
    for (int i = 0; i < G::kRawSlots; ++i) {
      mbar_init(&b.raw_full[i], 1);
      mbar_init(&b.raw_empty[i], G::kConvWarps);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&b.sc_full[i], 2);
      mbar_init(&b.sc_empty[i], kRT == 1 ? 4 : 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.p_ready[i], 4);
      mbar_init(&b.o_done[i], 1);
    }
    mbar_init(&b.s_free, 4);
    mbar_init(&b.q_full, 8);
    mbar_init(&b.o_free, 8);
    mbar_init(&b.sync, 8);
    mbar_init(&b.done, kS8 ? 1 : 2);
    sh.abort = 0;
    for (int i = 0; i < kBadRing; ++i) sh.bad[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Ctx x{a, &sh, smem, box};
  AttnOwned owned{};
  AttnWork work;
  const bool any = attn_find_work<G::kThreads>(a, G::kShape, &sh.find, work);
  if (threadIdx.x == 0) sh.work = work;
  __syncthreads();
  if (any) {
    // Registers per warpgroup, of what the launch has: bf16 72 + 2 * 216 = 504 = 3 * 168;
    // int8 72 + 2 * 144 + 2 * 56 = 472 <= 5 * 96.
    if (warp < 4) {
      regs_dec<72>();
      if (warp == 0) {
        load_warp<D, kS8, kRT>(x, mk, mv);
      } else if (warp == 1 || (!kS8 && warp == 2)) {
        mma_warp<D, kS8, kRT>(x, warp == 1, kS8 || warp == 2);
      } else {
        if constexpr (kS8) scale_warps<D, kRT>(x);
        else clean_warp<D, kRT>(x);
      }
    } else if (warp < 12) {
      regs_inc<kS8 ? 144 : 216>();
      owned = row_warps<D, kS8, kQF32, kRT>(x);
    } else {
      if constexpr (kS8) {
        regs_dec<56>();
        convert_warps<D, kRT>(x);
      }
    }
    __syncwarp();
  }
  if (warp == 4 && lane == 0) attn_post_owned(a, owned);
  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (sh.abort && warp == 0 && lane == 0) {
    // copies that nobody waited for may still be in flight
    auto drain = [](uint64_t* bars, int n) {
      for (int i = 0; i < n; ++i)
        for (uint32_t ph = 0; ph < 2; ++ph) mbar_drain(&bars[i], ph, 10000000ull);
    };
    drain(kS8 ? b.raw_full : b.full, kS8 ? G::kRawSlots : G::kSlots);
    if (!kS8) drain(b.tail_full, G::kSlots);
  }
  if (sh.abort && (warp == 1 || (!kS8 && warp == 2))) umma_commit_one(elect_one(), &b.done);
  if (warp == 1) {
    // without an abort every product has been waited for
    if (sh.abort && lane == 0) mbar_drain(&b.done, 0, 100000000ull);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(sh.tmem, 512);
  }
}

template <int D, bool kS8, bool kQF32, int kRT>
cudaError_t launch_tiles(const AttnArgs& a, cudaStream_t stream) {
  using G = Tg<D, kS8, kRT>;
  constexpr int kSmem = G::kBytes + (int)sizeof(TShared);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  uint32_t box = 8;
  while (box < (uint32_t)kTok && a.cache.page_size % (2 * box) == 0) box *= 2;
  CUtensorMap mk, mv;
  const KvView& c = a.cache;
  if (!make_tmap_kv(&mk, c.k, kS8, D, c.page_size, c.n_heads, c.n_pages, c.st_token, c.st_head, c.st_page, box) ||
      !make_tmap_kv(&mv, c.v, kS8, D, c.page_size, c.n_heads, c.n_pages, c.st_token, c.st_head, c.st_page, box))
    return cudaErrorInvalidValue;
  auto kern = attn_tiles_kernel<D, kS8, kQF32, kRT>;
  static std::atomic<uint64_t> set{0};
  const cudaError_t err = set_once(set, (const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3(a.grid), dim3(G::kThreads), kSmem, stream, a, mk, mv, box);
}

template <int D, bool kS8>
cudaError_t launch_typed(const AttnArgs& a, int rows_per_tile, bool q_f32, cudaStream_t stream) {
  if (rows_per_tile == 128)
    return q_f32 ? launch_tiles<D, kS8, true, 1>(a, stream) : launch_tiles<D, kS8, false, 1>(a, stream);
  return q_f32 ? launch_tiles<D, kS8, true, 2>(a, stream) : launch_tiles<D, kS8, false, 2>(a, stream);
}

}  // namespace

cudaError_t launch_attn_tiles(const AttnArgs& a, int rows_per_tile, bool q_f32, bool cache_s8, int head_dim,
                              cudaStream_t stream) {
  if (head_dim == 128)
    return cache_s8 ? launch_typed<128, true>(a, rows_per_tile, q_f32, stream)
                    : launch_typed<128, false>(a, rows_per_tile, q_f32, stream);
  return cache_s8 ? launch_typed<64, true>(a, rows_per_tile, q_f32, stream)
                  : launch_typed<64, false>(a, rows_per_tile, q_f32, stream);
}

}  // namespace qmm

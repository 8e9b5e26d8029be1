// Low-rank adapters of many requests beside a shared projection:
//     out[m] = base[m] + s_a B_a (A_a x_m),   a = ids[m]
// with x_m of K values, A_a [r][K], B_a [N][r], r up to 256.
//
// Bound: bytes.  base and out are 8 N bytes a row and X 2 K; the products are
// 2 r (K + N) operations a row, a few per byte for ordinary ranks.  So the
// kernels keep rows of one adapter together (each adapter's A and B are read
// once per tile of rows) and stream X, base and out once.  Here: calls of few rows,
// one launch, 16 rows to a tile and mma.sync; and how many rows are brought together
// for lora_umma.cu.
//
// A call of few rows is a chain of latencies: the rows' ids, X and A, the sums' meeting,
// B and base.  256 rows over 40 adapters of ranks 5 to 64 at K = N = 4096 (33 MB) take
// 17.9 us, of which 3 find the rows, 4 are the first product, 4 the meeting and 5 the
// second (4.9 at a copy's rate); 8 rows at K = 1024, N = 2048 and rank 16 6.3 us.
//
// The inner sums h = A x are fp32.  For the second product h * s_a is written
// as two bf16 terms, h = hi + lo within 2^-16 |h|: with one term (2^-8) the
// rounding of h would be far above the fp32 rounding of out.
#include <algorithm>
#include <atomic>

#include "beside.h"
#include "kv_cache.h"
#include "lora_work.cuh"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kTile = 16;                 // rows of an item of a call of few rows, all of one adapter
constexpr int kRouteThreads = 1024;
constexpr int kThreads = 256;
constexpr int kMaxCluster = kLoraMaxCluster;

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// ---- rows by adapter ---------------------------------------------------------
// One block.  Its first `segs` warps take a stretch of the rows each and count them
// by adapter in a column of the table; the counts' sums over warps and adapters
// give every row a place that keeps the rows' order, so that a prompt's rows stay
// together and the items are the same from run to run.
__global__ void __launch_bounds__(kRouteThreads)
lora_route_kernel(LoraArgs a, LoraWork w, bool copy_none, int segs) {
  extern __shared__ int smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int buckets = a.n_adapters + 1;   // the last: no adapter
  const int pitch = segs + 1;             // [buckets][segs]: a warp's rows of a bucket, then its next place among them
  int* table = smem;
  int* home = smem + pitch * buckets;     // [buckets]: an adapter's bucket (itself, or none), -1 for a bad rank
  int* first = home + buckets;            // [buckets]: the bucket's first place
  __shared__ int2 warp_sums[32];
  __shared__ int2 carry;
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int seg = ((a.M + segs - 1) / segs + 31) / 32 * 32;
  const int begin = min(warp * seg, a.M), end = warp < segs ? min(begin + seg, a.M) : begin;
  constexpr int kAhead = 8;               // loads under way
  int id[kAhead];
  auto load_ids = [&](int m0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) id[u] = m0 + u * 32 + lane < end ? a.ids[m0 + u * 32 + lane] : -1;
  };
  load_ids(begin);
  for (int i = tid; i < pitch * buckets; i += kRouteThreads) table[i] = 0;
  for (int b = tid; b < buckets; b += kRouteThreads) {
    const int r = a.ranks != nullptr && b < a.n_adapters ? a.ranks[b] : 1;
    home[b] = r < 0 || r > a.max_rank ? -1 : r == 0 ? a.n_adapters : b;
  }
  if (tid == 0) carry = make_int2(0, 0);
  __syncthreads();
  // the bucket of row m with adapter `of`; -1 past the rows
  auto bucket_of = [&](int m, int of, bool report) {
    if (m >= end) return -1;
    if (of == -1) return a.n_adapters;
    const int b = of < 0 || of >= a.n_adapters ? -1 : home[of];
    if (b >= 0) return b;
    if (report) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    return a.n_adapters;
  };
  // lanes of the same bucket; in a prompt all are, which is found out faster
  auto same_as = [&](int b) {
    const bool one = __all_sync(0xffffffffu, b == __shfl_sync(0xffffffffu, b, 0));
    return one ? 0xffffffffu : __match_any_sync(0xffffffffu, b);
  };
  for (int m0 = begin; m0 < end; m0 += 32 * kAhead) {
    if (m0 != begin) load_ids(m0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (m0 + u * 32 >= end) break;
      const int b = bucket_of(m0 + u * 32 + lane, id[u], true);
      const uint32_t same = same_as(b);
      if (b >= 0 && lane == __ffs(same) - 1) table[b * pitch + warp] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // per bucket: places of the warps' rows among its rows, and their number behind them
  for (int b = warp; b < buckets; b += kRouteThreads / 32) {
    const int n = lane < segs ? table[b * pitch + lane] : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    __syncwarp();
    if (lane < segs) table[b * pitch + lane] = s - n;
    if (lane == 31) table[b * pitch + segs] = s;
  }
  __syncthreads();
  for (int b0 = 0; b0 < buckets; b0 += kRouteThreads) {
    const int b = b0 + tid;
    const int n = b < buckets ? table[b * pitch + segs] : 0;
    const bool none = b == a.n_adapters;
    const int t = none && !copy_none ? 0 : (n + kLoraTile - 1) / kLoraTile;
    int2 s = make_int2(n, t);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
      if (lane >= o) s.x += x, s.y += y;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    const int2 sums = lane < warp ? warp_sums[lane] : make_int2(0, 0);
    int2 before = carry;
    before.x += __reduce_add_sync(0xffffffffu, sums.x), before.y += __reduce_add_sync(0xffffffffu, sums.y);
    const int start = before.x + s.x - n, tile0 = before.y + s.y - t;
    if (b < buckets) first[b] = start;
    if (none) w.head[0] = tile0, w.head[1] = tile0 + t;
    // an adapter's tiles, by its warp
    for (uint32_t left = __ballot_sync(0xffffffffu, t > 0); left != 0; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const int lt = __shfl_sync(0xffffffffu, t, l), ln = __shfl_sync(0xffffffffu, n, l);
      const int lf = __shfl_sync(0xffffffffu, start, l), l0 = __shfl_sync(0xffffffffu, tile0, l);
      const int lb = b0 + warp * 32 + l;
      for (int i = lane; i < lt; i += 32)
        w.tiles[l0 + i] =
            make_int4(lb == a.n_adapters ? -1 : lb, lf + i * kLoraTile, min(kLoraTile, ln - i * kLoraTile), 0);
    }
    __syncthreads();
    if (tid == kRouteThreads - 1) carry = make_int2(start + n, tile0 + t);
    __syncthreads();
  }
  const bool once = begin + 32 * kAhead >= end;   // the ids are still at hand
  for (int m0 = begin; m0 < end; m0 += 32 * kAhead) {
    if (!once) load_ids(m0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (m0 + u * 32 >= end) break;
      const int m = m0 + u * 32 + lane, b = bucket_of(m, id[u], false);
      const uint32_t same = same_as(b);
      if (b >= 0) w.rows[first[b] + table[b * pitch + warp] + __popc(same & ((1u << lane) - 1u))] = m;
      __syncwarp();
      if (b >= 0 && lane == __ffs(same) - 1) table[b * pitch + warp] += __popc(same);
      __syncwarp();
    }
  }
}

// ---- the products ------------------------------------------------------------
// The first n of eight bf16 values, zeros behind them.
QMM_DEV uint4 keep8(uint4 v, int n) {
  uint32_t* p = &v.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n <= 2 * i) p[i] = 0;
    else if (n == 2 * i + 1) p[i] &= 0xFFFFu;
  }
  return v;
}

// Four columns from `col` of a row, as far as they exist.
template <bool kVec>
QMM_DEV float4 load4(const float* row, int col, int N) {
  if constexpr (kVec) return col < N ? *reinterpret_cast<const float4*>(row + col) : make_float4(0, 0, 0, 0);
  return make_float4(col < N ? row[col] : 0.f, col + 1 < N ? row[col + 1] : 0.f, col + 2 < N ? row[col + 2] : 0.f,
                     col + 3 < N ? row[col + 3] : 0.f);
}
template <bool kVec>
QMM_DEV void store4(float* row, int col, int N, float4 v) {
  if constexpr (kVec) {
    if (col < N) *reinterpret_cast<float4*>(row + col) = v;
  } else {
    if (col < N) row[col] = v.x;
    if (col + 1 < N) row[col + 1] = v.y;
    if (col + 2 < N) row[col + 2] = v.z;
    if (col + 3 < N) row[col + 3] = v.w;
  }
}

// A warp's part of h for 16 rows and 8 kNT ranks from j0: chunks c0..c1 of 32 k.
// Both operands come straight from memory, 16 bytes (eight consecutive k) per
// lane: which k a fragment position stands for is free as long as both operands
// agree.  All loads of kU chunks are under way before the first product.
template <int kNT, int kU>
QMM_DEV void inner_part(const LoraArgs& a, const __nv_bfloat16* x0, const __nv_bfloat16* x1, const __nv_bfloat16* A,
                        int rank, int j0, int c0, int c1, float (&acc)[8][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c = c0; c < c1; c += kU) {
    uint4 p[kU], q[kU], b[kU][kNT];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = (c + u) * 32 + 8 * tig;
      const bool in = c + u < c1 && k < a.K;
      p[u] = in && x0 != nullptr ? ldg128(x0 + k) : zero;
      q[u] = in && x1 != nullptr ? ldg128(x1 + k) : zero;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const int j = j0 + 8 * n + g;
        b[u][n] = in && j < rank ? ldg128(A + j * a.a_rank + k) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        mma_bf16_16816(acc[n], p[u].x, q[u].x, p[u].y, q[u].y, b[u][n].x, b[u][n].y);
        mma_bf16_16816(acc[n], p[u].z, q[u].z, p[u].w, q[u].w, b[u][n].z, b[u][n].w);
      }
  }
}

// A warp's part of out: 16 rows, units of 32 columns from u0 in steps of `step`.
// Columns are dealt to fragment positions so that a lane's accumulators are four
// neighbouring columns of a row.  What the first unit reads is asked for by
// start(), long before h is there; the next unit's base is under way during the
// products of one.  kRC: chunks of 32 ranks, whose h stays in registers; 0: any.
template <bool kVec, int kRC>
struct Outer {
  const LoraArgs& a;
  const __nv_bfloat16* B;
  int rank;
  int64_t m0, m1;
  int u0, u1, step;
  uint4 b[kRC > 0 ? kRC : 3][4];
  float4 y[2][2];

  QMM_DEV void load_base(int u, float4 (&to)[2][2]) const {
    const int tig = threadIdx.x & 3;
    const float4 none = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int col = u * 32 + 16 * p + 4 * tig;
      to[0][p] = a.base != nullptr && m0 >= 0 && u < u1 ? load4<kVec>(a.base + m0 * a.ldb, col, a.N) : none;
      to[1][p] = a.base != nullptr && m1 >= 0 && u < u1 ? load4<kVec>(a.base + m1 * a.ldb, col, a.N) : none;
    }
  }
  QMM_DEV void load_b(int u, int c, uint4 (&to)[4]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int col = u * 32 + 16 * (n >> 1) + 4 * (g >> 1) + (g & 1) + 2 * (n & 1), j = c * 32 + 8 * tig;
      to[n] = j < rank && col < a.N && u < u1 ? ldg128(B + col * a.b_row + j) : make_uint4(0, 0, 0, 0);
    }
  }
  QMM_DEV void start() {
    if constexpr (kRC > 0) {
#pragma unroll
      for (int c = 0; c < kRC; ++c) load_b(u0, c, b[c]);
    } else {                                              // two chunks ahead of the products
      load_b(u0, 0, b[0]);
      load_b(u0, 1, b[1]);
    }
    load_base(u0, y);
  }
  QMM_DEV void products(float (&acc)[4][4], const uint4 (&h)[4], const uint4 (&w)[4], int left) const {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const uint4 v = keep8(w[n], left);
      mma_bf16_16816(acc[n], h[2].x, h[3].x, h[2].y, h[3].y, v.x, v.y);
      mma_bf16_16816(acc[n], h[2].z, h[3].z, h[2].w, h[3].w, v.z, v.w);
      mma_bf16_16816(acc[n], h[0].x, h[1].x, h[0].y, h[1].y, v.x, v.y);
      mma_bf16_16816(acc[n], h[0].z, h[1].z, h[0].w, h[1].w, v.z, v.w);
    }
  }
  // h: rows of hs values, the two terms
  QMM_DEV void finish(const uint16_t* hi, const uint16_t* lo, int hs) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int chunks = kRC > 0 ? kRC : (rank + 31) / 32;
    uint4 h[kRC > 0 ? kRC : 1][4];
    auto load_h = [&](int c, uint4 (&to)[4]) {
      const int j = c * 32 + 8 * tig;
      to[0] = *reinterpret_cast<const uint4*>(hi + g * hs + j);
      to[1] = *reinterpret_cast<const uint4*>(hi + (g + 8) * hs + j);
      to[2] = *reinterpret_cast<const uint4*>(lo + g * hs + j);
      to[3] = *reinterpret_cast<const uint4*>(lo + (g + 8) * hs + j);
    };
    auto store = [&](int u, const float (&acc)[4][4]) {
      bool nan0 = false, nan1 = false;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        nan0 |= acc[n][0] != acc[n][0] || acc[n][1] != acc[n][1];
        nan1 |= acc[n][2] != acc[n][2] || acc[n][3] != acc[n][3];
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int col = u * 32 + 16 * p + 4 * tig;
        const float(&e)[4] = acc[2 * p], (&f)[4] = acc[2 * p + 1];
        if (m0 >= 0 && !nan0)
          store4<kVec>(a.out + m0 * a.ldo, col, a.N,
                       make_float4(y[0][p].x + e[0], y[0][p].y + e[1], y[0][p].z + f[0], y[0][p].w + f[1]));
        if (m1 >= 0 && !nan1)
          store4<kVec>(a.out + m1 * a.ldo, col, a.N,
                       make_float4(y[1][p].x + e[2], y[1][p].y + e[3], y[1][p].z + f[2], y[1][p].w + f[3]));
      }
      if (nan0 || nan1) {                                  // an infinity in B, or NaN all the same
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int64_t m = i < 8 ? m0 : m1;
          const int col = u * 32 + i / 4 % 2 * 16 + 4 * tig + i % 4, at = (g + (i < 8 ? 0 : 8)) * hs;
          if ((i < 8 ? nan0 : nan1) && m >= 0 && col < a.N)
            a.out[m * a.ldo + col] = (a.base != nullptr ? a.base[m * a.ldb + col] : 0.f) +
                                     sum_of_terms(hi + at, lo + at, B + col * a.b_row, rank);
        }
      }
    };
    if constexpr (kRC > 0) {
#pragma unroll
      for (int c = 0; c < kRC; ++c) load_h(c, h[c]);
      for (int u = u0; u < u1; u += step) {
        float acc[4][4] = {};
        float4 next[2][2];
        load_base(u + step, next);
#pragma unroll
        for (int c = 0; c < kRC; ++c) {
          products(acc, h[c], b[c], rank - c * 32 - 8 * tig);
          load_b(u + step, c, b[c]);
        }
        store(u, acc);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) y[i][p] = next[i][p];
      }
    } else {
      float acc[4][4] = {};
      for (int u = u0, c = 0, ahead = u0, chunk = 2; u < u1;) {
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          if (u >= u1) break;
          if (chunk == chunks) chunk = 0, ahead += step;
          load_b(ahead, chunk++, b[(e + 2) % 3]);
          load_h(c, h[0]);
          products(acc, h[0], b[e], rank - c * 32 - 8 * tig);
          if (++c < chunks) continue;
          store(u, acc);
          c = 0, u += step;
          load_base(u, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] = 0.f;
        }
      }
    }
  }
};

// An item of a call of few rows: up to 16 rows of one adapter.
struct Item {
  int rows, rank;   // rows 0: none left for this cluster; rank 0: no adapter
  int adapter;
  float scale;
};

struct alignas(16) Smem {
  float part[kThreads / 32 * 16 * 68];   // sums of a warp: 16 rows by 64 ranks, beside or above the others'
  int rows[kTile];
  int counts[kThreads / 32];
  int ranks[kThreads];
  float scales[kThreads];
};
static_assert(sizeof(Smem) % 16 == 0, "h follows, read 16 bytes at a time");

constexpr int kOwnRows = 1536;            // rows of a call that may find its items in the kernel itself
// rows counted by adapter, in words
__host__ __device__ __forceinline__ int table_size(int n_adapters) { return (n_adapters + 1 + 127) / 128 * 128; }

// The item of this cluster, found by every block for itself: the rows are counted by
// adapter, an adapter's rows make items of 16 in their order, numbered by adapter and
// the rows without one last.  The row numbers go to rows[]; table holds
// table_size(n_adapters) words.
QMM_DEV Item own_item(const LoraArgs& a, int item, bool copy_none, int* table, Smem& sm) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int buckets = a.n_adapters + (copy_none ? 1 : 0), size = table_size(a.n_adapters);
  const int per = (a.M + kThreads - 1) / kThreads;         // groups of 32 rows per warp
  // the ids' loads and those of a small set's ranks and scales go together
  int id[kOwnRows / kThreads];                             // -1: past the rows, or nothing to do for the row
#pragma unroll
  for (int i = 0; i < kOwnRows / kThreads; ++i) {
    const int m = (warp * per + i) * 32 + lane;
    id[i] = -1;
    if (i < per && m < a.M) {
      id[i] = a.ids[m];
      if (id[i] < -1 || id[i] >= a.n_adapters) {
        if (blockIdx.x == 0) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
        id[i] = -1;
      }
      if (id[i] < 0 && copy_none) id[i] = a.n_adapters;
    }
  }
  const bool few = a.n_adapters <= kThreads;
  if (few && t < a.n_adapters) {
    sm.ranks[t] = a.ranks != nullptr ? a.ranks[t] : a.max_rank;
    sm.scales[t] = a.scales != nullptr ? a.scales[t] : 1.f;
  }
  for (int i = t * 4; i < size; i += kThreads * 4) *reinterpret_cast<int4*>(table + i) = make_int4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwnRows / kThreads; ++i)
    if (id[i] >= 0) atomicAdd(&table[id[i]], 1);
  __syncthreads();
  // every warp looks for the item's adapter, 128 of them at a time
  Item it{0, 0, -1, 1.f};
  int first = 0;
  for (int b0 = 0, before = 0; b0 < buckets; b0 += 128) {
    const int4 n = *reinterpret_cast<const int4*>(table + b0 + lane * 4);
    const int x = (n.x + kTile - 1) / kTile, y = x + (n.y + kTile - 1) / kTile, z = y + (n.z + kTile - 1) / kTile;
    const int w = z + (n.w + kTile - 1) / kTile;
    const int all = __reduce_add_sync(0xffffffffu, w);
    if (item >= before + all) {
      before += all;
      continue;
    }
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    const int at = item - before - (s - w);                // the item among this lane's four
    const int owner = __ffs(__ballot_sync(0xffffffffu, at >= 0 && at < w)) - 1;
    const int q = at < x ? 0 : at < y ? 1 : at < z ? 2 : 3;
    const int tile = at - (q == 0 ? 0 : q == 1 ? x : q == 2 ? y : z);
    const int rows = q == 0 ? n.x : q == 1 ? n.y : q == 2 ? n.z : n.w;
    it.adapter = __shfl_sync(0xffffffffu, b0 + lane * 4 + q, owner);
    first = __shfl_sync(0xffffffffu, tile * kTile, owner);
    it.rows = min(kTile, __shfl_sync(0xffffffffu, rows, owner) - first);
    break;
  }
  if (it.rows == 0) return it;                             // alike in every thread
  if (it.adapter < a.n_adapters) {
    if (few) {
      it.rank = sm.ranks[it.adapter], it.scale = sm.scales[it.adapter];
    } else {
      it.rank = a.ranks != nullptr ? a.ranks[it.adapter] : a.max_rank;
      if (a.scales != nullptr) it.scale = a.scales[it.adapter];
    }
  }
  // the rows' places among the adapter's
  uint32_t mine[kOwnRows / kThreads];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kOwnRows / kThreads; ++i) {
    mine[i] = __ballot_sync(0xffffffffu, id[i] == it.adapter);
    n += __popc(mine[i]);
  }
  if (lane == 0) sm.counts[warp] = n;
  __syncthreads();
  int place = -first;
  for (int w = 0; w < warp; ++w) place += sm.counts[w];
#pragma unroll
  for (int i = 0; i < kOwnRows / kThreads; ++i) {
    const int at = place + __popc(mine[i] & ((1u << lane) - 1u));
    if (id[i] == it.adapter && at >= 0 && at < kTile) sm.rows[at] = (warp * per + i) * 32 + lane;
    place += __popc(mine[i]);
  }
  __syncthreads();
  if (it.rank < 0 || it.rank > a.max_rank) {
    if (t == 0) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    it.rank = 0;
  }
  return it;
}

// The two halves of a barrier of the cluster's blocks.
QMM_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
QMM_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A cluster takes an item: up to 16 rows of one adapter.  First its blocks and
// their warps share K; every block adds up the blocks' sums over shared memory, in
// order, and keeps h as two bf16 terms.  Then the blocks and warps share the columns
// of out.
template <bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
lora_rows_kernel(LoraArgs a, int rs, int cluster, bool copy_none) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int hs = rs + 8;                                   // row stride of h: rows fall on different banks
  uint16_t* hi = reinterpret_cast<uint16_t*>(smem_raw + sizeof(Smem));
  uint16_t* lo = hi + kTile * hs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  const int item = blockIdx.x / cluster, block = blockIdx.x % cluster;
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const Item it = own_item(a, item, copy_none, reinterpret_cast<int*>(lo + kTile * hs), sm);
  if (it.rows == 0) return;
  const int rank = it.rank;
  const int units = (a.N + 31) / 32;
  const int n0 = (int)((int64_t)units * block / cluster), n1 = (int)((int64_t)units * (block + 1) / cluster);
  if (rank == 0) {                                         // no adapter: base as it is
    if (!copy_none) return;
    for (int r = warp; r < it.rows; r += kThreads / 32) {
      const int64_t m = sm.rows[r];
      for (int c = n0 * 32 + lane * 4; c < min(n1 * 32, a.N); c += 128)
        store4<kVec>(a.out + m * a.ldo, c, a.N,
                     a.base != nullptr ? load4<kVec>(a.base + m * a.ldb, c, a.N) : make_float4(0, 0, 0, 0));
    }
    return;
  }
  const int64_t m0 = g < it.rows ? sm.rows[g] : -1, m1 = g + 8 < it.rows ? sm.rows[g + 8] : -1;   // this lane's rows
  const __nv_bfloat16* x0 = m0 >= 0 ? a.X + m0 * a.ldx : nullptr;
  const __nv_bfloat16* x1 = m1 >= 0 ? a.X + m1 * a.ldx : nullptr;
  const __nv_bfloat16* A = a.A + it.adapter * a.a_slot;
  const __nv_bfloat16* B = a.B + it.adapter * a.b_slot;
  const int chunks = (a.K + 31) / 32;
  constexpr int kWarps = kThreads / 32;
  const uint32_t part_addr = umma::smem_u32(sm.part);
  auto all = [&](auto outer) {
    // The warps share K, and the ranks by 64 where there are more.  Sums lie by share
    // of K, row, rank.
    const int groups = rank <= 64 ? 1 : rank <= 128 ? 2 : 4, shares = kWarps / groups, pitch = groups * 64 + 4;
    const int share = block * shares + warp / groups, j0 = warp % groups * 64, left = rank - j0;
    const int c0 = (int)((int64_t)chunks * share / (cluster * shares));
    const int c1 = (int)((int64_t)chunks * (share + 1) / (cluster * shares));
    float acc[8][4] = {};
    if (left <= 0) {
    } else if (left <= 16) inner_part<2, 4>(a, x0, x1, A, rank, j0, c0, c1, acc);
    else if (left <= 32) inner_part<4, 3>(a, x0, x1, A, rank, j0, c0, c1, acc);
    else inner_part<8, 2>(a, x0, x1, A, rank, j0, c0, c1, acc);
    float* mine = sm.part + (warp / groups * 16 + g) * pitch + j0 + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      *reinterpret_cast<float2*>(mine + 8 * n) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + 8 * pitch + 8 * n) = make_float2(acc[n][2], acc[n][3]);
    }
    outer.start();
    __syncthreads();
    // the block's sums, in place of its first share's: four ranks of a row at a time
    for (int i = tid; i < groups * 256; i += kThreads) {
      float* at = sm.part + i / (groups * 16) * pitch + i % (groups * 16) * 4;
      float4 s = *reinterpret_cast<const float4*>(at);
      for (int k = 1; k < shares; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(at + k * 16 * pitch);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      *reinterpret_cast<float4*>(at) = s;
    }
    cluster_arrive();
    cluster_wait();
    for (int i = tid; i < groups * 256; i += kThreads) {
      const int r = i / (groups * 16), j = i % (groups * 16) * 4;
      if (j >= rs) continue;
      float4 s = cluster_sum(part_addr + (uint32_t)((r * pitch + j) * 4), cluster);
      s.x = j < rank ? s.x * it.scale : 0.f;
      s.y = j + 1 < rank ? s.y * it.scale : 0.f;
      s.z = j + 2 < rank ? s.z * it.scale : 0.f;
      s.w = j + 3 < rank ? s.w * it.scale : 0.f;
      put_terms(hi + r * hs + j, lo + r * hs + j, s);
    }
    __syncwarp();
    cluster_arrive();
    __syncthreads();
    outer.finish(hi, lo, hs);
  };
  if (rank <= 32) all(Outer<kVec, 1>{a, B, rank, m0, m1, n0 + warp, n1, kWarps});
  else if (rank <= 64) all(Outer<kVec, 2>{a, B, rank, m0, m1, n0 + warp, n1, kWarps});
  else all(Outer<kVec, 0>{a, B, rank, m0, m1, n0 + warp, n1, kWarps});
  __syncwarp();
  cluster_wait();                                          // no block leaves while another reads its sums
}

template <bool kVec>
cudaError_t launch_rows(const LoraArgs& a, int items, bool copy_none, cudaStream_t stream) {
  const int rs = (a.max_rank + 31) / 32 * 32;
  auto bytes = [](int stride, int adapters) {
    return sizeof(Smem) + (size_t)2 * kTile * (stride + 8) * 2 + (size_t)table_size(adapters) * 4;
  };
  const size_t most = bytes((int)kLoraMaxRank, (int)kLoraMaxAdapters);
  static std::atomic<uint64_t> done{0};
  cudaError_t err = set_once(done, reinterpret_cast<const void*>(lora_rows_kernel<kVec>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes(rs, a.n_adapters);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Blocks of an item: the more the better, as long as all items' are on the GPU at
  // once (64 rows over 40 adapters at K = N = 4096: 4 blocks 17.4 us, 6 16.0, 8, which do
  // not all fit, 21.7).  How many clusters of a size fit goes by how they pack into
  // the GPU's parts: asked once per device and size, for the largest rank.
  static std::atomic<int> fit[64][kMaxCluster + 1];
  int dev = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  int cluster = kMaxCluster;
  for (; cluster > 1; --cluster) {
    std::atomic<int>& known = fit[dev & 63][cluster];
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
      attr[0].val.clusterDim.x = cluster;
      cfg.gridDim = dim3((unsigned)cluster);
      cfg.numAttrs = 1;
      cfg.dynamicSmemBytes = most;
      if ((err = cudaOccupancyMaxActiveClusters(&n, lora_rows_kernel<kVec>, &cfg)) != cudaSuccess) return err;
      known.store(n, std::memory_order_relaxed);
      cfg.dynamicSmemBytes = bytes(rs, a.n_adapters);
    }
    if (items <= n) break;
  }
  attr[0].val.clusterDim.x = cluster;
  cfg.gridDim = dim3((unsigned)(items * cluster));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora_rows_kernel<kVec>, a, rs, cluster, copy_none);
}

// No call of up to this many rows is routed.
constexpr int kNoWorkspace = 256;

// Calls of few rows go without a routing launch and sums in memory, at the cost of
// reading an adapter's matrices once per 16 rows instead of once per 128, mostly from
// L2, and of mma.sync.  So the limit is one of the bytes read again, and a higher one
// where adapters have few rows each, which leave tiles of 128 nearly empty.  Not routed
// and routed: 512 rows over 40 adapters at K = N = 4096 and ranks up to 64 20 and 41 us, up
// to 128 32 and 47, up to 256 (134 MB) 52 and 60; 1500 rows, ranks up to 64 (98 MB) 34 and
// 49; 1500 rows over 5 at K = 1024, N = 2048 and rank 16 17 and 22.  The other way, few
// adapters: 1500 prompt rows at 4608, ranks up to 64 (111 MB) 35 and 33, 380 rows at 4096, up
// to 256 (100 MB) 36 and 32, 1500 at K = 8192, N = 12288, up to 64 (246 MB) 74 and 56.
bool own_rows(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank) {
  if (M <= kNoWorkspace) return true;
  if (M > kOwnRows) return false;
  const int64_t again = M / kTile * std::max<int64_t>(max_rank, 16) * (K + N) * 2;
  return again <= (M <= 48 * n_adapters ? 140 : 96) * (int64_t)1000000;
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank) {
  (void)K, (void)N;
  if (M <= kNoWorkspace) return 0;   // from there on asked for either way: own_rows' limits are a matter of speed
  return 256 + pad256((size_t)lora_max_tiles(M, n_adapters) * sizeof(int4)) + pad256((size_t)M * 4) +
         pad256((size_t)M * 2 * lora_rank_stride(max_rank) * 2);
}

cudaError_t launch_lora_add(const LoraArgs& a, void* workspace, cudaStream_t stream) {
  const bool copy_none = a.base != a.out;
  if (own_rows(a.M, a.K, a.N, a.n_adapters, a.max_rank)) {
    // d adapters in use make d + (M - d) / 16 items at most
    const int d = (int)std::min<int64_t>(a.n_adapters + 1, a.M), items = d + (a.M - d) / kTile;
    const bool vec = a.N % 4 == 0 && aligned(a.out, 16) && a.ldo % 4 == 0 &&
                     (a.base == nullptr || (aligned(a.base, 16) && a.ldb % 4 == 0));
    return vec ? launch_rows<true>(a, items, copy_none, stream) : launch_rows<false>(a, items, copy_none, stream);
  }
  uint8_t* p = static_cast<uint8_t*>(workspace);
  LoraWork w;
  w.head = reinterpret_cast<int*>(p);
  p += 256;
  w.tiles = reinterpret_cast<int4*>(p);
  p += pad256((size_t)lora_max_tiles(a.M, a.n_adapters) * sizeof(int4));
  w.rows = reinterpret_cast<int*>(p);
  p += pad256((size_t)a.M * 4);
  w.h = reinterpret_cast<uint16_t*>(p);
  // counting tables of as many warps as shared memory holds
  static std::atomic<uint64_t> done{0};
  constexpr int kRouteSmem = 200 * 1024;
  cudaError_t err = set_once(done, reinterpret_cast<const void*>(lora_route_kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem);
  if (err != cudaSuccess) return err;
  const int buckets = a.n_adapters + 1, segs = std::min(32, kRouteSmem / 4 / buckets - 3);
  if ((err = launch_pdl(lora_route_kernel, dim3(1), dim3(kRouteThreads), (size_t)(segs + 3) * buckets * 4, stream, a,
                        w, copy_none, segs)) != cudaSuccess)
    return err;
  return launch_lora_products(a, w, copy_none, stream);
}

}  // namespace qmm

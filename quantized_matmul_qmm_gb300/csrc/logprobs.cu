// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits.  With t_j = scale * (x_j - m), m the row's largest logit:
//     S = sum_j exp(t_j) = N + R   (N: how many logits equal m, R: the others)
//     log p_i = t_i - log S,   H = log S - (sum_j t_j exp(t_j)) / S
// N and R stay apart, so that log S = log N + log1p(R / N) keeps its relative
// accuracy where one token holds nearly all of a row.
//
// Bound: bytes, each logit read once, by a cluster of up to 16 blocks per row: one
// launch, no workspace.  A row is cut into segments of 128 16-byte vectors, dealt
// to the cluster's warps; a warp streams its segments with no barrier, the next
// one's loads under way, and leaves its statistics in the first block's shared memory.
//
// Measured against a copy's rate: 1024 rows of 151936 in fp32 with one alternative
// (623 MB) 98 us, 0.95; 512 rows in bf16 43 us, 0.54: two rounds of the 304 blocks that the
// GPU holds (304 rows take 24 us, 608 44), in which 13 to 14 instructions a logit, as many
// as in fp32, keep 72 % of the issue slots busy.  Few rows wait for one another's steps: 64
// rows 12 us, with five alternatives 15.7 (5.8 at that rate); a row with 20 of them 8.9.
//
// Alternatives cost the stream the maxima of pieces, four to a segment: the k-th
// largest of 64 groups' maxima (of threads' logits, or of segments in a cluster) is a
// value that at least k logits reach, so that only the pieces that reach it (about
// 1.3 k) are read again.  Logits are kept by a 64-bit key, their value in an
// order-preserving integer form and the complement of their index, so that keys
// differ, equal logits fall by rising index and the choice is exact whatever the
// order of work.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

#include "beside.h"
#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kAhead = 4;             // vectors of a segment per lane, each of another piece
constexpr int kSegVecs = 32 * kAhead; // vectors of a segment (of one of its steps in rows of more than Block::kSegs)
constexpr int kMaxCluster = 16;
constexpr int kUnit = 256;            // elements that a warp reads again at a time

// The two blocks: of long rows, alone or in a cluster, and of short ones.
template <bool kLong, bool kTop>
struct Block {
  static constexpr int kThreads = kLong ? 512 : 128, kWarps = kThreads / 32, kPerSm = kLong ? 2 : 8;
  static constexpr int kSegs = 512, kPieces = kTop ? kSegs * kAhead : 4;
  static constexpr int kCluster = kLong ? kMaxCluster : 1;
  static constexpr int kPool = kTop ? kWarps * kUnit : 1;   // candidates of one step of reading again
  static constexpr int kKeep = kTop ? kThreads : 1;         // candidates that may wait for the next step
};
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Statistics relative to the maximum m: n terms equal to it, r the sum of the
// others' 2^t, w the sum of t 2^t (t in the log2 domain).
struct Stats {
  float m, n, r, w;
};

QMM_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two parts of a row.  m is at least -FLT_MAX, so that differences are defined.
QMM_DEV Stats join(const Stats& a, const Stats& b, float c) {
  const bool up = b.m > a.m;
  const Stats hi = up ? b : a, lo = up ? a : b;
  if (hi.m == lo.m) return Stats{hi.m, hi.n + lo.n, hi.r + lo.r, hi.w + lo.w};
  const float t = fmaxf((lo.m - hi.m) * c, -1e30f), f = exp2_fast(t), s = lo.n + lo.r;
  // sum of (t + t_j) 2^(t + t_j) = 2^t (t s + w_lo)
  return Stats{hi.m, hi.n, fmaf(s, f, hi.r), hi.w + (f > 0.f ? f * fmaf(t, s, lo.w) : 0.f)};
}

// The same statistics relative to a larger m.
QMM_DEV Stats raise_to(const Stats& a, float m, float c) {
  const float t = fmaxf((a.m - m) * c, -1e30f), f = exp2_fast(t), s = a.n + a.r;
  return Stats{m, 0.f, s * f, f > 0.f ? f * fmaf(t, s, a.w) : 0.f};
}

QMM_DEV void put_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// A barrier of all blocks of a row.
QMM_DEV void block_sync(int cluster) {
  if (cluster > 1) umma::cluster_sync();
  else __syncthreads();
}

QMM_DEV uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 becomes 0
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
QMM_DEV float value_of(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }
QMM_DEV uint64_t key_of(float x, uint32_t index) { return (uint64_t)order_of(x) << 32 | (0xFFFFFFFFu - index); }
constexpr uint32_t kOrderMinusInf = 0x007FFFFFu;   // order_of(-inf): not an alternative

template <bool kBf16>
struct Vec {
  static constexpr int kN = kBf16 ? 8 : 4;
  uint4 q;
  QMM_DEV float at(int i) const {
    if constexpr (kBf16) {
      const uint32_t w = u4_get(q, i / 2);
      return i & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
    } else {
      return __uint_as_float(u4_get(q, i));
    }
  }
};

// A row as 16-byte vectors: `head` elements before the first boundary, `full`
// vectors, and what remains.  Elements outside the vectors (at most 14) are the edge,
// one per lane.
template <bool kBf16>
struct Row {
  const uint8_t* x;
  const uint8_t* vecs;
  int head, full, V;
  QMM_DEV Row(const uint8_t* row, int n) : x(row), V(n) {
    constexpr int kN = Vec<kBf16>::kN, kSize = kBf16 ? 2 : 4;
    head = min((int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / kSize, V);
    full = (V - head) / kN;
    vecs = row + head * kSize;
  }
  QMM_DEV float at(int i) const {
    if constexpr (kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[i]);
    return reinterpret_cast<const float*>(x)[i];
  }
  // Vector v, or -infinity where there is none.
  QMM_DEV Vec<kBf16> vec(int v) const {
    const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    Vec<kBf16> r;
    r.q = make_uint4(none, none, none, none);
    if (v < full) r.q = ldg128_stream(vecs + (int64_t)v * 16);
    return r;
  }
  // Lane's edge element, or -1.
  QMM_DEV int edge(int lane) const {
    const int behind = head + full * Vec<kBf16>::kN + lane - head;
    return lane < head ? lane : behind < V ? behind : -1;
  }
};

template <typename B>
struct alignas(16) Shared {
  Stats stats[B::kCluster * B::kWarps];   // of the cluster's warps
  uint32_t piece_max[B::kPieces + 4];     // order of a piece's largest logit; the edge's behind them
  uint64_t pool[B::kPool + B::kKeep];     // candidates
  uint64_t best[kMaxTop];                 // the largest so far, falling
  uint64_t warp_key[B::kCluster * B::kWarps];
  uint32_t group_max[B::kWarps][32];
  uint16_t list[B::kPieces + 1];          // pieces to read again, rising
  int warp_count[B::kWarps];
  Stats row;
  int n_pool;
  uint32_t floor_order;
};

// The k largest of the pool's n keys, falling, into sm.best; returns how many.
// Many candidates (rows with far more than k equal logits) are thinned first.
template <typename B>
QMM_DEV int settle(Shared<B>& sm, int n, int k) {
  constexpr int kThreads = B::kThreads, kWarps = B::kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (n > kThreads) {
    // Raise a bar until k to 2 k threads' largest keys lie above it, by bisection
    // over the keys, which differ, so that it ends: at most 2 k threads' keys stay.
    constexpr int kEach = (B::kPool + B::kKeep) / kThreads;
    uint64_t mine[kEach], most = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      mine[i] = tid + i * kThreads < n ? sm.pool[tid + i * kThreads] : 0;
      most = max(most, mine[i]);
    }
    uint64_t above = most;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) above = max(above, __shfl_xor_sync(0xffffffffu, above, o));
    if (lane == 0) sm.warp_key[warp] = above;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) above = max(above, sm.warp_key[w]);   // nothing lies above it
    uint64_t bar = 0;
    int count = kThreads;
    while (count > 2 * k) {
      const uint64_t mid = bar + (above - bar) / 2;
      const int c = __syncthreads_count(most > mid);
      if (c >= k) bar = mid, count = c;
      else above = mid;
    }
    if (tid == 0) sm.n_pool = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (mine[i] > bar) sm.pool[atomicAdd(&sm.n_pool, 1)] = mine[i];
    __syncthreads();
    n = sm.n_pool;
  }
  // a key's place is the number of larger ones
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t mine = sm.pool[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += sm.pool[j] > mine;
    if (place < k) sm.best[place] = mine;
  }
  __syncthreads();
  return min(n, k);
}

// The k largest logits of a row into sm.best, by the whole block; returns how
// many there are (logits of -infinity are none).  lane_top: the largest of those that
// this thread has seen, in rows of one block.
template <bool kBf16, typename B>
QMM_DEV int find_top(Shared<B>& sm, const Row<kBf16>& x, int k, int segs, int steps, int cluster, float lane_top) {
  constexpr int kThreads = B::kThreads, kWarps = B::kWarps;
  constexpr int kN = Vec<kBf16>::kN, kLoads = kUnit / kN / 32;   // pieces' steps that a warp reads at a time
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the k-th largest of 64 groups' maxima: groups of threads, or of segments
  const int pieces = segs * kAhead, all = pieces + 1;   // with the edge
  uint32_t most = order_of(lane_top);
  if (cluster > 1) {
    most = 0;
    for (int i = tid; i < segs; i += kThreads) {
      const uint4 v = *reinterpret_cast<const uint4*>(sm.piece_max + i * kAhead);
      most = max(most, max(max(v.x, v.y), max(v.z, v.w)));
    }
  }
  sm.group_max[warp][lane] = most;
  __syncthreads();
  if (warp == 0) {                        // by one warp: by all of them it took longer
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w += 2) {
      even = max(even, sm.group_max[w][lane]);
      odd = max(odd, sm.group_max[w + 1][lane]);
    }
    int even_place = 0, odd_place = 0;    // how many come before; of equals, the even warps' first
#pragma unroll
    for (int l = 0; l < 32; ++l) {
      const uint32_t e = __shfl_sync(0xffffffffu, even, l), o = __shfl_sync(0xffffffffu, odd, l);
      even_place += (e > even || (e == even && l < lane)) + (o > even);
      odd_place += (e >= odd) + (o > odd || (o == odd && l < lane));
    }
    const uint32_t kth = even_place == k - 1 ? even : odd_place == k - 1 ? odd : 0u;
    const uint32_t order = __reduce_max_sync(0xffffffffu, kth);
    if (lane == 0) sm.floor_order = max(order, kOrderMinusInf + 1), sm.n_pool = 0;
  }
  __syncthreads();
  const uint32_t floor_order = sm.floor_order;
  // the pieces that reach it
  const int each = (all + kThreads - 1) / kThreads;
  int mine = 0;
  for (int i = tid * each; i < min((tid + 1) * each, all); ++i) mine += sm.piece_max[i] >= floor_order;
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) sm.warp_count[warp] = at;
  __syncthreads();
  at -= mine;
  int listed = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += sm.warp_count[w];
    listed += sm.warp_count[w];
  }
  for (int i = tid * each; i < min((tid + 1) * each, all); ++i)
    if (sm.piece_max[i] >= floor_order) sm.list[at++] = (uint16_t)i;
  __syncthreads();
  // read again, kLoads steps of pieces per warp at a time
  const int units = listed * steps;
  uint64_t bar = (uint64_t)(floor_order - 1) << 32 | 0xFFFFFFFFu;   // keys above it are candidates
  uint32_t skip = floor_order - 1;        // pieces that do not come above it hold no candidate
  int bar_seg = -1;                       // of several steps: the segment that the bar lies in
  int have = 0;                           // of sm.best
  Vec<kBf16> next[kLoads];
  int next_at[kLoads];                    // index of the lane's first element
  auto load = [&](int unit0) {
    if (steps > 1 && unit0 < units && sm.list[unit0 / steps] / kAhead > bar_seg) skip = (uint32_t)(bar >> 32);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int unit = unit0 + u, i = steps == 1 ? unit : unit / steps, step = unit - i * steps;
      const int piece = unit < units ? sm.list[i] : -1;
      const bool none = piece < 0 || piece == pieces || sm.piece_max[piece] <= skip;
      const int v = none ? x.full : (piece / kAhead * steps + step) * kSegVecs + piece % kAhead * 32 + lane;
      next_at[u] = x.head + v * kN;
      next[u] = x.vec(v);
      if (piece == pieces && step == 0 && x.edge(lane) >= 0) {
        next_at[u] = x.edge(lane);
        const uint32_t w = __float_as_uint(x.at(next_at[u]));
        next[u].q.x = kBf16 ? w >> 16 | 0xFF800000u : w;
      }
    }
  };
  load(warp * kLoads);
  for (int u0 = 0; u0 < units; u0 += kWarps * kLoads) {
    Vec<kBf16> q[kLoads];
    int at0[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) q[u] = next[u], at0[u] = next_at[u];
    load(u0 + (kWarps + warp) * kLoads);
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float f = q[u].at(i);
        const uint64_t key = key_of(f, (uint32_t)(at0[u] + i));
        if (f == f && key > bar) sm.pool[atomicAdd(&sm.n_pool, 1)] = key;   // not NaN
      }
    __syncthreads();
    const int n = sm.n_pool;
    if (u0 + kWarps * kLoads >= units) return settle(sm, n, k);
    __syncthreads();
    if (n > B::kKeep) {
      // the pool has room for one more step beside these
      have = settle(sm, n, k);
      if (tid < have) sm.pool[tid] = sm.best[tid];
      if (tid == 0) sm.n_pool = have;
      if (have == k) {
        // A piece that equals the bar has larger indexes and is skipped, but for the edge,
        // which comes last in the list, and for the bar's own segment where it has several
        // steps: a later piece's first step lies before an earlier one's second.
        bar = sm.best[k - 1];
        skip = (uint32_t)(bar >> 32) - (steps > 1);
        bar_seg = (int)((0xFFFFFFFFu - (uint32_t)bar - x.head) / ((uint32_t)steps * kSegVecs * kN));
      }
      __syncthreads();
    }
  }
  return 0;
}

template <bool kBf16, bool kLong, bool kTop>
__global__ void __launch_bounds__(Block<kLong, kTop>::kThreads, Block<kLong, kTop>::kPerSm)
token_logprobs_kernel(LogprobArgs a, int cluster, int segs, int steps) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using B = Block<kLong, kTop>;
  Shared<B>& sm = *reinterpret_cast<Shared<B>*>(smem_raw);
  constexpr int kN = Vec<kBf16>::kN, kThreads = B::kThreads, kWarps = B::kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const Row<kBf16> x(static_cast<const uint8_t*>(a.logits) + (int64_t)row * a.ld * (kBf16 ? 2 : 4), a.V);
  const float c = a.scale * kLog2e;
  const int k = a.top_k;

  // This warp's segments, in steps of 32 lanes by kAhead vectors.
  const int wid = rank * kWarps + warp, warps = cluster * kWarps;
  Vec<kBf16> next[kAhead];
  auto load = [&](int seg, int step) {
    const int v0 = seg < segs ? (seg * steps + step) * kSegVecs + lane : x.full;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = x.vec(v0 + u * 32);
  };
  load(wid, 0);
  // the tokens' logits, long before they are needed
  int token = -1;
  float token_x = 0.f;
  if (rank == 0 && tid < a.G) {
    token = a.tokens[(int64_t)row * a.ld_tokens + tid];
    if (token >= 0 && token < a.V) token_x = x.at(token);
  }
  // the edge, by the last warp: it has the fewest segments
  float edge_x = -INFINITY;
  const bool edge_warp = wid == warps - 1;
  if (edge_warp && x.edge(lane) >= 0) edge_x = x.at(x.edge(lane));
  block_sync(cluster);   // every block of the cluster runs, so that the first one's shared memory can be written
  const uint32_t first_stats = umma::mapa_shared(umma::smem_u32(&sm.stats[wid]), 0);
  const uint32_t first_pieces = umma::mapa_shared(umma::smem_u32(sm.piece_max), 0);

  Stats st = {-FLT_MAX, 0.f, 0.f, 0.f};   // m is the warp's, n, r and w the lane's
  uint64_t key = 0;                        // of the warp's largest logit, where one alternative is asked for
  float lane_top = edge_x;                 // the lane's largest
  for (int seg = wid; seg < segs; seg += warps) {
    uint32_t piece_order[kAhead] = {};
    for (int step = 0; step < steps; ++step) {
      Vec<kBf16> q[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) q[u] = next[u];
      if (step + 1 < steps) load(seg, step + 1);
      else load(seg + warps, 0);
      uint32_t order = 0;
      float top = -INFINITY;
      if constexpr (kTop) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          float most = -INFINITY;
#pragma unroll
          for (int i = 0; i < kN; ++i) most = fmaxf(most, q[u].at(i));
          top = fmaxf(top, most);
          const uint32_t o = __reduce_max_sync(0xffffffffu, order_of(most));
          piece_order[u] = max(piece_order[u], o), order = max(order, o);
        }
        lane_top = fmaxf(lane_top, top);
      } else {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < kN; ++i) top = fmaxf(top, q[u].at(i));
        order = __reduce_max_sync(0xffffffffu, order_of(top));
      }
      const float m = value_of(order);
      if (m >= st.m) {
        // a new maximum (or the same again): its own terms are counted apart
        if (!kTop && k == 1 && (m > st.m || key == 0)) {
          uint32_t at = 0xFFFFFFFFu;
          const uint32_t first = x.head + ((seg * steps + step) * kSegVecs + lane) * kN;
#pragma unroll
          for (int u = kAhead - 1; u >= 0; --u)
#pragma unroll
            for (int i = kN - 1; i >= 0; --i)
              if (q[u].at(i) == m) at = first + u * 32 * kN + i;
          key = (uint64_t)order << 32 | (0xFFFFFFFFu - __reduce_min_sync(0xffffffffu, at));
        }
        if (m > st.m) st = raise_to(st, m, c);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float t = (q[u].at(i) - st.m) * c, e = exp2_fast(t);
            if (t < 0.f) st.r += e;
            else st.n += e;                              // 1, or NaN
            st.w = fmaf(fmaxf(t, -1e30f), e, st.w);       // -infinity: -1e30 * 0
          }
      } else {
        const uint64_t minus_m = f2_pack(-st.m, -st.m), cc = f2_pack(c, c);
        uint64_t r2 = f2_pack(st.r, 0.f), w2 = f2_pack(st.w, 0.f);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int i = 0; i < kN; i += 2) {
            const uint64_t t2 = f2_mul(f2_add(f2_pack(q[u].at(i), q[u].at(i + 1)), minus_m), cc);
            float t0, t1;
            f2_unpack(t2, t0, t1);
            const uint64_t e2 = f2_pack(exp2_fast(t0), exp2_fast(t1));
            r2 = f2_add(r2, e2);
            w2 = f2_fma(f2_pack(fmaxf(t0, -1e30f), fmaxf(t1, -1e30f)), e2, w2);
          }
        float lo, hi;
        f2_unpack(r2, lo, hi);
        st.r = lo + hi;
        f2_unpack(w2, lo, hi);
        st.w = lo + hi;
      }
    }
    if (kTop && lane == 0)
      asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(first_pieces + 16u * seg),
                   "r"(piece_order[0]), "r"(piece_order[1]), "r"(piece_order[2]), "r"(piece_order[3])
                   : "memory");
  }
  if (edge_warp) {
    const uint32_t order = __reduce_max_sync(0xffffffffu, order_of(fmaxf(edge_x, -INFINITY)));   // NaN: -infinity
    if (kTop && lane == 0) put_u32(first_pieces + 16u * segs, order);
    const float m = value_of(order);
    if (!kTop && k == 1 && order > kOrderMinusInf) {
      const uint32_t at = edge_x == m ? (uint32_t)x.edge(lane) : 0xFFFFFFFFu;
      key = max(key, (uint64_t)order << 32 | (0xFFFFFFFFu - __reduce_min_sync(0xffffffffu, at)));
    }
    if (m > st.m) st = raise_to(st, m, c);
    const float t = (edge_x - st.m) * c, e = exp2_fast(t);
    if (t < 0.f) st.r += e;
    else st.n += e;
    st.w = fmaf(fmaxf(t, -1e30f), e, st.w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.n += __shfl_xor_sync(0xffffffffu, st.n, o);
    st.r += __shfl_xor_sync(0xffffffffu, st.r, o);
    st.w += __shfl_xor_sync(0xffffffffu, st.w, o);
  }
  if (lane == 0)
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(first_stats), "f"(st.m), "f"(st.n), "f"(st.r),
                 "f"(st.w)
                 : "memory");
  if (!kTop && lane == 0 && k == 1)
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(umma::mapa_shared(umma::smem_u32(&sm.warp_key[wid]), 0)),
                 "l"(key)
                 : "memory");
  block_sync(cluster);
  if (rank != 0) return;

  if (warp == 0) {
    st = lane < warps ? sm.stats[lane] : Stats{-FLT_MAX, 0.f, 0.f, 0.f};
    for (int i = lane + 32; i < warps; i += 32) st = join(st, sm.stats[i], c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stats b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.n, o),
                       __shfl_xor_sync(0xffffffffu, st.r, o), __shfl_xor_sync(0xffffffffu, st.w, o)};
      st = join(st, b, c);
    }
    if (lane == 0) sm.row = st;
    if (!kTop && k == 1) {
      key = 0;
      for (int i = lane; i < warps; i += 32) key = max(key, sm.warp_key[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
      if (lane == 0) sm.best[0] = key;
    }
  }
  __syncthreads();
  st = sm.row;
  const float total = st.n + st.r;
  const bool sound = total > 0.f && st.m < INFINITY;   // false for NaN as well
  const float log_sum = logf(st.n) + log1pf(st.r / st.n);
  if (tid == 0 && a.entropy != nullptr) a.entropy[row] = sound ? fmaf(-st.w / total, kLn2, log_sum) : NAN;
  for (int g = tid; g < a.G; g += kThreads) {
    if (g >= kThreads) {
      token = a.tokens[(int64_t)row * a.ld_tokens + g];
      if (token >= 0 && token < a.V) token_x = x.at(token);
    }
    if (token < 0 || token >= a.V) {
      if (token != -1) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      if (a.write_other) a.logprobs[(int64_t)row * a.G + g] = a.other;
      continue;
    }
    a.logprobs[(int64_t)row * a.G + g] = sound ? (token_x - st.m) * a.scale - log_sum : NAN;
  }
  if (k == 0) return;
  int have = sound ? 1 : 0;
  if constexpr (kTop) have = sound ? find_top(sm, x, k, segs, steps, cluster, lane_top) : 0;
  if (tid < k) {
    int32_t id = -1;
    float l = sound ? -INFINITY : NAN;
    if (tid < have) {
      const uint64_t key = sm.best[tid];
      id = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
      l = (value_of((uint32_t)(key >> 32)) - st.m) * a.scale - log_sum;
    }
    a.top_ids[(int64_t)row * k + tid] = id;
    a.top_logprobs[(int64_t)row * k + tid] = l;
  }
}

template <bool kBf16, bool kLong, bool kTop>
cudaError_t launch_typed(const LogprobArgs& a, int cluster, int segs, int steps, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0}, done_size{0};
  constexpr auto kern_typed = token_logprobs_kernel<kBf16, kLong, kTop>;
  const void* kern = reinterpret_cast<const void*>(kern_typed);
  cudaError_t err = set_once(done, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  if ((err = set_once(done_size, kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                      (int)sizeof(Shared<Block<kLong, kTop>>))) != cudaSuccess)
    return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.M * cluster);
  cfg.blockDim = dim3(Block<kLong, kTop>::kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared<Block<kLong, kTop>>);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern_typed, a, cluster, segs, steps);
}

template <bool kLong>
cudaError_t launch_block(const LogprobArgs& a, int cluster, int segs, int steps, cudaStream_t stream) {
  if (a.top_k > 1)
    return a.bf16 ? launch_typed<true, kLong, true>(a, cluster, segs, steps, stream)
                  : launch_typed<false, kLong, true>(a, cluster, segs, steps, stream);
  return a.bf16 ? launch_typed<true, kLong, false>(a, cluster, segs, steps, stream)
                : launch_typed<false, kLong, false>(a, cluster, segs, steps, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  const int64_t vecs = a.V / (a.bf16 ? 8 : 4);   // a row's, wherever it begins: no more than this
  const int64_t least = std::max<int64_t>(1, (vecs + kSegVecs - 1) / kSegVecs);
  using Long = Block<true, true>;
  using Short = Block<false, true>;
  static_assert(Long::kSegs == Short::kSegs, "one way to cut rows");
  const int steps = (int)((least + Long::kSegs - 1) / Long::kSegs);
  const int segs = (int)((least + steps - 1) / steps);
  // Short blocks, eight to an SM, where a row gives no more than their warps work, or
  // where there are more rows than the long ones take at once: many rows then stand at
  // different steps, and the alternatives' latency is spread over them.  Long and short
  // blocks, fp32 without padding: 1000 rows of 8000, one alternative 17.3 and 10.4 us, 20 of
  // them 34.6 and 18.7; 2000 rows of 100000 131 and 129, 171 and 149; 400 rows of 8000 9.0
  // and 7.0, 16.7 and 13.7, of 32000 14.9 and 16.7, 22.9 and 24.0; but 512 rows of 151936, which
  // leave an SM four of them, 54.5 and 87.4.
  const int64_t at_once = (int64_t)Long::kPerSm * attn_sm_count();
  if (segs <= Short::kWarps || (a.M > at_once && segs <= 32) || a.M > 3 * at_once)
    return launch_block<false>(a, 1, segs, steps, stream);
  // Blocks of a row: as many as fit on the GPU at once (two per SM) when there are
  // few rows, while each warp keeps a segment.
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)a.M * 2 * cluster <= at_once &&
         segs >= 2 * cluster * Long::kWarps)
    cluster *= 2;
  return launch_block<true>(a, cluster, segs, steps, stream);
}

}  // namespace qmm

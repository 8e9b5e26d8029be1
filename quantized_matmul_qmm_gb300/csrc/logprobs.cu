// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits.  With t_j = scale * (x_j - m), m the row's largest logit:
//     S = sum_j exp(t_j) = N + R   (N: how many logits equal m, R: the others)
//     log p_i = t_i - log S,   H = log S - (sum_j t_j exp(t_j)) / S
// N and R stay apart, so that log S = log N + log1p(R / N) keeps its relative
// accuracy where one token holds nearly all of a row.
//
// Bound: bytes, each logit read once.  A cluster of up to 16 blocks takes a
// row; a block's tile of it lies in registers while the tile's maximum, sums and
// candidates for the alternatives are found, and what the blocks found meets in
// the first block's shared memory: one launch, no workspace.
//
// Alternatives are kept by a 64-bit key: the logit in an order-preserving
// integer form, then the complement of its index, so that keys differ, equal
// logits fall by rising index and the choice is exact whatever the order of work.
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "beside.h"
#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 8;          // 16-byte vectors of a tile per thread
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Running statistics relative to the maximum m: n terms equal to it, r the sum
// of the others' 2^t, w the sum of t 2^t (t in the log2 domain).
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

template <bool kBf16>
QMM_DEV float load_one(const void* row, int64_t i) {
  if constexpr (kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[i]);
  return static_cast<const float*>(row)[i];
}

// Vector `v` of a row that begins `off` elements after a 16-byte boundary:
// elements v * kN - off ..; what lies outside the row reads as -infinity.
template <bool kBf16>
QMM_DEV Vec<kBf16> load_vec(const void* row, int off, int v, int V) {
  constexpr int kN = Vec<kBf16>::kN;
  const int64_t e = (int64_t)v * kN - off;
  Vec<kBf16> r;
  if (e >= 0 && e + kN <= V) {
    r.q = ldg128_stream(static_cast<const uint8_t*>(row) + e * (kBf16 ? 2 : 4));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = kBf16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (e + i < 0 || e + i >= V) continue;
      if constexpr (kBf16) {
        const uint32_t b = static_cast<const uint16_t*>(row)[e + i];
        w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | b << 16 : (w[i / 2] & 0xFFFF0000u) | b;
      } else {
        w[i] = static_cast<const uint32_t*>(row)[e + i];
      }
    }
    r.q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

// Block `rank` of the cluster's part of a result, as it lies in the first block.
struct alignas(16) Part {
  Stats s;
  uint32_t count;           // alternatives
  uint64_t best[kMaxTop];   // falling
};

struct Shared {
  Part parts[kMaxCluster];
  uint64_t best[2][kMaxTop];          // this block's alternatives, falling
  // Candidates of a tile: at most 2 k threads' elements (64 at most each)
  uint64_t pool[2 * kMaxTop * 64 + kMaxTop];
  Stats warp_stats[kWarps];
  uint64_t warp_max[kWarps];
  int n_pool;
};

// The k largest of pool[0..n), falling, into `to`: each key's rank is the
// number of larger ones (keys differ).
QMM_DEV void rank_into(const uint64_t* pool, int n, int k, uint64_t* to) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = pool[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += pool[j] > mine;
    if (rank < k) to[rank] = mine;
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
token_logprobs_kernel(LogprobArgs a, int cluster) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  constexpr int kN = Vec<kBf16>::kN;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const uint8_t* x = static_cast<const uint8_t*>(a.logits) + (int64_t)row * a.ld * (kBf16 ? 2 : 4);
  const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / (kBf16 ? 2 : 4));
  const int vecs = (int)(((int64_t)a.V + off + kN - 1) / kN);
  const int part = (vecs + cluster - 1) / cluster;
  const int begin = min(rank * part, vecs), end = min(begin + part, vecs);
  const float c = a.scale * kLog2e;
  const int k = a.top_k;

  Stats st = {-FLT_MAX, 0.f, 0.f, 0.f};
  int have = 0;              // alternatives so far, in sm.best[cur]
  int cur = 0;
  for (int base = begin; base < end; base += kUnroll * kThreads) {
    Vec<kBf16> q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = base + u * kThreads + tid;
      q[u] = load_vec<kBf16>(x, off, v < end ? v : vecs + 1, a.V);   // past the row: -infinity
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) top = fmaxf(top, q[u].at(i));
    const float m = fmaxf(st.m, top);
    Stats tile = {m, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float t = (q[u].at(i) - m) * c, e = exp2_fast(t);
        if (t < 0.f) tile.r += e;
        else tile.n += e;                            // 1, or NaN
        tile.w = fmaf(fmaxf(t, -1e30f), e, tile.w);   // -infinity: -1e30 * 0
      }
    st = join(tile, st, c);

    if (k == 0) continue;
    // Candidates: what exceeds the last of the block's alternatives.
    const uint64_t least = have == k ? sm.best[cur][k - 1] : (uint64_t)kOrderMinusInf << 32 | 0xFFFFFFFFu;
    const uint32_t top_order = order_of(top);
    uint64_t mine = 0;
    if (top_order >= (uint32_t)(least >> 32) && top_order > kOrderMinusInf) {
#pragma unroll
      for (int u = kUnroll - 1; u >= 0; --u)
#pragma unroll
        for (int i = kN - 1; i >= 0; --i)
          if (q[u].at(i) == top) mine = key_of(top, (uint32_t)((base + u * kThreads + tid) * kN - off + i));
    }
    uint64_t bar = least;                            // keys above it are candidates
    int n = __syncthreads_count(mine > bar);
    if (n == 0) continue;
    if (n > 2 * k) {
      // Raise the bar until k to 2 k threads' largest lie above it: bisection over
      // the keys, which differ, so that it ends.
      uint64_t best = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      if (lane == 0) sm.warp_max[warp] = best;
      __syncthreads();
      uint64_t above = 0;                            // nothing lies above it
#pragma unroll
      for (int w = 0; w < kWarps; ++w) above = max(above, sm.warp_max[w]);
      while (n > 2 * k) {
        const uint64_t mid = bar + (above - bar) / 2;
        const int nm = __syncthreads_count(mine > mid);
        if (nm >= k) bar = mid, n = nm;
        else above = mid;
      }
    }
    if (tid == 0) sm.n_pool = 0;
    __syncthreads();
    if (mine > bar) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint64_t key = key_of(q[u].at(i), (uint32_t)((base + u * kThreads + tid) * kN - off + i));
          if (q[u].at(i) <= top && key > bar) sm.pool[atomicAdd(&sm.n_pool, 1)] = key;   // not NaN
        }
    }
    if (tid < have) {
      // the block's alternatives so far compete as well
      const uint64_t key = sm.best[cur][tid];
      sm.pool[atomicAdd(&sm.n_pool, 1)] = key;
    }
    __syncthreads();
    const int pooled = sm.n_pool;
    rank_into(sm.pool, pooled, k, sm.best[cur ^ 1]);
    cur ^= 1;
    have = min(k, pooled);
    __syncthreads();
  }

  // The block's statistics: warps, then the first warp.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stats b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.n, o),
                     __shfl_xor_sync(0xffffffffu, st.r, o), __shfl_xor_sync(0xffffffffu, st.w, o)};
    st = join(st, b, c);
  }
  if (lane == 0) sm.warp_stats[warp] = st;
  umma::cluster_sync();   // also: every block of the cluster runs, and its shared memory can be written
  if (warp == 0) {
    st = lane < kWarps ? sm.warp_stats[lane] : Stats{-FLT_MAX, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stats b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.n, o),
                       __shfl_xor_sync(0xffffffffu, st.r, o), __shfl_xor_sync(0xffffffffu, st.w, o)};
      st = join(st, b, c);
    }
    const uint32_t to = umma::mapa_shared(umma::smem_u32(&sm.parts[rank]), 0);
    if (lane == 0) {
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to), "f"(st.m), "f"(st.n), "f"(st.r),
                   "f"(st.w)
                   : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + (uint32_t)offsetof(Part, count)), "r"(have)
                   : "memory");
    }
    if (lane < have)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + (uint32_t)offsetof(Part, best) + 8u * lane),
                   "l"(sm.best[cur][lane])
                   : "memory");
  }
  umma::cluster_sync();
  if (rank != 0) return;

  // The row's statistics, the same in every thread.
  st = sm.parts[0].s;
  for (int p = 1; p < cluster; ++p) st = join(st, sm.parts[p].s, c);
  const float total = st.n + st.r;
  const bool sound = total > 0.f && st.m < INFINITY;   // false for NaN as well
  const float log_sum = logf(st.n) + log1pf(st.r / st.n);
  if (tid == 0 && a.entropy != nullptr) a.entropy[row] = sound ? fmaf(-st.w / total, kLn2, log_sum) : NAN;
  for (int g = tid; g < a.G; g += kThreads) {
    const int token = a.tokens[(int64_t)row * a.ld_tokens + g];
    if (token < 0 || token >= a.V) {
      if (token != -1) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      continue;
    }
    const float l = (load_one<kBf16>(x, token) - st.m) * a.scale - log_sum;
    a.logprobs[(int64_t)row * a.G + g] = sound ? l : NAN;
  }
  if (k == 0) return;
  // A key's place among all is its place in its own list and, in each other
  // list, the number of larger keys.
  int all = 0;
  for (int p = 0; p < cluster; ++p) all += sm.parts[p].count;
  for (int i = tid; i < cluster * kMaxTop; i += kThreads) {
    const int p = i / kMaxTop, at = i % kMaxTop;
    if (at >= (int)sm.parts[p].count) continue;
    const uint64_t mine = sm.parts[p].best[at];
    int place = at;
    for (int o = 0; o < cluster && place < k; ++o) {
      if (o == p) continue;
      int lo = 0, hi = sm.parts[o].count;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sm.parts[o].best[mid] > mine) lo = mid + 1;
        else hi = mid;
      }
      place += lo;
    }
    if (place >= k || !sound) continue;
    a.top_ids[(int64_t)row * k + place] = (int32_t)(0xFFFFFFFFu - (uint32_t)mine);
    a.top_logprobs[(int64_t)row * k + place] = (value_of((uint32_t)(mine >> 32)) - st.m) * a.scale - log_sum;
  }
  for (int i = tid; i < k; i += kThreads) {
    if (sound && i < all) continue;
    a.top_ids[(int64_t)row * k + i] = -1;
    a.top_logprobs[(int64_t)row * k + i] = sound ? -INFINITY : NAN;
  }
}

template <bool kBf16>
cudaError_t launch_typed(const LogprobArgs& a, int cluster, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0}, done_size{0};
  const void* kern = reinterpret_cast<const void*>(token_logprobs_kernel<kBf16>);
  cudaError_t err = set_once(done, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  if ((err = set_once(done_size, kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared))) != cudaSuccess)
    return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.M * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<kBf16>, a, cluster);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  // Blocks of a row: enough to fill the SMs twice when there are few rows, while
  // each keeps at least half a tile.
  const int sms = attn_sm_count();
  const int vecs = (int)((a.V + (a.bf16 ? 7 : 3)) / (a.bf16 ? 8 : 4)) + 1;
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)a.M * cluster < 2 * sms && vecs / (2 * cluster) >= kUnroll * kThreads / 2)
    cluster *= 2;
  return a.bf16 ? launch_typed<true>(a, cluster, stream) : launch_typed<false>(a, cluster, stream);
}

}  // namespace qmm

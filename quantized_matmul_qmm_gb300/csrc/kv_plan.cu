// The plan of one step of a paged cache: from each request's cached length L
// and its number n of new tokens, the pages that the step takes, the new
// entries of the block table, the slot and the position of every new token,
// and for drafted trees the mask of each token's ancestors.
//
//   have = ceil(L / P), need = ceil((L + n) / P)      pages before and after
//   cu   = exclusive sum of n, base = exclusive sum of need - have
//   table[r][c] = free[base[r] + c - have[r]]         for have <= c < need
//   token i of r: p = L + i, slot = table[r][p / P] * P + p % P
//
// Every block sums all requests again in its own shared memory (a few KB that
// sit in L2), so that one launch does everything and no block waits for
// another; then each thread takes tokens and finds its request by bisection.
// A new page is written by the thread of its first token.  The work is a few
// bytes per token: what bounds it is the latency of one launch, three loads
// that depend on one another (lengths, free list, stores) and two block sums, 3.7
// us in a graph for 8 requests (a call by itself 6.4, its CPU time); the chain of
// loads along a tree's parents, 7.3 us for trees of up to 64 nodes of 256 requests
// (a call 7.5); and, of 1001 prompts of up to 1023 tokens, 9.3 us (a call 11.8),
// instructions: about three quarters of them per token (a bisection of ten steps,
// three divisions by the page size, two narrow stores), the others the sums.
#include <algorithm>

#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kPlanThreads = 512;

// Exclusive sums over the block of one pair per thread; totals in `tot`.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t (*warp_sum)[2], int64_t (&tot)[2]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += ua, ib += ub;
  }
  if (lane == 31) warp_sum[w][0] = ia, warp_sum[w][1] = ib;
  __syncthreads();
  int64_t ba = 0, bb = 0, ta = 0, tb = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    const int64_t sa = warp_sum[i][0], sb = warp_sum[i][1];
    if (i < w) ba += sa, bb += sb;
    ta += sa, tb += sb;
  }
  a = ba + ia - a;
  b = bb + ib - b;
  tot[0] = ta;
  tot[1] = tb;
}

__device__ __forceinline__ int32_t clamp_i32(int64_t v) { return (int32_t)min(v, (int64_t)INT32_MAX); }

__global__ void __launch_bounds__(kPlanThreads)
kv_plan_kernel(const KvPlanArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                    // [R]: exclusive sums of the new tokens
  int32_t* s_base = sm + a.R;            // [R]: exclusive sums of the pages taken
  int32_t* s_ctx = sm + 2 * a.R;         // [R]
  __shared__ int64_t warp_sum[kPlanThreads / 32][2];
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const uint32_t P = a.page_size;
  for (int r = threadIdx.x; r < a.R; r += kPlanThreads) {
    int32_t L = a.ctx[r], n = a.fresh[r];
    if (L < 0 || n < 0) {                // such a request gets nothing
      if (blockIdx.x == 0) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      L = n = 0;
    }
    const uint32_t have = ((uint32_t)L + P - 1) / P;
    const int64_t need = ((int64_t)L + n + P - 1) / P;
    s_ctx[r] = L;
    s_cu[r] = n;
    s_base[r] = (int32_t)(need - have);
  }
  __syncthreads();
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  int64_t tok = 0, pg = 0, tot[2];
  for (int r = r0; r < r1; ++r) tok += s_cu[r], pg += s_base[r];
  block_scan2(tok, pg, warp_sum, tot);
  for (int r = r0; r < r1; ++r) {
    const int32_t n = s_cu[r], t = s_base[r];
    s_cu[r] = clamp_i32(tok);
    s_base[r] = clamp_i32(pg);
    if (blockIdx.x == 0) a.cu[r] = clamp_i32(tok);
    tok += n;
    pg += t;
  }
  __syncthreads();
  const int64_t total = tot[0];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.cu[a.R] = clamp_i32(total);
    a.taken[0] = clamp_i32(tot[1]);
    if (total > a.max_tokens) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    if (tot[1] > a.n_free) set_status(a.dev_status, QMM_ERR_NO_PAGES);
  }
  for (int64_t t64 = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x; t64 < a.max_tokens;
       t64 += (int64_t)gridDim.x * kPlanThreads) {
    const int t = (int)t64;
    uint32_t* mrow = a.mask != nullptr ? a.mask + (int64_t)t * a.ld_mask : nullptr;
    if (t >= total) {                    // past the step's tokens
      a.slots[t] = -1;
      a.positions[t] = 0;
      if (mrow != nullptr)
        for (int w = 0; w < a.mask_words; ++w) mrow[w] = 0;
      continue;
    }
    int lo = 0, hi = a.R;                // the last r with cu[r] <= t (empty requests share a start)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int i = t - s_cu[lo];
    const int32_t L = s_ctx[lo];
    const uint32_t p = (uint32_t)L + (uint32_t)i;   // < 2^32
    const uint32_t col = p / P, off = p % P, have = ((uint32_t)L + P - 1) / P;
    int32_t page = -1;
    if (col < a.max_blocks) {
      int32_t* entry = a.table + (int64_t)lo * a.ld_table + col;
      if (col < have) {
        page = *entry;
      } else {
        const int64_t f = (int64_t)s_base[lo] + (col - have);
        if (f < a.n_free) {
          page = a.free_pages[f];
          if (off == 0) *entry = page;
        }
      }
    } else {
      set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    }
    a.slots[t] = page < 0 ? -1 : (int64_t)page * P + off;
    int depth = i;
    if (mrow != nullptr) {
      // the chain of ancestors has falling indexes, so that each word is done
      // before the next lower one begins
      const int32_t* par = a.parents + (t - i);
      depth = -1;
      int at = i, w = a.mask_words - 1;
      uint32_t bits = 0;
      if (i >= 32 * a.mask_words) {
        set_status(a.dev_status, QMM_ERR_INVALID_ARG);
        at = -1;
      }
      while (at >= 0) {
        for (; w > (at >> 5); --w) mrow[w] = bits, bits = 0;
        bits |= 1u << (at & 31);
        ++depth;
        const int up = par[at];
        if (up >= at || up < -1) {       // not an earlier token of the request
          set_status(a.dev_status, QMM_ERR_INVALID_ARG);
          break;
        }
        at = up;
      }
      for (; w >= 0; --w) mrow[w] = bits, bits = 0;
      depth = max(depth, 0);
    }
    a.positions[t] = (int32_t)min((int64_t)L + depth, (int64_t)INT32_MAX);
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t)a.R * 12;
  static std::atomic<uint64_t> set{0};
  const cudaError_t err = set_once(set, (const void*)kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)(kPlanMaxRequests * 12));
  if (err != cudaSuccess) return err;
  const int64_t blocks = ((int64_t)a.max_tokens + kPlanThreads - 1) / kPlanThreads;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(blocks, 2 * attn_sm_count()));
  return launch_pdl(kv_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, stream, a);
}

}  // namespace qmm

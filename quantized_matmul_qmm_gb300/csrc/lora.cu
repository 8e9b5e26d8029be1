// Low-rank adapters of many requests beside a shared projection:
//     out[m] = base[m] + s_a B_a (A_a x_m),   a = ids[m]
// with x_m of K values, A_a [r][K], B_a [N][r], r up to 256.
//
// Bound: bytes.  base and out are 8 N bytes a row and X 2 K; the products are
// 2 r (K + N) operations a row, a few per byte for ordinary ranks.  So the
// kernels keep rows of one adapter together (each adapter's A and B are read
// once per tile of rows) and stream X, base and out once; mma.sync carries the
// products.
//
// The inner sums h = A x are fp32.  For the second product h * s_a is written
// as two bf16 terms, h = hi + lo within 2^-16 |h|: with one term (2^-9) the
// rounding of h would be far above the fp32 rounding of out.
#include <algorithm>

#include "beside.h"
#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kTile = 64;                 // rows of an item, all of one adapter
constexpr int kRouteThreads = 1024;
constexpr int kThreads = 256;
constexpr int kColBlock = 512;            // output columns of a block of the second product
constexpr int kMaxSplit = 8;              // parts of K

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

int64_t max_tiles(int64_t M, int64_t n_adapters) { return M / kTile + std::min(n_adapters + 1, M); }
int rank_stride(int64_t max_rank) { return (int)((max_rank + 31) / 32 * 32); }
int k_split(int64_t M, int64_t K) {
  const int64_t tiles = (M + kTile - 1) / kTile;
  int64_t split = 1;
  while (split < kMaxSplit && tiles * split < 2 * attn_sm_count() && K / (2 * split) >= 256) split *= 2;
  return (int)split;
}

struct Workspace {
  int* head;      // [0]: tiles of rows with an adapter, [1]: all tiles
  int4* tiles;    // adapter (-1: none), first place in rows, rows
  int* rows;      // [M] row numbers by adapter
  float* part;    // [split][M][rank_stride] inner sums by place in rows
};

// ---- rows by adapter ---------------------------------------------------------
// One block: counts per adapter, their sums, the tiles, then every row's place.
// Rows of one warp with one adapter stay together, so that a prompt's rows do.
__global__ void __launch_bounds__(kRouteThreads)
lora_route_kernel(LoraArgs a, Workspace w, bool copy_none) {
  extern __shared__ int counts[];         // [n_adapters + 1]: rows, then the next place
  __shared__ int2 warp_sums[32];
  __shared__ int2 carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int buckets = a.n_adapters + 1;   // the last: no adapter
  for (int i = tid; i < buckets; i += kRouteThreads) counts[i] = 0;
  if (tid == 0) carry = make_int2(0, 0);
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  __syncthreads();
  auto bucket_of = [&](int m, bool report) {
    const int id = a.ids[m];
    if (id == -1) return a.n_adapters;
    if (id < 0 || id >= a.n_adapters) {
      if (report) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      return a.n_adapters;
    }
    if (a.ranks == nullptr) return id;
    const int r = a.ranks[id];
    if (r < 0 || r > a.max_rank) {
      if (report) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      return a.n_adapters;
    }
    return r == 0 ? a.n_adapters : id;
  };
  for (int m0 = 0; m0 < a.M; m0 += kRouteThreads) {
    const int m = m0 + tid, b = m < a.M ? bucket_of(m, true) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && lane == __ffs(same) - 1) atomicAdd(&counts[b], __popc(same));
  }
  __syncthreads();
  for (int b0 = 0; b0 < buckets; b0 += kRouteThreads) {
    const int b = b0 + tid;
    const int n = b < buckets ? counts[b] : 0;
    const bool none = b == a.n_adapters;
    const int t = none && !copy_none ? 0 : (n + kTile - 1) / kTile;
    int2 s = make_int2(n, t);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
      if (lane >= o) s.x += x, s.y += y;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int2 before = carry;
    for (int i = 0; i < warp; ++i) before.x += warp_sums[i].x, before.y += warp_sums[i].y;
    const int first = before.x + s.x - n, tile0 = before.y + s.y - t;
    if (b < buckets) {
      counts[b] = first;
      for (int i = 0; i < t; ++i)
        w.tiles[tile0 + i] = make_int4(none ? -1 : b, first + i * kTile, min(kTile, n - i * kTile), 0);
      if (none) w.head[0] = tile0, w.head[1] = tile0 + t;
    }
    __syncthreads();
    if (tid == kRouteThreads - 1) carry = make_int2(first + n, tile0 + t);
    __syncthreads();
  }
  for (int m0 = 0; m0 < a.M; m0 += kRouteThreads) {
    const int m = m0 + tid, b = m < a.M ? bucket_of(m, false) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, b);
    const int leader = __ffs(same) - 1;
    int at = 0;
    if (b >= 0 && lane == leader) at = atomicAdd(&counts[b], __popc(same));
    at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
    if (b >= 0) w.rows[at] = m;
  }
}

// ---- h = A x ------------------------------------------------------------------
// A block takes a tile of 64 rows and one part of K; its warps 16 rows by half of
// that part each.  Both operands come straight from memory as 16-byte loads of
// eight consecutive k per lane: which k a fragment position stands for is free as
// long as both operands agree.
__global__ void __launch_bounds__(kThreads)
lora_shrink_kernel(LoraArgs a, Workspace w, int rs) {
  __shared__ float half[4][32][33];
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int tile = blockIdx.x;
  if (tile >= w.head[0]) return;
  const int4 it = w.tiles[tile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int group = warp & 3, kh = warp >> 2;
  const int rank = a.ranks != nullptr ? a.ranks[it.x] : a.max_rank;
  const int chunks = (a.K + 31) / 32;                      // of 32 k
  const int parts = 2 * gridDim.y, part = 2 * blockIdx.y + kh;
  const int c0 = (int)((int64_t)chunks * part / parts), c1 = (int)((int64_t)chunks * (part + 1) / parts);
  const int r0 = group * 16 + g, r1 = r0 + 8;              // this lane's rows of the tile
  const __nv_bfloat16* x0 = r0 < it.z ? a.X + (int64_t)w.rows[it.y + r0] * a.ldx : nullptr;
  const __nv_bfloat16* x1 = r1 < it.z ? a.X + (int64_t)w.rows[it.y + r1] * a.ldx : nullptr;
  const __nv_bfloat16* A = a.A + it.x * a.a_slot;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int j0 = 0; j0 < rank; j0 += 64) {
    float acc[8][4] = {};
    if (group * 16 < it.z) {
#pragma unroll 2
      for (int c = c0; c < c1; ++c) {
        const int k = c * 32 + 8 * tig;
        const uint4 p = x0 != nullptr && k < a.K ? ldg128(x0 + k) : zero;
        const uint4 q = x1 != nullptr && k < a.K ? ldg128(x1 + k) : zero;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (j0 + 8 * n >= rank) break;
          const int j = j0 + 8 * n + g;
          const uint4 b = j < rank && k < a.K ? ldg128(A + j * a.a_rank + k) : zero;
          mma_bf16_16816(acc[n], p.x, q.x, p.y, q.y, b.x, b.y);
          mma_bf16_16816(acc[n], p.z, q.z, p.w, q.w, b.z, b.w);
        }
      }
    }
    if (kh == 1) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) half[group][lane][n * 4 + i] = acc[n][i];
    }
    __syncthreads();
    if (kh == 0) {
      float* to = w.part + ((int64_t)blockIdx.y * a.M + it.y) * rs;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int j = j0 + 8 * n + 2 * tig;
        if (j0 + 8 * n >= rs) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += half[group][lane][n * 4 + i];
        if (r0 < it.z) *reinterpret_cast<float2*>(to + (int64_t)r0 * rs + j) = make_float2(acc[n][0], acc[n][1]);
        if (r1 < it.z) *reinterpret_cast<float2*>(to + (int64_t)r1 * rs + j) = make_float2(acc[n][2], acc[n][3]);
      }
    }
    __syncthreads();
  }
}

// ---- out = base + (s h) B^T -----------------------------------------------------
QMM_DEV uint32_t two_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

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

// A block takes a tile of 64 rows and 512 columns.  The tile's h lies in shared
// memory as two bf16 terms; a warp's columns are dealt to fragment positions so
// that a lane's accumulators are four neighbouring columns of a row.
template <bool kVec>
__global__ void __launch_bounds__(kThreads)
lora_expand_kernel(LoraArgs a, Workspace w, int rs, int split) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  umma::pdl_wait();
  const int tile = blockIdx.x;
  if (tile >= w.head[1]) return;
  const int4 it = w.tiles[tile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const int group = warp & 3, ch = warp >> 2;
  const int col0 = blockIdx.y * kColBlock;
  if (it.x < 0) {                                          // no adapter: base as it is
    for (int r = warp; r < it.z; r += kThreads / 32) {
      const int64_t m = w.rows[it.y + r];
      for (int c = col0 + lane * 4; c < min(col0 + kColBlock, a.N); c += 128)
        store4<kVec>(a.out + m * a.ldo, c, a.N,
                     a.base != nullptr ? load4<kVec>(a.base + m * a.ldb, c, a.N) : make_float4(0, 0, 0, 0));
    }
    return;
  }
  const int rank = a.ranks != nullptr ? a.ranks[it.x] : a.max_rank;
  const float scale = a.scales != nullptr ? a.scales[it.x] : 1.f;
  const int chunks = (rank + 31) / 32;
  const int hs = chunks * 32 + 8;                          // row stride of h: rows fall on different banks
  uint16_t* hi = reinterpret_cast<uint16_t*>(smem_raw);
  uint16_t* lo = hi + kTile * hs;
  for (int i = tid; i < kTile * chunks * 8; i += kThreads) {
    const int r = i / (chunks * 8), j = i % (chunks * 8) * 4;
    float4 h = make_float4(0, 0, 0, 0);
    if (r < it.z) {
      for (int s = 0; s < split; ++s) {                    // in order: the same sums every time
        const float4 p = *reinterpret_cast<const float4*>(w.part + ((int64_t)s * a.M + it.y + r) * rs + j);
        h.x += p.x, h.y += p.y, h.z += p.z, h.w += p.w;
      }
      h.x = j < rank ? h.x * scale : 0.f;
      h.y = j + 1 < rank ? h.y * scale : 0.f;
      h.z = j + 2 < rank ? h.z * scale : 0.f;
      h.w = j + 3 < rank ? h.w * scale : 0.f;
    }
    const uint32_t a0 = two_bf16(h.x, h.y), a1 = two_bf16(h.z, h.w);
    *reinterpret_cast<uint2*>(hi + r * hs + j) = make_uint2(a0, a1);
    *reinterpret_cast<uint2*>(lo + r * hs + j) =
        make_uint2(two_bf16(h.x - bf16lo_to_f32(a0), h.y - bf16hi_to_f32(a0)),
                   two_bf16(h.z - bf16lo_to_f32(a1), h.w - bf16hi_to_f32(a1)));
  }
  __syncthreads();
  const int r0 = group * 16 + g, r1 = r0 + 8;
  if (group * 16 >= it.z) return;
  const int64_t m0 = r0 < it.z ? w.rows[it.y + r0] : -1, m1 = r1 < it.z ? w.rows[it.y + r1] : -1;
  const __nv_bfloat16* B = a.B + it.x * a.b_slot;
  for (int cb = col0 + ch * 64; cb < min(col0 + kColBlock, a.N); cb += 128) {
    float4 y0[4], y1[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = cb + 16 * p + 4 * tig;
      y0[p] = y1[p] = make_float4(0, 0, 0, 0);
      if (a.base != nullptr) {
        if (m0 >= 0) y0[p] = load4<kVec>(a.base + m0 * a.ldb, col, a.N);
        if (m1 >= 0) y1[p] = load4<kVec>(a.base + m1 * a.ldb, col, a.N);
      }
    }
    float acc[8][4] = {};
    for (int c = 0; c < chunks; ++c) {
      const int j = c * 32 + 8 * tig;
      const uint4 h0 = *reinterpret_cast<const uint4*>(hi + r0 * hs + j);
      const uint4 h1 = *reinterpret_cast<const uint4*>(hi + r1 * hs + j);
      const uint4 l0 = *reinterpret_cast<const uint4*>(lo + r0 * hs + j);
      const uint4 l1 = *reinterpret_cast<const uint4*>(lo + r1 * hs + j);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int col = cb + 16 * (n >> 1) + 4 * (g >> 1) + (g & 1) + 2 * (n & 1);
        uint4 b = make_uint4(0, 0, 0, 0);
        if (j < rank && col < a.N) b = keep8(ldg128(B + col * a.b_row + j), rank - j);
        mma_bf16_16816(acc[n], l0.x, l1.x, l0.y, l1.y, b.x, b.y);
        mma_bf16_16816(acc[n], l0.z, l1.z, l0.w, l1.w, b.z, b.w);
        mma_bf16_16816(acc[n], h0.x, h1.x, h0.y, h1.y, b.x, b.y);
        mma_bf16_16816(acc[n], h0.z, h1.z, h0.w, h1.w, b.z, b.w);
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = cb + 16 * p + 4 * tig;
      const float(&e)[4] = acc[2 * p], (&f)[4] = acc[2 * p + 1];
      if (m0 >= 0)
        store4<kVec>(a.out + m0 * a.ldo, col, a.N,
                     make_float4(y0[p].x + e[0], y0[p].y + e[1], y0[p].z + f[0], y0[p].w + f[1]));
      if (m1 >= 0)
        store4<kVec>(a.out + m1 * a.ldo, col, a.N,
                     make_float4(y1[p].x + e[2], y1[p].y + e[3], y1[p].z + f[2], y1[p].w + f[3]));
    }
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank) {
  if (M == 0) return 0;
  return 256 + pad256((size_t)max_tiles(M, n_adapters) * sizeof(int4)) + pad256((size_t)M * 4) +
         pad256((size_t)k_split(M, K) * M * rank_stride(max_rank) * 4);
}

cudaError_t launch_lora_add(const LoraArgs& a, void* workspace, cudaStream_t stream) {
  const int tiles = (int)max_tiles(a.M, a.n_adapters);
  const int rs = rank_stride(a.max_rank), split = k_split(a.M, a.K);
  uint8_t* p = static_cast<uint8_t*>(workspace);
  Workspace w;
  w.head = reinterpret_cast<int*>(p);
  p += 256;
  w.tiles = reinterpret_cast<int4*>(p);
  p += pad256((size_t)tiles * sizeof(int4));
  w.rows = reinterpret_cast<int*>(p);
  p += pad256((size_t)a.M * 4);
  w.part = reinterpret_cast<float*>(p);
  const bool in_place = a.base == a.out;
  lora_route_kernel<<<1, kRouteThreads, (a.n_adapters + 1) * sizeof(int), stream>>>(a, w, !in_place);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  if ((err = launch_pdl(lora_shrink_kernel, dim3(tiles, split), dim3(kThreads), 0, stream, a, w, rs)) != cudaSuccess)
    return err;
  const bool vec = a.N % 4 == 0 && aligned(a.out, 16) && a.ldo % 4 == 0 &&
                   (a.base == nullptr || (aligned(a.base, 16) && a.ldb % 4 == 0));
  const size_t smem = (size_t)2 * kTile * (rs + 8) * 2;
  const dim3 grid(tiles, (a.N + kColBlock - 1) / kColBlock);
  static std::atomic<uint64_t> done[2];
  auto kern = vec ? lora_expand_kernel<true> : lora_expand_kernel<false>;
  err = set_once(done[vec], reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                 2 * kTile * ((int)kLoraMaxRank + 8) * 2);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, grid, dim3(kThreads), smem, stream, a, w, rs, split);
}

}  // namespace qmm

// The adapters' two products in calls of many rows, on tcgen05:
//     h_m = s_a A_a x_m,  as two bf16 terms;   out[m] = base[m] + h_m B_a^T.
//
// Bound: bytes, 2 K a row for the first and 8 a value of out (base in, out back) for
// the second.  The products are 2 r operations for 2 bytes of X, and 4 r (both
// terms) for 8 bytes of out: from ranks of about 100 on more than mma.sync (600
// TFLOP/s measured on this part) does in that time.
//
// Measured: 4097 prompt rows over 6 adapters of ranks 8 to 64 at K = N = 4608 (192 MB)
// 55 us with the routing's 7, 0.52 of a copy's rate; 16000 rows 168 us, 0.66.  2048 rows at
// K = 2048, N = 12288 and ranks 100 to 256 70 us, 0.48.  What is lost: three launches
// that cannot overlap (the second product's blocks take a whole SM's shared memory), the
// first's meeting over the cluster, and in the second what its registers hold of base
// under way.
//
// Both kernels take 128 rows of one adapter at a time, the tensor cores' height;
// partly filled tiles cost products, not bytes.
#include <algorithm>
#include <atomic>

#include "attn_umma.cuh"
#include "kv_cache.h"
#include "lora_work.cuh"

namespace qmm {
namespace {

using namespace umma;

constexpr int kChunk = 64;                                  // k or ranks of a stage: 128 bytes, one swizzle row
constexpr int kTileBytes16 = 128 * kChunk * 2;

// ---- h = s A x -----------------------------------------------------------------
// A cluster takes a tile, its blocks a part of K each.  A block's threads copy the
// rows' 16-byte pieces (rows lie anywhere) and the adapter's into the swizzled
// layout of the operands, several stages ahead; one thread issues the products of
// a stage for all ranks at once.  The blocks' sums meet over shared memory, 128
// ranks at a time: each block adds up its share of the rows, in order, and writes
// their two terms.
constexpr int kInnerThreads = 256;
constexpr int kInnerRanks = 128;                            // whose sums meet at a time
constexpr int kInnerPitch = kInnerRanks + 4;                // floats of a row of sums
constexpr int kInnerSums = 128 * kInnerPitch * 4;
constexpr int kInnerMaxStages = 4;
// Two blocks on an SM and never three, of whichever calls: each may hold 256 columns of
// TMEM while it waits for its cluster, so that a third would wait for columns, and two
// clusters' blocks could wait for one another's.  By shared memory, whatever registers
// they take: an SM has 228 KB, of which a block uses one besides its own.
constexpr int kInnerLeast = 77 * 1024, kInnerMost = 112 * 1024;
static_assert(3 * (kInnerLeast + 1024) > 228 * 1024 && 2 * (kInnerMost + 1024) <= 228 * 1024, "two blocks on an SM");
static_assert(1024 + kInnerSums <= kInnerLeast, "the sums");

struct InnerParams {
  LoraArgs a;
  LoraWork w;
  int rs, stages, stage_bytes, cluster;
  uint32_t tmem_cols;
};

template <int kPending>
QMM_DEV void wait_copies(int pending) {
  if (pending == kPending) cp_async_wait<kPending>();
  else if constexpr (kPending > 0) wait_copies<kPending - 1>(pending);
}

__global__ void __launch_bounds__(kInnerThreads, 2)
lora_inner_kernel(const InnerParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t done[kInnerMaxStages], last;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = smem_align(smem_raw, 1024);
  const LoraArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int block = blockIdx.x % p.cluster;
  if (tid == 0) {
    for (int s = 0; s < kInnerMaxStages; ++s) mbar_init(&done[s], 1);
    mbar_init(&last, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const int clusters = gridDim.x / p.cluster;
  // the first tile is read beside their number: there is room for as many as clusters
  int4 it = p.w.tiles[blockIdx.x / p.cluster];
  const int tiles = p.w.head[0];
  const int piece = tid & 7, row0 = tid >> 3;               // this thread's 16 bytes of rows row0 + 32 i
  uint32_t done_uses = 0;                                   // stages filled so far
  uint32_t last_par = 0;
  bool ok = true;

  for (int tile = blockIdx.x / p.cluster; tile < tiles; tile += clusters) {
    if (tile >= clusters) it = p.w.tiles[tile];
    const int rank = a.ranks != nullptr ? a.ranks[it.x] : a.max_rank;
    const float scale = a.scales != nullptr ? a.scales[it.x] : 1.f;
    const int n16 = (rank + 15) / 16 * 16;                  // ranks of the products
    const int chunks = (a.K + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * block / p.cluster), c1 = (int)((int64_t)chunks * (block + 1) / p.cluster);
    const __nv_bfloat16* x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 32 * i;
      x[i] = r < it.z ? a.X + (int64_t)p.w.rows[it.y + r] * a.ldx : nullptr;
    }
    const __nv_bfloat16* A = a.A + it.x * a.a_slot;
    auto copy = [&](int c, int s) {
      const uint32_t to = smem_u32(smem) + (uint32_t)s * p.stage_bytes + (uint32_t)((piece ^ (row0 & 7)) << 4);
      const int k = c * kChunk + piece * 8;
      const bool in = k < a.K;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = in && x[i] != nullptr;
        cp_async16_zfill(to + (uint32_t)(row0 + 32 * i) * 128, there ? x[i] + k : a.X, there ? 16 : 0);
      }
      for (int j = row0; j < n16; j += 32) {
        const bool there = in && j < rank;
        cp_async16_zfill(to + kTileBytes16 + (uint32_t)j * 128, there ? A + j * a.a_rank + k : a.A, there ? 16 : 0);
      }
    };
    const uint32_t idesc = idesc_f16(128, n16, true);
    const int n = c1 - c0;
    for (int i = 0; i < n + p.stages - 1; ++i) {
      if (i < n) {
        const uint32_t use = done_uses + i;                 // of the ring
        const int s = use % p.stages;
        // the products that read this stage's last contents
        if (use >= (uint32_t)p.stages)
          ok = ok && mbar_wait(&done[s], (use / p.stages - 1) & 1, &abort_flag, a.dev_status);
        if (ok) copy(c0 + i, s);
      }
      cp_async_commit();
      const int j = i - (p.stages - 1);
      if (j < 0) continue;
      wait_copies<kInnerMaxStages - 1>(p.stages - 1);
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0 && ok) {
        tc_fence_after();
        const int s = (done_uses + j) % p.stages;
        const uint64_t dx = desc_kmajor_sw128(smem_u32(smem) + s * p.stage_bytes);
        const uint64_t da = desc_kmajor_sw128(smem_u32(smem) + s * p.stage_bytes + kTileBytes16);
#pragma unroll
        for (int k = 0; k < kChunk / 16; ++k) umma_f16(tmem, dx + 2 * k, da + 2 * k, idesc, j > 0 || k > 0);
        umma_commit(&done[s]);
        if (j == n - 1) umma_commit(&last);
      }
    }
    done_uses += n;
    if (n > 0) {
      ok = ok && mbar_wait(&last, last_par, &abort_flag, a.dev_status);
      last_par ^= 1;
    }
    // A block that gave up goes on with the others: its sums are not valid, and the
    // status says so.
    tc_fence_after();
    __syncthreads();                                        // the stages are free
    float* sums = reinterpret_cast<float*>(smem);           // [128][kInnerPitch]
    const uint32_t sums_addr = smem_u32(sums);
    const int q = warp & 3, half = warp >> 2;
    for (int j0 = 0; j0 < rank; j0 += kInnerRanks) {
      for (int jj = 32 * half; jj < kInnerRanks && 32 * q < it.z && j0 + jj < n16; jj += 64) {
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(j0 + jj), r);
        tmem_wait_ld();
        float* to = sums + (32 * q + lane) * kInnerPitch + jj;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<uint4*>(to + i) =
              n > 0 ? make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]) : make_uint4(0, 0, 0, 0);
      }
      tc_fence_before();
      cluster_sync();
      // this block's rows, neighbouring lanes at neighbouring ranks: the other blocks'
      // memory is read in whole rows (scattered 16-byte reads took 10 times as long)
      const int share = (it.z + p.cluster - 1) / p.cluster, r0 = block * share;
      const int quads = min(kInnerRanks, p.rs - j0) / 4;    // of four ranks, in a row
      const int all = min(share, it.z - r0) * quads;
      for (int i0 = tid; i0 < all; i0 += 2 * kInnerThreads) {
        int r[2], j[2];
        uint32_t at[2];
        bool in[2];
        float4 s[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = i0 + e * kInnerThreads;
          r[e] = r0 + i / quads, j[e] = i % quads * 4;
          at[e] = sums_addr + (uint32_t)(r[e] * kInnerPitch + j[e]) * 4;
          in[e] = i < all && j0 + j[e] < n16;
        }
        cluster_sums(at, in, p.cluster, s);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int left = rank - j0 - j[e];
          s[e].x = left > 0 ? s[e].x * scale : 0.f;
          s[e].y = left > 1 ? s[e].y * scale : 0.f;
          s[e].z = left > 2 ? s[e].z * scale : 0.f;
          s[e].w = left > 3 ? s[e].w * scale : 0.f;
          if (e == 1 && i0 + kInnerThreads >= all) break;
          uint16_t* to = p.w.h + (int64_t)(it.y + r[e]) * 2 * p.rs + j0 + j[e];
          put_terms(to, to + p.rs, s[e]);
        }
      }
      cluster_sync();
    }
    tc_fence_after();
    fence_proxy_async_smem();
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ---- out = base + h B^T ----------------------------------------------------------
// A block per SM walks over units of 128 rows by 128 columns.  One warp loads the
// two terms of h and the rows of B by TMA, 64 ranks a stage, and another issues the
// products of both terms with the same B into one of four accumulators; three groups of
// four warps take the units in turn.  A warp owns 32 rows, 32 columns at a time: their base
// values are on their way into registers two such steps ahead, the accumulator goes
// through the warp's corner of shared memory so that rows are read and written 128
// bytes at a time, and no warp waits for another.  14 warps leave a thread 128
// registers, where two steps' values fit; with 16 of these warps and one step ahead
// 4097 rows at K = N = 4608 took 56.6 us, so 55.0.
constexpr int kGroups = 3;
constexpr int kEpiWarps = 4 * kGroups;
constexpr int kOuterThreads = (kEpiWarps + 2) * 32;
constexpr int kCols = 128;
constexpr int kBuffers = 4;
constexpr int kStages = 3;
constexpr int kStageBytes = 3 * kTileBytes16;               // both terms of h, B
constexpr int kPitch = 32 + 4;                              // floats of a row of a warp's corner
constexpr int kCorner = 32 * kPitch * 4;
constexpr int kOuterSmem = 1024 + kStages * kStageBytes + kEpiWarps * kCorner;

struct OuterParams {
  LoraArgs a;
  LoraWork w;
  int rs, col_blocks;
  bool copy_none;
};

// A unit of the walk, in few registers.
struct Unit {
  int adapter, first, size, col0;   // -1: none; first place; rows and the rank above them, 0: past the end
  QMM_DEV int rows() const { return size & 0xFFFF; }
  QMM_DEV int rank() const { return size >> 16; }
  QMM_DEV int chunks() const { return (rank() + kChunk - 1) / kChunk; }
  // Blocks of 32 rows that the accumulator holds: where one or two hold the rows they
  // are there four times or twice, so that all warps of a group have columns to take.
  QMM_DEV int blocks() const { return rows() <= 32 ? 1 : rows() <= 64 ? 2 : 4; }
};

// The units first, first + step, .. of a warp's walk.  What they are is read for 32 of
// them at a time, one per lane: one chain of dependent loads in 32 units.
template <bool kAdapters>
struct Walk {
  const OuterParams& p;
  uint32_t units, at, step;   // the unit at hand
  int left = 0;               // of those in the lanes, behind it
  Unit mine;

  QMM_DEV Walk(const OuterParams& params, uint32_t all, uint32_t from, uint32_t by)
      : p(params), units(all), at(from), step(by) {
    fetch();
  }
  QMM_DEV void fetch() {
    const uint32_t i = at + (threadIdx.x & 31) * step;
    mine = Unit{-1, 0, 0, 0};
    left = 31;
    if (i < units) {
      const uint32_t tile = i / (uint32_t)p.col_blocks;
      const int4 t = p.w.tiles[tile];
      const int rank = t.x < 0 ? 0 : p.a.ranks != nullptr ? p.a.ranks[t.x] : p.a.max_rank;
      mine = Unit{t.x, t.y, t.z | rank << 16, (int)(i - tile * p.col_blocks) * kCols};
    }
  }
  QMM_DEV Unit unit() const {
    const int l = 31 - left;
    return Unit{kAdapters ? __shfl_sync(0xffffffffu, mine.adapter, l) : 0, __shfl_sync(0xffffffffu, mine.first, l),
                __shfl_sync(0xffffffffu, mine.size, l), __shfl_sync(0xffffffffu, mine.col0, l)};
  }
  QMM_DEV bool there() const { return at < units; }
  QMM_DEV void next() {
    at += step;
    if (--left < 0) fetch();
  }
};

template <bool kVec>
__global__ void __launch_bounds__(kOuterThreads, 1)
lora_outer_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmH32,
                  const __grid_constant__ CUtensorMap tmB, const OuterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], tfull[kBuffers], tempty[kBuffers];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = smem_align(smem_raw, 1024);
  const LoraArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int b = 0; b < kBuffers; ++b) mbar_init(&tfull[b], 1), mbar_init(&tempty[b], 4);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmH);
    tma_prefetch_desc(&tmB);
  }
  if (warp == kEpiWarps) {
    tmem_alloc(&tmem_slot, kBuffers * kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  const uint32_t units = (uint32_t)p.w.head[p.copy_none ? 1 : 0] * p.col_blocks;

  if (warp == kEpiWarps) {
    // fills the stages
    Walk<true> f(p, units, blockIdx.x, gridDim.x);
    uint32_t filled = 0;
    bool ok = true;
    for (; f.there() && ok; f.next()) {
      const Unit u = f.unit();
      const int chunks = u.chunks();
      for (int c = 0; c < chunks && ok; ++c, ++filled) {
        const int s = filled % kStages;
        if (filled >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], (filled / kStages - 1) & 1, &abort_flag, a.dev_status));
        if (!ok) break;
        if (lane == 0) {
          uint8_t* to = smem + s * kStageBytes;
          mbar_arrive_expect_tx(&full[s], kStageBytes);
          const int blocks = u.blocks();
          if (blocks == 4) {
            tma_load_2d(to, &tmH, &full[s], c * kChunk, u.first);
            tma_load_2d(to + kTileBytes16, &tmH, &full[s], p.rs + c * kChunk, u.first);
          } else {
            for (int i = 0; i < 8; ++i)
              tma_load_2d(to + i * (kTileBytes16 / 4), &tmH32, &full[s], (i >> 2) * p.rs + c * kChunk,
                          u.first + 32 * (i & (blocks - 1)));
          }
          tma_load_3d(smem_u32(to + 2 * kTileBytes16), &tmB, &full[s], c * kChunk, u.col0, u.adapter);
        }
        __syncwarp();
      }
    }
    // copies already issued land before the block leaves, also where a wait gave up
    for (uint32_t u = filled > kStages ? filled - kStages : 0; u < filled; ++u)
      mbar_drain(&full[u % kStages], (u / kStages) & 1);
  } else if (warp == kEpiWarps + 1) {
    // issues the products: all lanes in step, one elected
    const uint32_t one = elect_one();
    uint32_t used = 0;
    Walk<true> m(p, units, blockIdx.x, gridDim.x);
    bool ok = true;
    for (int n = 0; m.there() && ok; m.next(), ++n) {
      const Unit u = m.unit();
      const int chunks = u.chunks(), rank = u.rank();
      const int buf = n % kBuffers;
      if (n >= kBuffers)
        ok = __all_sync(0xffffffffu, mbar_wait(&tempty[buf], (n / kBuffers - 1) & 1, &abort_flag, a.dev_status));
      const uint32_t d = tmem + buf * kCols;
      for (int c = 0; c < chunks && ok; ++c, ++used) {
        const int s = used % kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (used / kStages) & 1, &abort_flag, a.dev_status));
        if (!ok) break;
        uint8_t* at = smem + s * kStageBytes;
        const int left = rank - c * kChunk;
        if (left < kChunk && left % 16 != 0 && rank < a.max_rank) {
          // what lies behind the adapter's rank in the last step of 16: zeros, since 0
          // times an infinity or NaN is none (h is zero there)
          const int piece = left / 8;
          for (int r = lane; r < kCols; r += 32) {
            uint8_t* row = at + 2 * kTileBytes16 + r * 128;
            uint4* v = reinterpret_cast<uint4*>(row + ((piece ^ (r & 7)) << 4));
            uint32_t w[4] = {v->x, v->y, v->z, v->w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int keep = left % 8 - 2 * i;            // values of this word that stay
              if (keep <= 0) w[i] = 0;
              else if (keep == 1) w[i] &= 0xFFFFu;
            }
            *v = make_uint4(w[0], w[1], w[2], w[3]);
            if (piece % 2 == 0)
              *reinterpret_cast<uint4*>(row + (((piece + 1) ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        constexpr uint32_t idesc = idesc_f16(128, kCols, true);
        const uint64_t b = desc_kmajor_sw128(smem_u32(at + 2 * kTileBytes16));
        const uint64_t hi = desc_kmajor_sw128(smem_u32(at)), lo = desc_kmajor_sw128(smem_u32(at + kTileBytes16));
        const int steps = min(kChunk / 16, (left + 15) / 16);
        // the smaller term first
#pragma unroll
        for (int k = 0; k < kChunk / 16; ++k)
          if (k < steps) umma_f16_one(one, d, lo + 2 * k, b + 2 * k, idesc, c > 0 || k > 0);
#pragma unroll
        for (int k = 0; k < kChunk / 16; ++k)
          if (k < steps) umma_f16_one(one, d, hi + 2 * k, b + 2 * k, idesc, 1);
        umma_commit_one(one, &empty[s]);
      }
      if (ok) umma_commit_one(one, &tfull[buf]);            // also without products: buffers take turns
    }
  } else {
    const int group = warp / 4, q = warp & 3;
    float* corner = reinterpret_cast<float*>(smem + kStages * kStageBytes + warp * kCorner);
    // four values of row 32 q + 4 v + lane / 8: columns cl + 0..3, or in steps of eight
    const int sub = lane >> 3, cl = kVec ? (lane & 7) * 4 : lane & 7;
    // The warp's rows of a unit: how many, and row numbers by lane; `run`: they follow
    // one another, as a prompt's do, so that an address is the last one's plus a step.
    struct Rows {
      int id;
      bool run;
    };
    auto rows_in = [&](const Unit& u) { return min(max(u.rows() - 32 * (q & (u.blocks() - 1)), 0), 32); };
    auto rows_of = [&](const Unit& u) {
      return Rows{lane < rows_in(u) ? p.w.rows[u.first + 32 * (q & (u.blocks() - 1)) + lane] : 0, false};
    };
    auto runs = [&](const Unit& u, Rows& r) {
      const int id0 = __shfl_sync(0xffffffffu, r.id, 0);    // by all lanes, whatever they hold
      r.run = __all_sync(0xffffffffu, lane >= rows_in(u) || r.id == id0 + lane);
    };
    // values of two steps
    float y[2][8][4] = {};
    auto load4 = [&](float (&to)[4], const float* from, int col) {
      if constexpr (kVec) {
        if (col < a.N) {
          const float4 t = *reinterpret_cast<const float4*>(from);
          to[0] = t.x, to[1] = t.y, to[2] = t.z, to[3] = t.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + 8 * e < a.N) to[e] = from[8 * e];
      }
    };
    auto load = [&](const Unit& u, const Rows& r, int j, float (&to)[8][4]) {
      const int blocks = u.blocks(), rows = rows_in(u);
      if (a.base == nullptr || j >= blocks) return;
      const int col = u.col0 + 32 * ((q & -blocks) + j) + cl;
      if (r.run) {
        const float* from = a.base + (int64_t)(__shfl_sync(0xffffffffu, r.id, 0) + sub) * a.ldb + col;
#pragma unroll
        for (int v = 0; v < 8; ++v, from += 4 * a.ldb)
          if (4 * v + sub < rows) load4(to[v], from, col);
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int m = __shfl_sync(0xffffffffu, r.id, 4 * v + sub);
          if (4 * v + sub < rows) load4(to[v], a.base + (int64_t)m * a.ldb + col, col);
        }
      }
    };
    Walk<false> walk(p, units, blockIdx.x + group * gridDim.x, kGroups * gridDim.x);
    Unit u = walk.unit();
    Rows ur = rows_of(u);
    runs(u, ur);
    load(u, ur, 0, y[0]);
    load(u, ur, 1, y[1]);
    for (int n = group; u.rows() > 0; n += kGroups) {
      walk.next();                                          // its rows are asked for long before they are needed
      const Unit next = walk.unit();
      Rows nr = rows_of(next);
      const int buf = n % kBuffers;
      const bool sums = u.rank() > 0;
      const int rows = rows_in(u);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], (n / kBuffers) & 1, &abort_flag, a.dev_status))) break;
      tc_fence_after();
      // columns 32 c .. of the unit: the sums and the base values at hand to out
      auto step = [&](int c, const float(&have)[8][4], bool last) {
        if (sums && rows > 0) {
          bool nan = false;
#pragma unroll
          for (int i = 0; i < 32; i += 16) {
            uint32_t r[16];
            tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * kCols + 32 * c + i), r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) nan |= __uint_as_float(r[e]) != __uint_as_float(r[e]);
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(corner + lane * kPitch + i + e) =
                  make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
          if (nan && lane < rows) {
            const int adapter = p.w.tiles[(blockIdx.x + (uint32_t)n * gridDim.x) / (uint32_t)p.col_blocks].x;
            const uint16_t* h = p.w.h + (int64_t)(u.first + 32 * (q & (u.blocks() - 1)) + lane) * 2 * p.rs;
            const __nv_bfloat16* B = a.B + adapter * a.b_slot;
#pragma unroll 1
            for (int i = 0, col = u.col0 + 32 * c; i < 32 && col < a.N; ++i, ++col) {
              float* s = corner + lane * kPitch + i;
              if (*s != *s) *s = sum_of_terms(h, h + p.rs, B + col * a.b_row, u.rank());
            }
          }
        }
        __syncwarp();
        if (last) {
          tc_fence_before();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
        const int col = u.col0 + 32 * c + cl;
        const float* d = corner + sub * kPitch + cl;
        auto store4 = [&](int v, float* to) {
          if constexpr (kVec) {
            float4 s = make_float4(have[v][0], have[v][1], have[v][2], have[v][3]);
            if (sums) {
              const float4 t = *reinterpret_cast<const float4*>(d + 4 * v * kPitch);
              s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
            }
            if (4 * v + sub < rows && col < a.N) *reinterpret_cast<float4*>(to) = s;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (4 * v + sub < rows && col + 8 * e < a.N)
                to[8 * e] = sums ? have[v][e] + d[4 * v * kPitch + 8 * e] : have[v][e];
          }
        };
        if (ur.run) {
          float* to = a.out + (int64_t)(__shfl_sync(0xffffffffu, ur.id, 0) + sub) * a.ldo + col;
#pragma unroll
          for (int v = 0; v < 8; ++v, to += 4 * a.ldo) store4(v, to);
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            store4(v, a.out + (int64_t)__shfl_sync(0xffffffffu, ur.id, 4 * v + sub) * a.ldo + col);
        }
        __syncwarp();
      };
      const int blocks = u.blocks();
      if (blocks == 4) {
        step(0, y[0], false);
        load(u, ur, 2, y[0]);
        step(1, y[1], false);
        load(u, ur, 3, y[1]);
      }
      // the last two steps of this warp, or its only one
      const int c = blocks == 4 ? 2 : q & -blocks;
      step(c, y[0], blocks == 1);
      runs(next, nr);
      load(next, nr, 0, y[0]);
      if (blocks > 1) step(c + 1, y[1], true);
      load(next, nr, 1, y[1]);
      u = next;
      ur = nr;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kBuffers * kCols);
  }
}

cudaError_t launch_inner(const LoraArgs& a, const LoraWork& w, cudaStream_t stream) {
  InnerParams p{};
  p.a = a;
  p.w = w;
  p.rs = lora_rank_stride(a.max_rank);
  const int n16 = (a.max_rank + 15) / 16 * 16;
  p.stage_bytes = kTileBytes16 + (n16 * 128 + 1023) / 1024 * 1024;
  // as many stages as 100 KB hold
  p.stages = std::max(2, std::min(kInnerMaxStages, 100 * 1024 / p.stage_bytes));
  p.tmem_cols = 32;
  while ((int)p.tmem_cols < n16) p.tmem_cols *= 2;
  // blocks of a tile: those of the tiles that the rows fill are on the GPU at once
  const int64_t filled = (a.M + kLoraTile - 1) / kLoraTile;
  const int chunks = (a.K + kChunk - 1) / kChunk, fit = 2 * attn_sm_count();
  p.cluster = kLoraMaxCluster;
  while (p.cluster > 1 && (filled * p.cluster > fit || 2 * p.cluster > chunks)) p.cluster /= 2;
  const int64_t most = lora_max_tiles(a.M, a.n_adapters);
  const int clusters = (int)std::min<int64_t>(most, std::max(1, fit / p.cluster));
  const size_t smem = std::max(kInnerLeast, 1024 + p.stages * p.stage_bytes);
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = set_once(done, reinterpret_cast<const void*>(lora_inner_kernel),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kInnerMost);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * p.cluster));
  cfg.blockDim = dim3(kInnerThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, lora_inner_kernel, p);
}

template <bool kVec>
cudaError_t launch_outer(const CUtensorMap& tmH, const CUtensorMap& tmH32, const CUtensorMap& tmB,
                         const OuterParams& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = set_once(done, reinterpret_cast<const void*>(lora_outer_kernel<kVec>),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kOuterSmem);
  if (err != cudaSuccess) return err;
  return launch_pdl(lora_outer_kernel<kVec>, dim3((unsigned)grid), dim3(kOuterThreads), kOuterSmem, stream, tmH,
                    tmH32, tmB, p);
}

}  // namespace

cudaError_t launch_lora_products(const LoraArgs& a, const LoraWork& w, bool copy_none, cudaStream_t stream) {
  OuterParams p{a, w, lora_rank_stride(a.max_rank), (a.N + kCols - 1) / kCols, copy_none};
  CUtensorMap tmH, tmH32, tmB;
  if (!make_tmap_2d(&tmH, true, w.h, (uint64_t)2 * p.rs, (uint64_t)a.M, (uint64_t)4 * p.rs, kChunk, 128) ||
      !make_tmap_2d(&tmH32, true, w.h, (uint64_t)2 * p.rs, (uint64_t)a.M, (uint64_t)4 * p.rs, kChunk, 32) ||
      !make_tmap_rows3(&tmB, a.B, (uint64_t)a.max_rank, (uint64_t)a.N, (uint64_t)a.n_adapters, (uint64_t)a.b_row * 2,
                       (uint64_t)a.b_slot * 2, kChunk, kCols))
    return cudaErrorInvalidValue;
  const cudaError_t err = launch_inner(a, w, stream);
  if (err != cudaSuccess) return err;
  // a block per SM: how many units there are only the device knows
  const int grid = (int)std::min<int64_t>(lora_max_tiles(a.M, a.n_adapters) * p.col_blocks, attn_sm_count());
  const bool vec = a.N % 4 == 0 && aligned(a.out, 16) && a.ldo % 4 == 0 &&
                   (a.base == nullptr || (aligned(a.base, 16) && a.ldb % 4 == 0));
  return vec ? launch_outer<true>(tmH, tmH32, tmB, p, grid, stream)
             : launch_outer<false>(tmH, tmH32, tmB, p, grid, stream);
}

}  // namespace qmm

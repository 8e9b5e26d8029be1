// The second product of the adapters in calls of many rows, on tcgen05:
//     out[m] = base[m] + h_m B_a^T,   h_m = s_a A_a x_m as two bf16 terms.
//
// Bound: bytes, 8 a value of out (base in, out back); the two terms' products are 4 r
// operations per 8 bytes, which mma.sync (600 TFLOP/s measured on this part) could
// not hide from ranks of about 100 on.
//
// A block takes 128 rows of one adapter and 128 columns.  Its base values are on
// their way into registers, in whole rows of 512 bytes, before anything else;
// meanwhile the terms of h and the rows of B arrive by TMA, 64 ranks at a time, and
// one thread issues the products of both terms with the same B.  The accumulator
// goes from tensor memory through shared memory, so that sums are stored in whole
// rows again.  Two blocks share an SM: one loads while the other stores.
#include <algorithm>
#include <atomic>

#include "kv_cache.h"
#include "lora_work.cuh"
#include "umma.cuh"

namespace qmm {
namespace {

using namespace umma;

constexpr int kThreads = 256;
constexpr int kCols = 128;
constexpr int kChunk = 64;                                  // ranks of a stage: 128 bytes, one swizzle row
constexpr int kTileBytes16 = 128 * kChunk * 2;
constexpr int kStageBytes = 3 * kTileBytes16;               // both terms of h, B
constexpr int kMaxChunks = (int)kLoraMaxRank / kChunk;
constexpr int kPitch = kCols + 4;                           // floats of a row of the accumulator in shared memory
constexpr int kOutBytes = 128 * kPitch * 4;
constexpr uint32_t kTmemCols = kCols;

struct OuterParams {
  LoraArgs a;
  LoraWork w;
  int rs, stages, col_blocks;
  bool copy_none;
};

template <bool kVec>
__global__ void __launch_bounds__(kThreads, 2)
lora_outer_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmB,
                  const OuterParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxChunks], done[2], last;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = smem_align(smem_raw, 1024);
  const LoraArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int c = 0; c < kMaxChunks; ++c) mbar_init(&full[c], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&done[s], 1);
    mbar_init(&last, 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmH);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  // parities of the barriers' next phases: a bit per chunk, per stage, and one
  uint32_t full_par = 0, done_par = 0, last_par = 0;
  const int64_t units = (int64_t)p.w.head[p.copy_none ? 1 : 0] * p.col_blocks;

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int4 it = p.w.tiles[unit / p.col_blocks];
    const int col0 = (int)(unit % p.col_blocks) * kCols;
    const bool none = it.x < 0;
    const int rank = none ? 0 : a.ranks != nullptr ? a.ranks[it.x] : a.max_rank;
    const int chunks = (rank + kChunk - 1) / kChunk;
    auto issue = [&](int c) {
      uint8_t* s = smem + c % p.stages * kStageBytes;
      mbar_arrive_expect_tx(&full[c], kStageBytes);
      tma_load_2d(s, &tmH, &full[c], c * kChunk, it.y);
      tma_load_2d(s + kTileBytes16, &tmH, &full[c], p.rs + c * kChunk, it.y);
      tma_load_3d(smem_u32(s + 2 * kTileBytes16), &tmB, &full[c], c * kChunk, col0, it.x);
    };
    if (tid == 0) {
      fence_proxy_async_smem();   // the last unit's reads of the accumulator precede the copies
      for (int c = 0; c < min(chunks, p.stages); ++c) issue(c);
    }

    // base, a whole row of the block's columns per warp and load
    const int my_row = warp * 16 + (lane & 15);
    const int row_id = my_row < it.z ? p.w.rows[it.y + my_row] : 0;
    auto col = [&](int i) { return kVec ? col0 + lane * 4 + i : col0 + lane + 32 * i; };   // of value i
    float y[16][4];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t m = __shfl_sync(0xffffffffu, row_id, r);
      const float* from = a.base + m * a.ldb;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[r][i] = 0.f;
      if (a.base == nullptr || warp * 16 + r >= it.z) continue;
      if constexpr (kVec) {
        if (col(0) < a.N) {
          const float4 v = *reinterpret_cast<const float4*>(from + col(0));
          y[r][0] = v.x, y[r][1] = v.y, y[r][2] = v.z, y[r][3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col(i) < a.N) y[r][i] = from[col(i)];
      }
    }

    float* acc = reinterpret_cast<float*>(smem);   // [128][kPitch], where the operands lay
    if (!none) {
      constexpr uint32_t idesc = idesc_f16(128, kCols, true);
      auto products = [&](int c) {
        const uint32_t s = smem_u32(smem + c % p.stages * kStageBytes);
        const int steps = min(kChunk / 16, (rank - c * kChunk + 15) / 16);
        const uint64_t b = desc_kmajor_sw128(s + 2 * kTileBytes16);
        for (int term = 1; term >= 0; --term) {    // the smaller one first
          const uint64_t h = desc_kmajor_sw128(s + term * kTileBytes16);
          for (int k = 0; k < steps; ++k)
            umma_f16(tmem, h + 2 * k, b + 2 * k, idesc, c > 0 || term == 0 || k > 0);
        }
      };
      bool ok = true;
      if (tid == 0) {
        for (int c = 0; c + 1 < chunks && ok; ++c) {
          ok = mbar_wait(&full[c], full_par >> c & 1, &abort_flag, a.dev_status);
          if (!ok) break;
          tc_fence_after();
          products(c);
          if (c + p.stages < chunks) {
            const int s = c % p.stages;
            umma_commit(&done[s]);
            ok = mbar_wait(&done[s], done_par >> s & 1, &abort_flag, a.dev_status);
            done_par ^= 1u << s;
            if (ok) issue(c + p.stages);
          }
        }
      }
      const int c = chunks - 1, rem = rank - c * kChunk;
      ok = ok && mbar_wait(&full[c], full_par >> c & 1, &abort_flag, a.dev_status);
      if (rem % 16 != 0 && rank < a.max_rank) {
        // what lies behind the adapter's rank in the last step of 16: zeros, since 0
        // times an infinity or NaN is none (h is zero there)
        if (ok && tid < kCols) {
          uint8_t* row = smem + c % p.stages * kStageBytes + 2 * kTileBytes16 + tid * 128;
          const int piece = rem / 8;
          uint4* at = reinterpret_cast<uint4*>(row + ((piece ^ (tid & 7)) << 4));
          uint32_t w[4] = {at->x, at->y, at->z, at->w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = rem % 8 - 2 * i;         // values of this word that stay
            if (n <= 0) w[i] = 0;
            else if (n == 1) w[i] &= 0xFFFFu;
          }
          *at = make_uint4(w[0], w[1], w[2], w[3]);
          if (piece % 2 == 0)
            *reinterpret_cast<uint4*>(row + (((piece + 1) ^ (tid & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncthreads();
      }
      if (tid == 0 && ok) {
        tc_fence_after();
        products(c);
        umma_commit(&last);
      }
      ok = ok && mbar_wait(&last, last_par, &abort_flag, a.dev_status);
      if (__syncthreads_or(!ok)) {
        // copies already issued land before the block leaves
        if (tid == 0)
          for (int i = 0; i < chunks; ++i) mbar_drain(&full[i], full_par >> i & 1);
        break;
      }
      full_par ^= (1u << chunks) - 1;
      last_par ^= 1;
      tc_fence_after();
      const int q = warp & 3, half = warp >> 2;
      if (32 * q < it.z) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t r[32];
          tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * 64 + 32 * j), r);
          tmem_wait_ld();
          float* to = acc + (32 * q + lane) * kPitch + half * 64 + 32 * j;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(to + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t m = __shfl_sync(0xffffffffu, row_id, r);
      if (warp * 16 + r >= it.z) continue;
      float* to = a.out + m * a.ldo;
      const float* v = acc + (warp * 16 + r) * kPitch - col0;
      if constexpr (kVec) {
        if (col(0) < a.N) {
          float4 s = make_float4(y[r][0], y[r][1], y[r][2], y[r][3]);
          if (!none) {
            const float4 d = *reinterpret_cast<const float4*>(v + col(0));
            s.x += d.x, s.y += d.y, s.z += d.z, s.w += d.w;
          }
          *reinterpret_cast<float4*>(to + col(0)) = s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col(i) < a.N) to[col(i)] = none ? y[r][i] : y[r][i] + v[col(i)];
      }
    }
    __syncthreads();   // the accumulator has been read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool kVec>
cudaError_t launch_typed(const CUtensorMap& tmH, const CUtensorMap& tmB, const OuterParams& p, int grid,
                         cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const size_t smem = 1024 + (size_t)std::max(kOutBytes, p.stages * kStageBytes);
  const cudaError_t err = set_once(done, reinterpret_cast<const void*>(lora_outer_kernel<kVec>),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   1024 + std::max(kOutBytes, 2 * kStageBytes));
  if (err != cudaSuccess) return err;
  return launch_pdl(lora_outer_kernel<kVec>, dim3((unsigned)grid), dim3(kThreads), smem, stream, tmH,
                    tmB, p);
}

}  // namespace

cudaError_t launch_lora_outer(const LoraArgs& a, const LoraWork& w, bool copy_none, cudaStream_t stream) {
  OuterParams p{a, w, lora_rank_stride(a.max_rank), a.max_rank > kChunk ? 2 : 1, (a.N + kCols - 1) / kCols, copy_none};
  CUtensorMap tmH, tmB;
  if (!make_tmap_2d(&tmH, true, w.h, (uint64_t)2 * p.rs, (uint64_t)a.M, (uint64_t)4 * p.rs, kChunk, 128) ||
      !make_tmap_rows3(&tmB, a.B, (uint64_t)a.max_rank, (uint64_t)a.N, (uint64_t)a.n_adapters, (uint64_t)a.b_row * 2,
                       (uint64_t)a.b_slot * 2, kChunk, kCols))
    return cudaErrorInvalidValue;
  // two blocks per SM walk over the units: how many tiles there are only the device knows
  const int grid = (int)std::min<int64_t>(lora_max_tiles(a.M, a.n_adapters) * p.col_blocks, 2 * attn_sm_count());
  const bool vec = a.N % 4 == 0 && aligned(a.out, 16) && a.ldo % 4 == 0 &&
                   (a.base == nullptr || (aligned(a.base, 16) && a.ldb % 4 == 0));
  return vec ? launch_typed<true>(tmH, tmB, p, grid, stream) : launch_typed<false>(tmH, tmB, p, grid, stream);
}

}  // namespace qmm

// New key and value rows into the paged cache: token t's rows go to slot
// slots[t] (page slot / P, place slot % P), as bf16 (one rounding to nearest
// even) or as int8 codes with a scale per (token, head), by packB's rule:
//     s = fl(amax / 127);  q = clamp(rint_even(fl(x / s)), -127, 127), 0 where s == 0.
//
// One warp per (token, head): it has the whole row of K and of V in registers
// (one vector load each), so that the maximum is a warp reduction and every
// byte is read and written once.  Bound by HBM; the loads do not depend on the
// slot, only the stores do.
#include <cuda_bf16.h>

#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kAppendThreads = 256;

// kN consecutive values of a lane: kN = head_dim / 32 (2 or 4).
template <bool kBf16, int kN>
__device__ __forceinline__ void load_row(const uint8_t* row, int lane, float (&x)[kN]) {
  if constexpr (kBf16) {
    uint32_t w[kN / 2];
    if constexpr (kN == 4) {
      const uint2 v = reinterpret_cast<const uint2*>(row)[lane];
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = reinterpret_cast<const uint32_t*>(row)[lane];
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) x[2 * i] = bf16lo_to_f32(w[i]), x[2 * i + 1] = bf16hi_to_f32(w[i]);
  } else if constexpr (kN == 4) {
    const float4 v = reinterpret_cast<const float4*>(row)[lane];
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = reinterpret_cast<const float2*>(row)[lane];
    x[0] = v.x, x[1] = v.y;
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <bool kS8, int kN>
__device__ __forceinline__ void store_row(uint8_t* row, float* scale, int lane, const float (&x)[kN]) {
  if constexpr (!kS8) {
    if constexpr (kN == 4) {
      reinterpret_cast<uint2*>(row)[lane] = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
    } else {
      reinterpret_cast<uint32_t*>(row)[lane] = bf16x2(x[0], x[1]);
    }
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = __fdiv_rn(m, 127.0f);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      int q = 0;
      if (s > 0.f) q = min(max(__float2int_rn(__fdiv_rn(x[i], s)), -127), 127);
      w |= ((uint32_t)q & 0xFFu) << (8 * i);
    }
    if constexpr (kN == 4) reinterpret_cast<uint32_t*>(row)[lane] = w;
    else reinterpret_cast<uint16_t*>(row)[lane] = (uint16_t)w;
    if (lane == 0) *scale = s;
  }
}

template <bool kBf16, bool kS8, int kN>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const KvAppendArgs a) {
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.T * a.cache.n_heads) return;
  const int t = (int)(row / a.cache.n_heads), h = (int)(row % a.cache.n_heads);
  const int64_t slot = a.slots[t];
  float k[kN], v[kN];
  load_row<kBf16, kN>(a.k + t * a.k_st + h * a.k_sh, lane, k);
  load_row<kBf16, kN>(a.v + t * a.v_st + h * a.v_sh, lane, v);
  const uint32_t P = a.cache.page_size;
  if (slot < 0 || slot >= a.cache.n_pages * (int64_t)P) {   // -1 marks a token that is not stored
    if (slot != -1 && lane == 0) set_status(a.dev_status, QMM_ERR_INVALID_ARG);
    return;
  }
  int64_t page, off;
  if (slot <= UINT32_MAX) {   // nearly always: the 32-bit division is several times shorter
    page = (uint32_t)slot / P;
    off = (uint32_t)slot % P;
  } else {
    page = slot / P;
    off = slot % P;
  }
  const int64_t at = page * a.cache.st_page + off * a.cache.st_token + h * a.cache.st_head;
  const int64_t sc = (page * a.cache.n_heads + h) * P + off;
  store_row<kS8, kN>(a.cache.k + at, a.cache.k_scale + sc, lane, k);
  store_row<kS8, kN>(a.cache.v + at, a.cache.v_scale + sc, lane, v);
}

template <bool kBf16, bool kS8>
cudaError_t launch_typed(const KvAppendArgs& a, int head_dim, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * a.cache.n_heads;
  const dim3 grid((unsigned)((rows + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
  return head_dim == 128 ? launch_pdl(kv_append_kernel<kBf16, kS8, 4>, grid, dim3(kAppendThreads), 0, stream, a)
                         : launch_pdl(kv_append_kernel<kBf16, kS8, 2>, grid, dim3(kAppendThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool rows_bf16, bool cache_s8, int head_dim,
                             cudaStream_t stream) {
  if (rows_bf16)
    return cache_s8 ? launch_typed<true, true>(a, head_dim, stream) : launch_typed<true, false>(a, head_dim, stream);
  return cache_s8 ? launch_typed<false, true>(a, head_dim, stream) : launch_typed<false, false>(a, head_dim, stream);
}

}  // namespace qmm

// New key and value rows into the paged cache: token t's rows go to slot
// slots[t] (page slot / P, place slot % P), as bf16 (one rounding to nearest
// even) or as int8 codes with a scale per (token, head), by packB's rule:
//     s = fl(amax / 127);  q = clamp(rint_even(fl(x / s)), -127, 127), 0 where s == 0.
//
// A warp takes a (token, head) pair: its key row in lanes 0..15, its value row in
// lanes 16..31, in registers as a whole, so that the maximum is a reduction over
// 16 lanes and every byte is read and written once, 16 bytes per lane and load.
// With many pairs a warp takes kPer that follow one another, has all their loads
// in flight and works out a token's place once.  Into bf16 bound by HBM: 16384
// tokens of 8 heads x 128 in fp32 29.7 us (201 MB, 1.0 of a copy's rate, over buffers
// of 1 GB in turn: half of a call's writes leave the L2 during the next), in bf16
// 21.5 (0.92).  Into int8 by issue slots: about 230 instructions per pair, 8191
// tokens in bf16 20.7 us (0.36 of a copy's rate; with a division per value and a
// warp per pair 26.0), 16384 in fp32 36.0 (0.69).  A few tokens cost a launch and
// two dependent loads, 1.4 us.
#include <cuda_bf16.h>

#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

constexpr int kAppendThreads = 256;

// kN consecutive values of a lane: kN = head_dim / 16 (4 or 8).
template <bool kBf16, int kN>
struct LaneRow {
  static constexpr int kWords = kBf16 ? kN / 2 : kN;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const uint8_t* row, int l) {
    if constexpr (kWords == 2) {
      const uint2 v = reinterpret_cast<const uint2*>(row)[l];
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(row)[l * (kWords / 4) + i / 4];
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kBf16) return (i & 1) ? bf16hi_to_f32(w[i >> 1]) : bf16lo_to_f32(w[i >> 1]);
    else return __uint_as_float(w[i]);
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <bool kBf16, bool kS8, int kN>
__device__ __forceinline__ void store_row(uint8_t* row, float* scale, int l, const LaneRow<kBf16, kN>& x) {
  if constexpr (!kS8) {
    uint32_t p[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) p[i] = kBf16 ? x.w[i] : bf16x2(x.at(2 * i), x.at(2 * i + 1));
    if constexpr (kN == 8) reinterpret_cast<uint4*>(row)[l] = make_uint4(p[0], p[1], p[2], p[3]);
    else reinterpret_cast<uint2*>(row)[l] = make_uint2(p[0], p[1]);
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, fabsf(x.at(i)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = __fdiv_rn(m, 127.0f);
    // rint(fl(x / s)) without a division: y = fl(x * fl(1 / s)) is within 2^-23 |y| +
    // 2^-24 |y| < 2.3e-5 of fl(x / s) (|y| <= 128, 1 / s neither overflowing nor
    // subnormal), so both round to the same integer unless y is that close to a
    // half.  Adding 1.5 * 2^23 rounds to the nearest even integer and leaves it in
    // the low bits.  Rows with a value near a half, and scales out of range, divide.
    const float r = __frcp_rn(s);
    uint32_t q[kN];
    bool divide = !(s > 0x1p-100f && s < 0x1p100f);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float y = __fmul_rn(x.at(i), r), t = __fadd_rn(y, 12582912.f);
      divide |= fabsf(y - __fsub_rn(t, 12582912.f)) > 0.4999f;
      q[i] = __float_as_uint(t);
    }
    if (divide) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        q[i] = s > 0.f ? (uint32_t)min(max(__float2int_rn(__fdiv_rn(x.at(i), s)), -127), 127) : 0u;
    }
    const uint32_t lo = pack_bytes(q[0], q[1], q[2], q[3]);
    if constexpr (kN == 8) reinterpret_cast<uint2*>(row)[l] = make_uint2(lo, pack_bytes(q[4], q[5], q[6], q[7]));
    else reinterpret_cast<uint32_t*>(row)[l] = lo;
    if (l == 0) *scale = s;
  }
}

template <bool kBf16, bool kS8, int kN, int kPer>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const KvAppendArgs a) {
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool value = lane >= 16;
  const int64_t rows = (int64_t)a.T * a.cache.n_heads;
  const int64_t first = ((int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5)) * kPer;
  if (first >= rows) return;
  const uint8_t* src = value ? a.v : a.k;
  const int64_t st = value ? a.v_st : a.k_st, sh = value ? a.v_sh : a.k_sh;
  uint8_t* dst = value ? a.cache.v : a.cache.k;
  float* scales = value ? a.cache.v_scale : a.cache.k_scale;
  const uint32_t heads = a.cache.n_heads, P = a.cache.page_size;
  // 32-bit divisions nearly always: several times shorter
  const int64_t t0 = first <= UINT32_MAX ? (uint32_t)first / heads : first / heads;
  const uint32_t h0 = (uint32_t)(first - t0 * heads);
  // the pairs' heads follow one another, and after the last head the next token's
  LaneRow<kBf16, kN> x[kPer];
  int64_t slot[kPer];                            // the token's, at its first pair; else -1
  const uint8_t* from = src + t0 * st + h0 * sh;
  const int64_t* at_slot = a.slots + t0;
  uint32_t h = h0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    slot[i] = -1;
    if (i == 0 || first + i < rows) {
      if (i == 0 || h == 0) slot[i] = *at_slot;
      x[i].load(from, l);
    }
    from += sh;
    if (++h == heads) h = 0, ++at_slot, from += st - heads * sh;
  }
  h = h0;
  uint8_t* to = nullptr;
  float* scale = nullptr;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i == 0 || h == 0) {                      // a token's first pair here
      to = nullptr;
      if (slot[i] >= 0 && slot[i] < a.cache.n_pages * (int64_t)P) {
        const int64_t page = slot[i] <= UINT32_MAX ? (uint32_t)slot[i] / P : slot[i] / P, off = slot[i] - page * P;
        to = dst + page * a.cache.st_page + off * a.cache.st_token + h * a.cache.st_head;
        if constexpr (kS8) scale = scales + (page * heads + h) * P + off;
      } else if (slot[i] != -1 && lane == 0) {   // -1 marks a token that is not stored
        set_status(a.dev_status, QMM_ERR_INVALID_ARG);
      }
    }
    if (to != nullptr && (i == 0 || first + i < rows)) {
      store_row<kBf16, kS8, kN>(to, scale, l, x[i]);
      to += a.cache.st_head;
      if constexpr (kS8) scale += P;
    }
    if (++h == heads) h = 0;
  }
}

// Pairs per warp: kMany once there are enough to fill the GPU's warps all the
// same (4000 tokens x 8 heads, fp32 to bf16: two pairs 9.2 us, one 10.1; from 8191
// tokens on four pairs are as fast as two, and 4000 would be below their limit).
constexpr int kMany = 2;
int64_t many_from() { return (int64_t)attn_sm_count() * 64 * kMany; }   // 64 warps per SM

template <bool kBf16, bool kS8, int kN>
cudaError_t launch_sized(const KvAppendArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * a.cache.n_heads;
  const bool many = rows >= many_from();
  const int64_t per_block = kAppendThreads / 32 * (many ? kMany : 1);
  const dim3 grid((unsigned)((rows + per_block - 1) / per_block));
  return many ? launch_pdl(kv_append_kernel<kBf16, kS8, kN, kMany>, grid, dim3(kAppendThreads), 0, stream, a)
              : launch_pdl(kv_append_kernel<kBf16, kS8, kN, 1>, grid, dim3(kAppendThreads), 0, stream, a);
}

template <bool kBf16, bool kS8>
cudaError_t launch_typed(const KvAppendArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch_sized<kBf16, kS8, 8>(a, stream) : launch_sized<kBf16, kS8, 4>(a, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool rows_bf16, bool cache_s8, int head_dim,
                             cudaStream_t stream) {
  if (rows_bf16)
    return cache_s8 ? launch_typed<true, true>(a, head_dim, stream) : launch_typed<true, false>(a, head_dim, stream);
  return cache_s8 ? launch_typed<false, true>(a, head_dim, stream) : launch_typed<false, false>(a, head_dim, stream);
}

}  // namespace qmm

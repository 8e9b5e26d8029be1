// What the adapter kernels share: the rows by adapter, and h as it lies between the
// two products of a routed call.
#pragma once

#include "beside.h"
#include "umma.cuh"

namespace qmm {

constexpr int kLoraTile = 128;            // rows of a routed item, all of one adapter

struct LoraWork {
  int* head;      // [0]: tiles of rows with an adapter, [1]: all tiles
  int4* tiles;    // adapter (-1: none), first place in rows, rows
  int* rows;      // [M] row numbers by adapter
  uint16_t* h;    // [M][2][rank_stride] bf16 by place in rows: s_a A_a x_m as two terms
};

inline int lora_rank_stride(int64_t max_rank) { return (int)((max_rank + 63) / 64 * 64); }
inline int64_t lora_max_tiles(int64_t M, int64_t n_adapters) {
  return M / kLoraTile + (n_adapters + 1 < M ? n_adapters + 1 : M);
}

constexpr int kLoraMaxCluster = 8;
// The sums over a cluster's blocks, in order, of the four floats at each of kN places
// of their shared memory, zeros where `in` is not set; all loads under way before the
// first addition.
template <int kN>
QMM_DEV void cluster_sums(const uint32_t (&addr)[kN], const bool (&in)[kN], int cluster, float4 (&s)[kN]) {
  float4 v[kN][kLoraMaxCluster];
#pragma unroll
  for (int o = 0; o < kLoraMaxCluster; ++o)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i][o] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (o < cluster && in[i])
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[i][o].x), "=f"(v[i][o].y), "=f"(v[i][o].z), "=f"(v[i][o].w)
                     : "r"(umma::mapa_shared(addr[i], o))
                     : "memory");
    }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    s[i] = v[i][0];
#pragma unroll
    for (int o = 1; o < kLoraMaxCluster; ++o)
      if (o < cluster) s[i].x += v[i][o].x, s[i].y += v[i][o].y, s[i].z += v[i][o].z, s[i].w += v[i][o].w;
  }
}
QMM_DEV float4 cluster_sum(uint32_t addr, int cluster) {
  const uint32_t at[1] = {addr};
  const bool in[1] = {true};
  float4 s[1];
  cluster_sums(at, in, cluster, s);
  return s[0];
}

// h as the two bf16 terms that the second product takes, four ranks at a time: the
// value rounded, and what that left.  A finite value does not round to infinity, which 0 in
// B would make NaN of; an infinity leaves nothing, since infinity less infinity is NaN.
QMM_DEV uint32_t two_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
QMM_DEV float below_inf(float x) {
  constexpr float kMost = 0x1.FEp127f;   // of bf16
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -kMost), kMost) : x;
}
QMM_DEV float left_of(float x, float rounded) {
  const float d = x - rounded;
  return fabsf(d) < INFINITY ? d : 0.f;
}
QMM_DEV void put_terms(uint16_t* hi, uint16_t* lo, const float4& s) {
  const uint32_t a = two_bf16(below_inf(s.x), below_inf(s.y)), b = two_bf16(below_inf(s.z), below_inf(s.w));
  *reinterpret_cast<uint2*>(hi) = make_uint2(a, b);
  *reinterpret_cast<uint2*>(lo) =
      make_uint2(two_bf16(left_of(s.x, bf16lo_to_f32(a)), left_of(s.y, bf16hi_to_f32(a))),
                 two_bf16(left_of(s.z, bf16lo_to_f32(b)), left_of(s.w, bf16hi_to_f32(b))));
}

// A row's sum over the ranks for one column, value by value, where the products gave NaN: an
// infinity in B times h's two terms can be infinities of both signs, or 0 times infinity
// for one of them, while it is an infinity times their sum.
QMM_DEV float sum_of_terms(const uint16_t* hi, const uint16_t* lo, const __nv_bfloat16* b, int rank) {
  float s = 0.f;
#pragma unroll 1
  for (int j = 0; j < rank && s == s; ++j)
    s = fmaf(bf16lo_to_f32(hi[j]) + bf16lo_to_f32(lo[j]), __bfloat162float(b[j]), s);
  return s;
}

// both products of a routed call (lora_umma.cu)
cudaError_t launch_lora_products(const LoraArgs& a, const LoraWork& w, bool copy_none, cudaStream_t stream);

}  // namespace qmm

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
// The sum over a cluster's blocks, in order, of the four floats at one place of
// their shared memory; all loads under way before the first addition.
QMM_DEV float4 cluster_sum(uint32_t addr, int cluster) {
  float4 v[kLoraMaxCluster];
#pragma unroll
  for (int o = 0; o < kLoraMaxCluster; ++o) {
    v[o] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (o < cluster)
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v[o].x), "=f"(v[o].y), "=f"(v[o].z), "=f"(v[o].w)
                   : "r"(umma::mapa_shared(addr, o))
                   : "memory");
  }
  float4 s = v[0];
#pragma unroll
  for (int o = 1; o < kLoraMaxCluster; ++o)
    if (o < cluster) s.x += v[o].x, s.y += v[o].y, s.z += v[o].z, s.w += v[o].w;
  return s;
}

// both products of a routed call (lora_umma.cu)
cudaError_t launch_lora_products(const LoraArgs& a, const LoraWork& w, bool copy_none, cudaStream_t stream);

}  // namespace qmm

// A block's output joined to the residual stream, and the next block's input:
//     u = branch_norm(branch);  sum = residual + scale * gate * u;  out = norm(sum)
//     rms:   v * w / sqrt(mean(v^2) + eps) + b
//     layer: (v - mean) * w / sqrt(mean((v - mean)^2) + eps) + b
// and int8 codes of out by the activation quantiser's rule (s = fl(amax / 127)).
//
// Bound: bytes.  Each value of residual, branch and gate is read once and each
// of sum and out written once; a row stays in its block's registers from the
// first load to the last store, through up to five reductions (two means, two
// squares, one maximum), so that nothing is read again.
#include <algorithm>

#include "beside.h"

namespace qmm {
namespace {

// Read once, and possibly written later by the same thread (sum may be the
// residual itself): a coherent load that leaves L1 to the weights.
QMM_DEV uint4 ld128_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Eight values of a row as they lie in memory.
template <bool kBf16>
struct Raw8 {
  uint4 q[kBf16 ? 1 : 2];
};
template <bool kBf16>
QMM_DEV Raw8<kBf16> load8(const void* base, int64_t elem) {
  Raw8<kBf16> r;
  const uint8_t* p = static_cast<const uint8_t*>(base) + elem * (kBf16 ? 2 : 4);
  r.q[0] = ld128_once(p);
  if constexpr (!kBf16) r.q[1] = ld128_once(p + 16);
  return r;
}
template <bool kBf16>
QMM_DEV float value8(const Raw8<kBf16>& r, int i) {
  if constexpr (kBf16) {
    const uint32_t w = u4_get(r.q[0], i / 2);
    return i & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
  } else {
    return __uint_as_float(u4_get(r.q[i / 4], i % 4));
  }
}

QMM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Where a thread's values lie: kVec: groups of eight (group threadIdx.x + g *
// blockDim.x), else single values (threadIdx.x + i * blockDim.x).
template <bool kVec>
QMM_DEV int place(int i) {
  return kVec ? ((int)threadIdx.x + (i / 8) * (int)blockDim.x) * 8 + i % 8 : (int)threadIdx.x + i * (int)blockDim.x;
}

// Sum (or maximum) over a row's threads; every thread gets the result.  One
// barrier: each reduction of a row has its own slot.
template <bool kMax>
QMM_DEV float row_reduce(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, w) : v + w;
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? slot[lane] : 0.f;   // maxima are of magnitudes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, w) : v + w;
  }
  return v;
}

// Eight (or single) fp32 values of a weight row that all blocks read: cached.
template <bool kVec, int kE>
QMM_DEV void load_row(const float* p, int D, float (&w)[kE]) {
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kE; i += 4)
      if (place<kVec>(i) < D) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p + place<kVec>(i)));
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (place<kVec>(i) < D) w[i] = __ldg(p + place<kVec>(i));
  }
}

template <bool kVec, int kE>
QMM_DEV void apply_norm(const NormSpec& n, int D, float (&v)[kE], float (*slots)[32]) {
  if (n.kind == QMM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) s += v[i];   // values past D are zeros
    const float mean = row_reduce<false>(s, slots[0]) / (float)D;
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] = place<kVec>(i) < D ? v[i] - mean : 0.f;
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) ss = fmaf(v[i], v[i], ss);
  const float inv = rsqrtf(row_reduce<false>(ss, slots[1]) / (float)D + n.eps);
  if (n.weight != nullptr) {
    float w[kE];
    load_row<kVec>(n.weight, D, w);
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (place<kVec>(i) < D) v[i] = v[i] * inv * w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) v[i] *= inv;
  }
  if (n.bias != nullptr) {
    float w[kE];
    load_row<kVec>(n.bias, D, w);
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (place<kVec>(i) < D) v[i] += w[i];
  }
}

// A row's values of one tensor, zeros past D.
template <bool kVec, bool kBf16, int kE>
struct RowLoad {
  Raw8<kBf16> raw[kVec ? kE / 8 : 1];
  float one[kVec ? 1 : kE];
  QMM_DEV void issue(const void* base, int64_t row, int D) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kE; i += 8) {
        raw[i / 8] = {};
        if (place<kVec>(i) < D) raw[i / 8] = load8<kBf16>(base, row + place<kVec>(i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        one[i] = 0.f;
        const int64_t at = row + place<kVec>(i);
        if (place<kVec>(i) < D)
          one[i] = kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at])
                         : static_cast<const float*>(base)[at];
      }
    }
  }
  QMM_DEV float at(int i) const {
    if constexpr (kVec) return value8<kBf16>(raw[i / 8], i % 8);
    return one[i];
  }
};

template <bool kVec, int kE>
QMM_DEV void store_row(void* base, bool bf16, int64_t row, int D, const float (&v)[kE]) {
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kE; i += 8) {
      if (place<kVec>(i) >= D) continue;
      const int64_t at = row + place<kVec>(i);
      if (bf16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
            make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]), pack_bf16(v[i + 4], v[i + 5]),
                       pack_bf16(v[i + 6], v[i + 7]));
      } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        p[0] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        p[1] = make_float4(v[i + 4], v[i + 5], v[i + 6], v[i + 7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if (place<kVec>(i) >= D) continue;
      const int64_t at = row + place<kVec>(i);
      if (bf16) static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v[i]);
      else static_cast<float*>(base)[at] = v[i];
    }
  }
}

// kE values of a row per thread; blockDim.y rows per block (more than one only
// where a row has one warp, which needs no barrier).
template <bool kVec, int kE, bool kResBf16, bool kBrBf16>
__global__ void __launch_bounds__(1024)
block_norm_kernel(NormArgs a) {
  __shared__ float slots[5][32];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;   // whole warps, and only where no barrier follows
  const int D = a.D;
  float v[kE];
  {
    RowLoad<kVec, kResBf16, kE> res;
    res.issue(a.residual, t * a.ldr, D);
    if (a.branch != nullptr) {
      RowLoad<kVec, kBrBf16, kE> br;
      br.issue(a.branch, t * a.ldb, D);
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = br.at(i);
      if (a.post.kind != 0) apply_norm<kVec>(a.post, D, v, slots);
      if (a.gate != nullptr) {
        if (a.gate_bf16) {
          RowLoad<kVec, true, kE> g;
          g.issue(a.gate, t * a.ldg, D);
#pragma unroll
          for (int i = 0; i < kE; ++i) v[i] *= g.at(i);
        } else {
          RowLoad<kVec, false, kE> g;
          g.issue(a.gate, t * a.ldg, D);
#pragma unroll
          for (int i = 0; i < kE; ++i) v[i] *= g.at(i);
        }
      }
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = place<kVec>(i) < D ? fmaf(a.scale, v[i], res.at(i)) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = res.at(i);
    }
  }
  if (a.sum != nullptr) store_row<kVec>(a.sum, kResBf16, t * a.lds, D, v);
  if (a.out == nullptr) return;
  if (a.pre.kind != 0) apply_norm<kVec>(a.pre, D, v, slots + 2);
  if (a.out_type != QMM_S8) {
    store_row<kVec>(a.out, a.out_type == QMM_BF16, t * a.ldo, D, v);
    return;
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i)
    if (place<kVec>(i) < D) amax = fmaxf(amax, fabsf(v[i]));
  const float s = __fdiv_rn(row_reduce<true>(amax, slots[4]), 127.0f);
  if (threadIdx.x == 0) a.s_x[t] = s;
  int8_t* codes = static_cast<int8_t*>(a.out) + t * a.ldo;
  uint32_t q[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i)
    q[i] = s > 0.f ? (uint32_t)min(max(__float2int_rn(__fdiv_rn(v[i], s)), -127), 127) & 0xFFu : 0u;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kE; i += 8)
      if (place<kVec>(i) < D)
        *reinterpret_cast<uint2*>(codes + place<kVec>(i)) =
            make_uint2(q[i] | q[i + 1] << 8 | q[i + 2] << 16 | q[i + 3] << 24,
                       q[i + 4] | q[i + 5] << 8 | q[i + 6] << 16 | q[i + 7] << 24);
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (place<kVec>(i) < D) codes[place<kVec>(i)] = (int8_t)q[i];
  }
}

template <bool kVec, int kE>
cudaError_t launch_typed(const NormArgs& a, dim3 grid, dim3 block, cudaStream_t stream) {
  if (a.residual_bf16) {
    if (a.branch_bf16) block_norm_kernel<kVec, kE, true, true><<<grid, block, 0, stream>>>(a);
    else block_norm_kernel<kVec, kE, true, false><<<grid, block, 0, stream>>>(a);
  } else {
    if (a.branch_bf16) block_norm_kernel<kVec, kE, false, true><<<grid, block, 0, stream>>>(a);
    else block_norm_kernel<kVec, kE, false, false><<<grid, block, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

// Whether rows of `size`-byte elements all begin on 16 bytes.
bool rows16(const void* p, int64_t ld, int size) { return p == nullptr || (aligned(p, 16) && ld * size % 16 == 0); }

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && rows16(a.residual, a.ldr, a.residual_bf16 ? 2 : 4) &&
                   rows16(a.branch, a.ldb, a.branch_bf16 ? 2 : 4) && rows16(a.gate, a.ldg, a.gate_bf16 ? 2 : 4) &&
                   rows16(a.sum, a.lds, a.residual_bf16 ? 2 : 4) &&
                   rows16(a.out, a.ldo, a.out_type == QMM_F32 ? 4 : a.out_type == QMM_BF16 ? 2 : 1) &&
                   aligned(a.post.weight, 16) && aligned(a.post.bias, 16) && aligned(a.pre.weight, 16) &&
                   aligned(a.pre.bias, 16);
  const int units = vec ? a.D / 8 : a.D;                  // groups or values of a row
  auto shape = [&](int per_thread, dim3& grid, dim3& block) {
    const int nt = std::min(1024, (units + 32 * per_thread - 1) / (32 * per_thread) * 32);
    block = dim3(nt, nt == 32 ? 4 : 1);
    grid = dim3((unsigned)((a.T + block.y - 1) / block.y));
  };
  dim3 grid, block;
  if (!vec) {
    if (units <= 8 * 1024) {
      shape(8, grid, block);
      return launch_typed<false, 8>(a, grid, block, stream);
    }
    shape(32, grid, block);
    return launch_typed<false, 32>(a, grid, block, stream);
  }
  if (a.T <= 304 && units <= 1024) {
    shape(1, grid, block);
    return launch_typed<true, 8>(a, grid, block, stream);
  }
  if (units <= 2048) {
    shape(2, grid, block);
    return launch_typed<true, 16>(a, grid, block, stream);
  }
  shape(4, grid, block);
  return launch_typed<true, 32>(a, grid, block, stream);
}

}  // namespace qmm

// A block's output joined to the residual stream, and the next block's input:
//     u = branch_norm(branch);  sum = residual + scale * gate * u;  out = norm(sum)
//     rms:   v * w / sqrt(mean(v^2) + eps) + b
//     layer: (v - mean) * w / sqrt(mean((v - mean)^2) + eps) + b
// and int8 codes of out by the activation quantiser's rule (s = fl(amax / 127)).
//
// Bound: bytes.  Each value of residual, branch and gate is read once and each
// of sum and out written once; a row stays in its threads' registers from the first
// load to the last store, through up to five reductions (two means, two squares,
// one maximum), so that nothing is read again.
//
// Measured against a copy's rate: 16384 rows of 4096 with a norm on either side, all
// fp32 but for out (940 MB), 146 us, 0.96; 4096 of 16384 150; 2049 of 4608 to int8 with a
// channel gate 27.5 us, 0.67; 5000 layer norms of 1000 over bf16 with a gate of rows 12.0 us,
// 0.62, of 1001 16.1, 0.46: rows that begin anywhere touch more sectors, and their ends
// go value by value.  Eight rows of 1024 1.7 us.
//
// A thread holds groups of four neighbouring values, so that a warp's accesses are
// whole in every type (16 bytes a lane in fp32, 8 in bf16, 4 in int8), also where
// rows begin at any element, as long as all tensors' rows do so alike.  Rows of
// tensors that do not go value by value.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "beside.h"
#include "kv_cache.h"
#include "umma.cuh"

namespace qmm {
namespace {

// Four values of a row as they lie in memory.  Read once, and possibly written
// later by the same thread (sum may be the residual itself): coherent loads that
// leave L1 to the weights.
template <bool kBf16>
struct Raw4 {
  uint32_t w[kBf16 ? 2 : 4];
  QMM_DEV float at(int i) const {
    if constexpr (kBf16) return i & 1 ? bf16hi_to_f32(w[i / 2]) : bf16lo_to_f32(w[i / 2]);
    else return __uint_as_float(w[i]);
  }
  QMM_DEV void load(const uint8_t* p) {
    if constexpr (kBf16)
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
  }
};

QMM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Sum (or maximum) over a row's threads; every thread gets the result.  One
// barrier: each reduction of a row has its own slot.
template <bool kMax>
QMM_DEV float row_reduce(float v, float* slot) {
  auto warp_max = [](float x) {            // of magnitudes, whose bits keep their order
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
  };
  if constexpr (kMax) {
    v = warp_max(v);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  if constexpr (kMax) return warp_max(lane < warps ? slot[lane] : 0.f);
  // as many lanes as warps, over and over
  const int span = warps <= 4 ? 4 : warps <= 8 ? 8 : 32, at = lane & (span - 1);
  v = at < warps ? slot[at] : 0.f;
  if (span == 32) {
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
  }
  if (span >= 8) v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 1);
}

// int8 codes of four values by the activation quantiser's rule, as one word.
// rint(fl(v / s)) without a division: y = fl(v * fl(1 / s)) is within 2^-23 |y| + 2^-24
// |y| < 2.3e-5 of fl(v / s) (|y| <= 128, 1 / s neither overflowing nor subnormal), so
// both round to the same integer unless y is that close to a half.  Adding 1.5 *
// 2^23 rounds to the nearest even integer and leaves it in the low bits.  Values
// near a half, and scales out of range, divide.
QMM_DEV uint32_t codes4(const float* v, float s, float r) {
  uint32_t q[4];
  bool divide = !(s > 0x1p-100f && s < 0x1p100f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = __fmul_rn(v[i], r), t = __fadd_rn(y, 12582912.f);
    divide |= fabsf(y - __fsub_rn(t, 12582912.f)) > 0.4999f;
    q[i] = __float_as_uint(t);
  }
  if (divide) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = s > 0.f ? (uint32_t)min(max(__float2int_rn(__fdiv_rn(v[i], s)), -127), 127) : 0u;
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// How a row's groups lie.
template <int kG, bool kOff>
struct Place {
  int e0;        // the first group's first element: a multiple of 4 less the row's offset
  int step;      // from a thread's group to its next
  int D;
  float inv_d;
  QMM_DEV int at(int g) const { return e0 + g * step; }
  QMM_DEV bool some(int g) const { return at(g) < D; }   // a group may begin before the row, but not end there
  QMM_DEV bool whole(int g) const { return kOff ? at(g) >= 0 && at(g) + 4 <= D : at(g) < D; }
  QMM_DEV bool in(int g, int i) const { return kOff ? at(g) + i >= 0 && at(g) + i < D : at(g) < D; }
  // no value of this thread's groups lies outside the row
  QMM_DEV bool all() const { return kOff ? e0 >= 0 && at(kG - 1) + 4 <= D : at(kG - 1) < D; }
};

// A row's values of one tensor, zeros outside it.
template <bool kBf16, int kG, bool kOff>
QMM_DEV void load_row(const void* base, int64_t row, const Place<kG, kOff>& pl, Raw4<kBf16> (&raw)[kG]) {
  constexpr int kSize = kBf16 ? 2 : 4;
  const uint8_t* p = static_cast<const uint8_t*>(base) + (row + pl.e0) * kSize;
#pragma unroll
  for (int g = 0; g < kG; ++g, p += pl.step * kSize) {
    raw[g] = {};
    if (pl.whole(g)) {
      raw[g].load(p);
    } else if (kOff && pl.some(g)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!pl.in(g, i)) continue;
        if constexpr (kBf16) raw[g].w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (i % 2 * 16);
        else raw[g].w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
    }
  }
}

// Four fp32 weights of group g, cached for all rows; zeros outside the row.
template <int kG, bool kOff>
QMM_DEV void weights4(const float* w, const Place<kG, kOff>& pl, int g, bool aligned16, float (&x)[4]) {
  const float* p = w + pl.at(g);
  if (!kOff && aligned16) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else if (pl.whole(g)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(p + i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pl.in(g, i) ? __ldg(p + i) : 0.f;
  }
}

// Those of all groups, all under way before the first is used.
template <int kG, bool kOff>
QMM_DEV void weights(const float* w, const Place<kG, kOff>& pl, bool aligned16, float (&x)[kG][4]) {
  if (!kOff && aligned16) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      // past the row: the last group's, whose products are not used
      const float4 a = __ldg(reinterpret_cast<const float4*>(w + min(pl.at(g), pl.D - 4)));
      x[g][0] = a.x, x[g][1] = a.y, x[g][2] = a.z, x[g][3] = a.w;
    }
  } else {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      x[g][0] = x[g][1] = x[g][2] = x[g][3] = 0.f;
      if (pl.some(g)) weights4(w, pl, g, aligned16, x[g]);
    }
  }
}

// With one group a thread asks for its weights before the reductions: a single
// row would wait for them after each.
template <int kG, bool kOff>
QMM_DEV void apply_norm(const NormSpec& n, const Place<kG, kOff>& pl, bool aligned16, float (&v)[4 * kG],
                        const float (&ahead)[2][4], float (*slots)[32]) {
  if (n.kind == QMM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * kG; ++i) s += v[i];   // values outside the row are zeros
    const float mean = row_reduce<false>(s, slots[0]) * pl.inv_d;
#pragma unroll
    for (int i = 0; i < 4 * kG; ++i) v[i] -= mean;
    if (!pl.all()) {
#pragma unroll
      for (int i = 0; i < 4 * kG; ++i)
        if (!pl.in(i / 4, i % 4)) v[i] = 0.f;
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * kG; ++i) ss = fmaf(v[i], v[i], ss);
  const float inv = rsqrtf(fmaf(row_reduce<false>(ss, slots[1]), pl.inv_d, n.eps));
  float x[kG][4];
  if (n.weight != nullptr) {
    if constexpr (kG > 1) weights(n.weight, pl, aligned16, x);
#pragma unroll
    for (int i = 0; i < 4 * kG; ++i) v[i] = v[i] * inv * (kG > 1 ? x[i / 4][i % 4] : ahead[0][i % 4]);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * kG; ++i) v[i] *= inv;
  }
  if (n.bias != nullptr) {
    if constexpr (kG > 1) weights(n.bias, pl, aligned16, x);
#pragma unroll
    for (int i = 0; i < 4 * kG; ++i)
      if (kOff || pl.some(i / 4)) v[i] += kG > 1 ? x[i / 4][i % 4] : ahead[1][i % 4];   // zeros stay outside the row
  }
}

template <int kG, bool kOff>
QMM_DEV void store_row(void* base, bool bf16, int64_t row, const Place<kG, kOff>& pl, const float (&v)[4 * kG]) {
  const int size = bf16 ? 2 : 4;
  uint8_t* p = static_cast<uint8_t*>(base) + (row + pl.e0) * size;
#pragma unroll
  for (int g = 0; g < kG; ++g, p += pl.step * size) {
    const float* x = v + 4 * g;
    if (pl.whole(g)) {
      if (bf16) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
      else *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else if (kOff && pl.some(g)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!pl.in(g, i)) continue;
        if (bf16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x[i]);
        else reinterpret_cast<float*>(p)[i] = x[i];
      }
    }
  }
}

// A thread's groups of a row on their way through shared memory: it copies just what
// it reads itself, so that no barrier guards the copies.
template <bool kBf16, int kG, bool kOff>
struct Copies {
  static constexpr int kSize = kBf16 ? 2 : 4, kBytes = 4 * kSize;
  // one group of the thread at `to`, the next blockDim.x groups on
  QMM_DEV static void issue(const void* base, int64_t row, const Place<kG, kOff>& pl, uint32_t to) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + (row + pl.e0) * kSize;
#pragma unroll
    for (int g = 0; g < kG; ++g, p += pl.step * kSize, to += blockDim.x * kBytes) {
      if (!pl.some(g)) continue;
      // up to the row's end; before its start lies the row before
      const uint32_t bytes = kOff ? (uint32_t)min((pl.D - pl.at(g)) * kSize, kBytes) : (uint32_t)kBytes;
      if constexpr (kBf16)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(bytes) : "memory");
      else
        umma::cp_async16_zfill(to, p, bytes);
    }
  }
  QMM_DEV static void fetch(uint32_t from, const Place<kG, kOff>& pl, Raw4<kBf16> (&raw)[kG]) {
#pragma unroll
    for (int g = 0; g < kG; ++g, from += blockDim.x * kBytes) {
      raw[g] = {};
      if (!pl.some(g)) continue;
      if constexpr (kBf16)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(raw[g].w[0]), "=r"(raw[g].w[1]) : "r"(from) : "memory");
      else
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(raw[g].w[0]), "=r"(raw[g].w[1]), "=r"(raw[g].w[2]), "=r"(raw[g].w[3])
                     : "r"(from)
                     : "memory");
      if (kOff && !pl.whole(g)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (pl.in(g, i)) continue;
          if constexpr (kBf16) raw[g].w[i / 2] &= i & 1 ? 0xFFFFu : 0xFFFF0000u;
          else raw[g].w[i] = 0;
        }
      }
    }
  }
};

// Threads of a block at most, and blocks per SM that the registers have to allow: two
// of rows of up to 4608 in line (2049 of them to int8 without a gate 25.8 us, with one block
// of 576 threads 34), eight of one-warp rows (20000 layer norms of 255 25.9 us, with six 29.1,
// although 16 values a lane then spill 48 to 224 bytes).
template <int kG, bool kOff, bool kRing>
struct Bounds {
  static constexpr int kThreads = kRing ? (kG == 2 && !kOff ? 576 : 1024) : kG == 1 ? 1024 : 128;
  static constexpr int kBlocks = kRing ? (kG == 2 && !kOff ? 2 : 1) : kG == 1 ? 1 : 8;
};

// A row per blockDim.x threads, kG groups of four values each; blockDim.y rows per
// block (more than one only where a row has one warp, which needs no barrier).
// kOff: rows begin at any element, row t (t * off_step) % 4 behind a boundary.
// kRing: blocks walk over the rows, and while they work on one the next one's values
// are on their way into shared memory.
template <bool kResBf16, bool kBrBf16, int kG, bool kOff, bool kRing>
__global__ void __launch_bounds__(Bounds<kG, kOff, kRing>::kThreads, Bounds<kG, kOff, kRing>::kBlocks)
block_norm_kernel(NormArgs a, int off_step, bool weights16, float inv_d) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float all_slots[kRing ? 2 : 1][5][32];
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;   // whole warps, and only where no barrier follows
  auto place = [&](int64_t row) {
    const int off = kOff ? (int)(row * off_step & 3) : 0;
    return Place<kG, kOff>{(int)threadIdx.x * 4 - off, (int)blockDim.x * 4, a.D, inv_d};
  };
  const bool has_branch = a.branch != nullptr;
  // a gate that is read like a weight, or like the rows
  const bool gate_row = has_branch && a.gate != nullptr && (a.ldg != 0 || a.gate_bf16);
  const uint32_t res_at = umma::smem_u32(ring) + threadIdx.x * (4 * (kResBf16 ? 2 : 4));
  const uint32_t br_at = umma::smem_u32(ring) + kG * blockDim.x * (4 * (kResBf16 ? 2 : 4)) +
                         threadIdx.x * (4 * (kBrBf16 ? 2 : 4));
  const uint32_t gate_at = umma::smem_u32(ring) + kG * blockDim.x * (4 * (kResBf16 ? 2 : 4) + 4 * (kBrBf16 ? 2 : 4)) +
                           threadIdx.x * (a.gate_bf16 ? 8 : 16);
  auto issue = [&](int64_t row) {
    if (row < a.T) {
      const Place<kG, kOff> pl = place(row);
      if (has_branch) Copies<kBrBf16, kG, kOff>::issue(a.branch, row * a.ldb, pl, br_at);
      Copies<kResBf16, kG, kOff>::issue(a.residual, row * a.ldr, pl, res_at);
      if (gate_row) {
        if (a.gate_bf16) Copies<true, kG, kOff>::issue(a.gate, row * a.ldg, pl, gate_at);
        else Copies<false, kG, kOff>::issue(a.gate, row * a.ldg, pl, gate_at);
      }
    }
    umma::cp_async_commit();
  };
  if constexpr (kRing) issue(t);
  int parity = 0;
  do {
    const Place<kG, kOff> pl = place(t);
    // two rows' slots: a warp may be one reduction ahead of another that still reads
    float (*slots)[32] = all_slots[parity];
    float v[4 * kG];
    float post_ahead[2][4] = {}, pre_ahead[2][4] = {};
    auto ask = [&](const NormSpec& n, float (&to)[2][4]) {
      if (kG > 1 || !pl.some(0)) return;
      if (n.weight != nullptr) weights4(n.weight, pl, 0, weights16, to[0]);
      if (n.bias != nullptr) weights4(n.bias, pl, 0, weights16, to[1]);
    };
    {
      Raw4<kResBf16> res[kG];
      Raw4<kBrBf16> br[kG];
      Raw4<false> gate[kG];    // bf16 rows take half of it
      // what waits in shared memory is fetched where it is needed, what comes from
      // memory is asked for before anything else
      auto get_branch = [&] {
        if constexpr (kRing) Copies<kBrBf16, kG, kOff>::fetch(br_at, pl, br);
        else load_row(a.branch, t * a.ldb, pl, br);
      };
      auto get_residual = [&] {
        if constexpr (kRing) Copies<kResBf16, kG, kOff>::fetch(res_at, pl, res);
        else load_row(a.residual, t * a.ldr, pl, res);
      };
      auto get_gate = [&] {
        if (!gate_row) return;
        if (a.gate_bf16) {
          Raw4<true> x[kG];
          if constexpr (kRing) Copies<true, kG, kOff>::fetch(gate_at, pl, x);
          else load_row(a.gate, t * a.ldg, pl, x);
#pragma unroll
          for (int g = 0; g < kG; ++g) gate[g].w[0] = x[g].w[0], gate[g].w[1] = x[g].w[1];
        } else {
          if constexpr (kRing) Copies<false, kG, kOff>::fetch(gate_at, pl, gate);
          else load_row(a.gate, t * a.ldg, pl, gate);
        }
      };
      if constexpr (kRing) {
        umma::cp_async_wait<0>();
      } else {
        if (has_branch) get_branch();
        get_residual();
        get_gate();
        if (has_branch) ask(a.post, post_ahead);
        ask(a.pre, pre_ahead);
      }
      if (has_branch) {
        if constexpr (kRing) get_branch();
#pragma unroll
        for (int i = 0; i < 4 * kG; ++i) v[i] = br[i / 4].at(i % 4);
        if (a.post.kind != 0) apply_norm(a.post, pl, weights16, v, post_ahead, slots);
        if (gate_row) {
          if constexpr (kRing) get_gate();
#pragma unroll
          for (int i = 0; i < 4 * kG; ++i) {
            const uint32_t w = gate[i / 4].w[i % 4 / 2];
            v[i] *= a.gate_bf16 ? (i & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w)) : gate[i / 4].at(i % 4);
          }
        } else if (a.gate != nullptr) {
          float x[kG][4];
          weights(static_cast<const float*>(a.gate), pl, weights16, x);
#pragma unroll
          for (int i = 0; i < 4 * kG; ++i) v[i] *= x[i / 4][i % 4];
        }
        if constexpr (kRing) get_residual();
#pragma unroll
        for (int i = 0; i < 4 * kG; ++i)
          v[i] = fmaf(a.scale, v[i], res[i / 4].at(i % 4));
        // outside the row: zeros, also where the last weights or gates there are no numbers
        if (!kOff && !pl.all()) {
#pragma unroll
          for (int i = 0; i < 4 * kG; ++i)
            if (!pl.some(i / 4)) v[i] = 0.f;
        }
      } else {
        if constexpr (kRing) get_residual();
#pragma unroll
        for (int i = 0; i < 4 * kG; ++i) v[i] = res[i / 4].at(i % 4);
      }
    }
    if constexpr (kRing) issue(t + gridDim.x);   // this row's values have been read and used
    if (a.sum != nullptr) store_row(a.sum, kResBf16, t * a.lds, pl, v);
    if (a.out != nullptr) {
      if (a.pre.kind != 0) apply_norm(a.pre, pl, weights16, v, pre_ahead, slots + 2);
      if (a.out_type != QMM_S8) {
        store_row(a.out, a.out_type == QMM_BF16, t * a.ldo, pl, v);
      } else {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * kG; ++i) amax = fmaxf(amax, fabsf(v[i]));
        const float s = __fdiv_rn(row_reduce<true>(amax, slots[4]), 127.0f), r = __frcp_rn(s);
        if (threadIdx.x == 0) a.s_x[t] = s;
        int8_t* codes = static_cast<int8_t*>(a.out) + t * a.ldo;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          if (!pl.some(g)) continue;
          const uint32_t q = codes4(v + 4 * g, s, r);
          if (!kOff) {
            *reinterpret_cast<uint32_t*>(codes + pl.at(g)) = q;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (pl.in(g, i)) codes[pl.at(g) + i] = (int8_t)(q >> (8 * i));
          }
        }
      }
    }
    t += gridDim.x;
    parity ^= 1;
  } while (kRing && t < a.T);
  if constexpr (kRing) umma::cp_async_wait<0>();
}

// Tensors whose rows begin each at another place: a block per row, value by value
// (values of a thread are blockDim.x apart), the row's fp32 values in shared memory.
__global__ void __launch_bounds__(1024)
block_norm_any_kernel(NormArgs a) {
  extern __shared__ float row[];
  __shared__ float slots[5][32];
  umma::pdl_launch_dependents();
  umma::pdl_wait();
  const int64_t t = blockIdx.x;
  const int D = a.D, first = threadIdx.x, step = blockDim.x;
  const float inv_d = 1.0f / (float)D;
  auto value = [](const void* p, bool bf16, int64_t i) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
  };
  auto put = [](void* p, bool bf16, int64_t i, float v) {
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
  };
  // each thread reads back only what it wrote
  auto norm = [&](const NormSpec& n, float (*slot)[32]) {
    float mean = 0.f;
    if (n.kind == QMM_NORM_LAYER) {
      float s = 0.f;
      for (int e = first; e < D; e += step) s += row[e];
      mean = row_reduce<false>(s, slot[0]) * inv_d;
    }
    float ss = 0.f;
    for (int e = first; e < D; e += step) ss = fmaf(row[e] - mean, row[e] - mean, ss);
    const float inv = rsqrtf(fmaf(row_reduce<false>(ss, slot[1]), inv_d, n.eps));
    for (int e = first; e < D; e += step) {
      float v = (row[e] - mean) * inv;
      if (n.weight != nullptr) v *= n.weight[e];
      if (n.bias != nullptr) v += n.bias[e];
      row[e] = v;
    }
  };
  if (a.branch != nullptr) {
    for (int e = first; e < D; e += step) row[e] = value(a.branch, a.branch_bf16, t * a.ldb + e);
    if (a.post.kind != 0) norm(a.post, slots);
    for (int e = first; e < D; e += step) {
      float u = row[e];
      if (a.gate != nullptr) u *= value(a.gate, a.gate_bf16, t * a.ldg + e);
      row[e] = fmaf(a.scale, u, value(a.residual, a.residual_bf16, t * a.ldr + e));
    }
  } else {
    for (int e = first; e < D; e += step) row[e] = value(a.residual, a.residual_bf16, t * a.ldr + e);
  }
  if (a.sum != nullptr)
    for (int e = first; e < D; e += step) put(a.sum, a.residual_bf16, t * a.lds + e, row[e]);
  if (a.out == nullptr) return;
  if (a.pre.kind != 0) norm(a.pre, slots + 2);
  if (a.out_type != QMM_S8) {
    for (int e = first; e < D; e += step) put(a.out, a.out_type == QMM_BF16, t * a.ldo + e, row[e]);
    return;
  }
  float amax = 0.f;
  for (int e = first; e < D; e += step) amax = fmaxf(amax, fabsf(row[e]));
  const float s = __fdiv_rn(row_reduce<true>(amax, slots[4]), 127.0f);
  if (threadIdx.x == 0) a.s_x[t] = s;
  int8_t* codes = static_cast<int8_t*>(a.out) + t * a.ldo;
  for (int e = first; e < D; e += step)
    codes[e] = (int8_t)(s > 0.f ? min(max(__float2int_rn(__fdiv_rn(row[e], s)), -127), 127) : 0);
}

template <int kG, bool kRing>
cudaError_t launch_groups(const NormArgs& a, bool even, int off_step, bool weights16, int groups,
                          cudaStream_t stream) {
  void (*kern[8])(NormArgs, int, bool, float) = {
      block_norm_kernel<false, false, kG, false, kRing>, block_norm_kernel<false, true, kG, false, kRing>,
      block_norm_kernel<true, false, kG, false, kRing>,  block_norm_kernel<true, true, kG, false, kRing>,
      block_norm_kernel<false, false, kG, true, kRing>,  block_norm_kernel<false, true, kG, true, kRing>,
      block_norm_kernel<true, false, kG, true, kRing>,   block_norm_kernel<true, true, kG, true, kRing>};
  const int nt = (groups + 32 * kG - 1) / (32 * kG) * 32;   // within Bounds by the rules below
  const int which = (even ? 0 : 4) + (a.residual_bf16 ? 2 : 0) + (a.branch_bf16 ? 1 : 0);
  const float inv_d = 1.0f / (float)a.D;
  if constexpr (!kRing) {
    const dim3 block(nt, nt == 32 ? 4 : 1);
    return launch_pdl(kern[which], dim3((unsigned)((a.T + block.y - 1) / block.y)), block, 0, stream, a, off_step,
                      weights16, inv_d);
  }
  const int bytes = (a.residual_bf16 ? 2 : 4) + (a.branch_bf16 ? 2 : 4) +
                    (a.gate != nullptr && (a.ldg != 0 || a.gate_bf16) ? (a.gate_bf16 ? 2 : 4) : 0);
  const size_t smem = (size_t)kG * nt * 4 * bytes;
  static std::atomic<uint64_t> done[8];
  cudaError_t err = set_once(done[which], reinterpret_cast<const void*>(kern[which]),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kG * 1024 * 4 * 12);
  if (err != cudaSuccess) return err;
  int per_sm = 0;
  if ((err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern[which], nt, smem)) != cudaSuccess) return err;
  const int grid = std::min(a.T, std::max(1, per_sm) * attn_sm_count());
  return launch_pdl(kern[which], dim3((unsigned)grid), dim3(nt), smem, stream, a, off_step, weights16, inv_d);
}

// Whether a tensor's rows begin where those of stride `ld0` do, between two
// boundaries of four elements (of `size` bytes).
bool in_step(const void* p, int64_t ld, int64_t ld0, int size) {
  return p == nullptr || (aligned(p, 4 * size) && (ld - ld0) % 4 == 0);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t stream) {
  const int res_size = a.residual_bf16 ? 2 : 4;
  const int64_t ld0 = a.ldr;
  // the row-by-row gate keeps step with the rest; one row for all is read like a weight in fp32
  const bool gate_row = a.gate != nullptr && a.ldg != 0;
  const bool even = a.D % 4 == 0 && ld0 % 4 == 0;
  bool together = in_step(a.residual, a.ldr, ld0, res_size) && in_step(a.sum, a.lds, ld0, res_size) &&
                  in_step(a.branch, a.ldb, ld0, a.branch_bf16 ? 2 : 4) &&
                  (!gate_row || in_step(a.gate, a.ldg, ld0, a.gate_bf16 ? 2 : 4)) &&
                  (a.out_type == QMM_S8 || in_step(a.out, a.ldo, ld0, a.out_type == QMM_BF16 ? 2 : 4));
  // a bf16 row for all tokens has to begin with the rows
  if (a.gate != nullptr && !gate_row && a.gate_bf16) together = together && even && aligned(a.gate, 8);
  const int groups = (a.D + (even ? 0 : 3) + 3) / 4;
  if (!together || groups > 4096) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t err = set_once(done, reinterpret_cast<const void*>(block_norm_any_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormMaxD * 4);
    if (err != cudaSuccess) return err;
    const int nt = std::min(1024, (a.D + 127) / 128 * 32);
    return launch_pdl(block_norm_any_kernel, dim3((unsigned)a.T), dim3(nt), (size_t)a.D * 4, stream, a);
  }
  const bool weights16 = aligned(a.post.weight, 16) && aligned(a.post.bias, 16) && aligned(a.pre.weight, 16) &&
                         aligned(a.pre.bias, 16) && (gate_row || aligned(a.gate, 16));
  const int off_step = (int)(ld0 % 4);
  // Times are of a post norm and a residual in fp32 where no other is named.
  // Few rows: a row's latency counts, so four values a thread, as long as the GPU holds
  // all threads at once (300 rows of 1024: 2.8 us, by the rules below 3.1; 1200, which
  // no longer fit: 6.4 and 5.4).
  const int64_t threads = (int64_t)a.T * ((groups + 31) / 32 * 32);
  if (groups <= 1024 && threads <= (int64_t)1280 * attn_sm_count())
    return launch_groups<1, false>(a, even, off_step, weights16, groups, stream);
  // A row that one warp holds has no barrier, and many such rows are on an SM: nothing
  // comes ahead (8000 rows of 256 7.8 us, ahead 9.2).  16 values a lane rather than
  // half-empty warps of eight (20000 layer norms of 255 25.7 us, with eight 33.5).
  if (groups <= 64) return launch_groups<2, false>(a, even, off_step, weights16, groups, stream);
  if (groups <= 96) return launch_groups<4, false>(a, even, off_step, weights16, groups, stream);
  // Other rows' warps wait for one another, so that without the next row's values on their
  // way an SM's memory traffic pauses: 2500 rows of 1024 8.6 us, with nothing ahead 9.1,
  // 4096 rows of 16384 146 and 199.  Very many short rows do without: they come and go at
  // different times (65536 of 1024 141 us, ahead 152; 30000 68.5 and 69.5, of 2048 131 and 129).
  if (a.T > 32768 && groups <= 384) return launch_groups<4, false>(a, even, off_step, weights16, groups, stream);
  // Eight values a thread up to 4608 in a row, 16 beyond (8000 rows of 4096 73.7 and 77.5 us,
  // 2500 of 6144 43.2 and 37.2).  Rows out of line take 16 earlier, for their ends' sake
  // (5000 of 2049 31.4 and 33.4, of 4095 63.5 and 59.2).
  if (groups <= (even ? 1152 : 640)) return launch_groups<2, true>(a, even, off_step, weights16, groups, stream);
  return launch_groups<4, true>(a, even, off_step, weights16, groups, stream);
}

}  // namespace qmm

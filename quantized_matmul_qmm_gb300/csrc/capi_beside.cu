// C-ABI entry points of what runs beside the projections: argument validation,
// then the launch.  Every check runs on the host before anything is queued.
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "beside.h"

using namespace qmm;

namespace {

qmm_status beside_status(cudaError_t e) {
  if (e == cudaSuccess) return QMM_OK;
  if (std::getenv("QMM_LOG")) std::fprintf(stderr, "qmm: CUDA error %s\n", cudaGetErrorString(e));
  return QMM_ERR_CUDA;
}

bool float_type(qmm_dtype t) { return t == QMM_F32 || t == QMM_BF16; }
uintptr_t size_of(qmm_dtype t) { return t == QMM_F32 ? 4 : t == QMM_BF16 ? 2 : 1; }

// A row stride of `rows` rows of `width` elements; what a single row's holds is not used.
bool rows_ok(int64_t stride, int64_t rows, int64_t width) {
  return rows <= 1 || (stride >= width && stride <= (INT64_MAX >> 3) / rows);   // byte offsets within 64 bits
}

bool norm_ok(const qmm_norm* n) {
  return n == nullptr || ((n->kind == QMM_NORM_RMS || n->kind == QMM_NORM_LAYER) && n->eps >= 0.f &&
                          std::isfinite(n->eps) && aligned(n->weight, 4) && aligned(n->bias, 4));
}
NormSpec spec_of(const qmm_norm* n) {
  return n == nullptr ? NormSpec{0, 0.f, nullptr, nullptr} : NormSpec{(int)n->kind, n->eps, n->weight, n->bias};
}

qmm_status lora_sizes(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank) {
  if (M < 0 || K < 1 || N < 1 || n_adapters < 1 || max_rank < 1) return QMM_ERR_INVALID_ARG;
  if (K % 8 != 0 || max_rank > kLoraMaxRank || n_adapters > kLoraMaxAdapters || K >= (int64_t)1 << 28 ||
      N >= (int64_t)1 << 24 || M >= (int64_t)1 << 24)
    return QMM_ERR_UNSUPPORTED;
  return QMM_OK;
}

// Strides of bf16 rows that are read 16 bytes at a time.
bool stride8(int64_t stride, int64_t count, int64_t least) {
  return count <= 1 || (stride >= least && stride <= (INT64_MAX >> 5) / count && stride % 8 == 0);
}

qmm_status token_logprobs(const void* logits, qmm_dtype type, int64_t M, int64_t V, int64_t ld, float scale,
                          const int32_t* tokens, int64_t ld_tokens, int64_t G, float* logprobs, float* entropy,
                          int64_t top_k, int32_t* top_ids, float* top_logprobs, int32_t* dev_status,
                          const float* other, cudaStream_t stream) {
  if (!float_type(type) || M < 0 || V < 1 || G < 0 || top_k < 0 || !(scale > 0.f && scale <= kMaxScale))
    return QMM_ERR_INVALID_ARG;
  if (!rows_ok(ld, M, V) || (G > 0 && !rows_ok(ld_tokens, M, G))) return QMM_ERR_INVALID_ARG;
  if (entropy == nullptr && G == 0 && top_k == 0) return QMM_ERR_INVALID_ARG;
  if (top_k > kMaxTop || V >= INT32_MAX - 65536 || G > 1024 || M >= (int64_t)1 << 26) return QMM_ERR_UNSUPPORTED;
  if (M == 0) return QMM_OK;
  if (logits == nullptr || !aligned(logits, size_of(type)) || !aligned(entropy, 4)) return QMM_ERR_INVALID_ARG;
  if (G > 0 && (tokens == nullptr || logprobs == nullptr || !aligned(tokens, 4) || !aligned(logprobs, 4)))
    return QMM_ERR_INVALID_ARG;
  if (top_k > 0 && (top_ids == nullptr || top_logprobs == nullptr || !aligned(top_ids, 4) ||
                    !aligned(top_logprobs, 4)))
    return QMM_ERR_INVALID_ARG;
  LogprobArgs a{};
  a.logits = logits;
  a.bf16 = type == QMM_BF16;
  a.M = (int)M;
  a.V = (int)V;
  a.ld = M > 1 ? ld : 0;
  a.scale = scale;
  a.tokens = tokens;
  a.ld_tokens = M > 1 ? ld_tokens : 0;
  a.G = (int)G;
  a.logprobs = logprobs;
  a.write_other = other != nullptr;
  a.other = other != nullptr ? *other : 0.f;
  a.entropy = entropy;
  a.top_k = (int)top_k;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.dev_status = dev_status;
  return beside_status(launch_token_logprobs(a, stream));
}

}  // namespace

extern "C" {

qmm_status qmm_block_norm(const void* residual, qmm_dtype residual_type, int64_t ldr, const void* branch,
                          qmm_dtype branch_type, int64_t ldb, const qmm_norm* branch_norm, const void* gate,
                          qmm_dtype gate_type, int64_t ldg, float scale, void* sum, int64_t lds,
                          const qmm_norm* norm, void* out, qmm_dtype out_type, int64_t ldo, float* s_x, int64_t T,
                          int64_t D, cudaStream_t stream) {
  if (!float_type(residual_type) || T < 0 || D < 1 || !norm_ok(norm)) return QMM_ERR_INVALID_ARG;
  if (T > 0 && ((sum == nullptr && out == nullptr) || residual == nullptr)) return QMM_ERR_INVALID_ARG;
  if (!rows_ok(ldr, T, D) || !aligned(residual, size_of(residual_type))) return QMM_ERR_INVALID_ARG;
  if (branch != nullptr) {
    if (!float_type(branch_type) || !rows_ok(ldb, T, D) || !aligned(branch, size_of(branch_type)) ||
        !norm_ok(branch_norm) || !std::isfinite(scale))
      return QMM_ERR_INVALID_ARG;
    if (gate != nullptr && (!float_type(gate_type) || !aligned(gate, size_of(gate_type)) ||
                            (ldg != 0 && !rows_ok(ldg, T, D))))
      return QMM_ERR_INVALID_ARG;
  }
  if (sum != nullptr) {
    if (!rows_ok(lds, T, D) || !aligned(sum, size_of(residual_type))) return QMM_ERR_INVALID_ARG;
    if (sum == residual && T > 1 && lds != ldr) return QMM_ERR_INVALID_ARG;
  }
  if (out != nullptr) {
    if ((!float_type(out_type) && out_type != QMM_S8) || !rows_ok(ldo, T, D) || out == residual || out == sum ||
        out == branch)
      return QMM_ERR_INVALID_ARG;
    if (out_type == QMM_S8 ? !aligned(out, 16) || (T > 1 && ldo % 16 != 0) || s_x == nullptr || !aligned(s_x, 4)
                           : !aligned(out, size_of(out_type)))
      return QMM_ERR_INVALID_ARG;
  }
  if (D > kNormMaxD || T > INT32_MAX) return QMM_ERR_UNSUPPORTED;
  if (T == 0) return QMM_OK;
  NormArgs a{};
  const bool many = T > 1;
  a.residual = residual;
  a.residual_bf16 = residual_type == QMM_BF16;
  a.ldr = many ? ldr : 0;
  a.branch = branch;
  if (branch != nullptr) {
    a.branch_bf16 = branch_type == QMM_BF16;
    a.ldb = many ? ldb : 0;
    a.post = spec_of(branch_norm);
    a.gate = gate;
    a.gate_bf16 = gate_type == QMM_BF16;
    a.ldg = many ? ldg : 0;
    a.scale = scale;
  }
  a.sum = sum;
  a.lds = many ? lds : 0;
  a.pre = spec_of(norm);
  a.out = out;
  a.out_type = (int)out_type;
  a.ldo = many ? ldo : 0;
  a.s_x = s_x;
  a.T = (int)T;
  a.D = (int)D;
  return beside_status(launch_block_norm(a, stream));
}

qmm_status qmm_lora_add_workspace_size(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank,
                                       size_t* ws_bytes) {
  if (ws_bytes == nullptr) return QMM_ERR_INVALID_ARG;
  const qmm_status st = lora_sizes(M, K, N, n_adapters, max_rank);
  if (st != QMM_OK) return st;
  *ws_bytes = lora_workspace_bytes(M, K, N, n_adapters, max_rank);
  return QMM_OK;
}

qmm_status qmm_lora_add(const qmm_lora_set* set, const void* X, int64_t ldx, const int32_t* ids, int64_t M,
                        const float* base, int64_t ldb, float* out, int64_t ldo, void* workspace, size_t ws_bytes,
                        int32_t* dev_status, cudaStream_t stream) {
  if (set == nullptr || set->A == nullptr || set->B == nullptr) return QMM_ERR_INVALID_ARG;
  const qmm_status st = lora_sizes(M, set->K, set->N, set->n_adapters, set->max_rank);
  if (st != QMM_OK) return st;
  if (!aligned(set->A, 16) || !aligned(set->B, 16) || !aligned(set->ranks, 4) || !aligned(set->scales, 4) ||
      !stride8(set->a_stride_slot, set->n_adapters, 8) || !stride8(set->a_stride_rank, set->max_rank, set->K) ||
      !stride8(set->b_stride_slot, set->n_adapters, 8) || !stride8(set->b_stride_row, set->N, set->max_rank))
    return QMM_ERR_INVALID_ARG;
  if (!stride8(ldx, M, set->K) || (base != nullptr && !rows_ok(ldb, M, set->N)) || !rows_ok(ldo, M, set->N))
    return QMM_ERR_INVALID_ARG;
  if (lora_units(M, set->N, set->n_adapters) > INT32_MAX) return QMM_ERR_UNSUPPORTED;
  if (M == 0) return QMM_OK;
  if (X == nullptr || ids == nullptr || out == nullptr || !aligned(X, 16) || !aligned(ids, 4) || !aligned(base, 4) ||
      !aligned(out, 4))
    return QMM_ERR_INVALID_ARG;
  if (base == out && M > 1 && ldb != ldo) return QMM_ERR_INVALID_ARG;
  const size_t need = lora_workspace_bytes(M, set->K, set->N, set->n_adapters, set->max_rank);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || ws_bytes < need)) return QMM_ERR_WORKSPACE;
  LoraArgs a{};
  a.A = static_cast<const __nv_bfloat16*>(set->A);
  a.B = static_cast<const __nv_bfloat16*>(set->B);
  a.a_slot = set->n_adapters > 1 ? set->a_stride_slot : 0;
  a.a_rank = set->max_rank > 1 ? set->a_stride_rank : 0;
  a.b_slot = set->n_adapters > 1 ? set->b_stride_slot : 0;
  a.b_row = set->N > 1 ? set->b_stride_row : 0;
  a.ranks = set->ranks;
  a.scales = set->scales;
  a.n_adapters = (int)set->n_adapters;
  a.max_rank = (int)set->max_rank;
  a.K = (int)set->K;
  a.N = (int)set->N;
  a.X = static_cast<const __nv_bfloat16*>(X);
  a.ldx = M > 1 ? ldx : 0;
  a.ids = ids;
  a.M = (int)M;
  a.base = base;
  a.ldb = M > 1 ? ldb : 0;
  a.out = out;
  a.ldo = M > 1 ? ldo : 0;
  a.dev_status = dev_status;
  return beside_status(launch_lora_add(a, workspace, stream));
}

qmm_status qmm_token_logprobs(const void* logits, qmm_dtype type, int64_t M, int64_t V, int64_t ld, float scale,
                              const int32_t* tokens, int64_t ld_tokens, int64_t G, float* logprobs, float* entropy,
                              int64_t top_k, int32_t* top_ids, float* top_logprobs, int32_t* dev_status,
                              cudaStream_t stream) {
  return token_logprobs(logits, type, M, V, ld, scale, tokens, ld_tokens, G, logprobs, entropy, top_k, top_ids,
                        top_logprobs, dev_status, nullptr, stream);
}

qmm_status qmm_token_logprobs_or(const void* logits, qmm_dtype type, int64_t M, int64_t V, int64_t ld, float scale,
                                 const int32_t* tokens, int64_t ld_tokens, int64_t G, float* logprobs, float* entropy,
                                 int64_t top_k, int32_t* top_ids, float* top_logprobs, int32_t* dev_status,
                                 float other, cudaStream_t stream) {
  return token_logprobs(logits, type, M, V, ld, scale, tokens, ld_tokens, G, logprobs, entropy, top_k, top_ids,
                        top_logprobs, dev_status, &other, stream);
}

}  // extern "C"

// Host-side declarations of what runs beside the projections: block norms,
// low-rank adapters and token log probabilities.
#pragma once

#include "qmm_internal.h"

namespace qmm {

// ---- block norm (block_norm.cu) ----
constexpr int64_t kNormMaxD = 32768;
struct NormSpec {
  int kind;             // 0 for none, else qmm_norm_kind
  float eps;
  const float* weight;  // [D] or null
  const float* bias;    // [D] or null
};
struct NormArgs {
  const void* residual;
  const void* branch;   // or null
  const void* gate;     // or null
  void* sum;            // or null
  void* out;            // or null
  float* s_x;           // int8 out
  int64_t ldr, ldb, ldg, lds, ldo;   // elements; ldg 0: one row for all tokens
  bool residual_bf16, branch_bf16, gate_bf16;
  int out_type;         // qmm_dtype
  float scale;
  NormSpec post, pre;   // of the branch, of the sum
  int T, D;
};
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t stream);

// ---- low-rank adapters (lora.cu) ----
constexpr int64_t kLoraMaxRank = 256, kLoraMaxAdapters = 8192;
struct LoraArgs {
  const __nv_bfloat16* A;
  const __nv_bfloat16* B;
  int64_t a_slot, a_rank, b_slot, b_row;   // elements
  const int32_t* ranks;
  const float* scales;
  int n_adapters, max_rank, K, N;
  const __nv_bfloat16* X;
  int64_t ldx;
  const int32_t* ids;
  int M;
  const float* base;   // or null
  int64_t ldb;
  float* out;
  int64_t ldo;
  int32_t* dev_status;
};
// tiles of rows and columns that a call's second product walks over, at most
inline int64_t lora_units(int64_t M, int64_t N, int64_t n_adapters) {
  return (M / 128 + (n_adapters + 1 < M ? n_adapters + 1 : M)) * ((N + 127) / 128);
}
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t n_adapters, int64_t max_rank);
cudaError_t launch_lora_add(const LoraArgs& a, void* workspace, cudaStream_t stream);

// ---- token log probabilities (logprobs.cu) ----
constexpr int kMaxTop = 32;
constexpr float kMaxScale = 0x1p127f;   // times log2(e) it is still finite
struct LogprobArgs {
  const void* logits;
  bool bf16;
  int M, V;
  int64_t ld;          // elements
  float scale;
  const int32_t* tokens;
  int64_t ld_tokens;
  int G;
  float* logprobs;
  bool write_other;    // `other` for tokens that are not scored
  float other;
  float* entropy;      // or null
  int top_k;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* dev_status;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);

}  // namespace qmm

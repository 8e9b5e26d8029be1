// TMA descriptors of a paged cache's sides.  As in tmap.cu, the driver's
// cuTensorMapEncodeTiled is reached through the runtime's entry-point query.
#include <cuda.h>

#include "kv_cache.h"

namespace qmm {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {           // once per process
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

}  // namespace

bool make_tmap_kv(CUtensorMap* map, const void* base, bool s8, int head_dim, uint32_t page_size, uint64_t n_heads,
                  uint64_t n_pages, int64_t st_token, int64_t st_head, int64_t st_page, uint32_t box_tokens) {
  const EncodeTiledFn encode = encode_tiled();
  if (encode == nullptr) return false;
  // A dimension of one row has no stride of its own: any valid one will do.
  auto stride = [&](int64_t s) { return (cuuint64_t)(s > 0 ? s : head_dim * (s8 ? 1 : 2)); };
  const cuuint64_t dims[4] = {(cuuint64_t)head_dim, page_size, n_heads, n_pages};
  const cuuint64_t strides[3] = {stride(st_token), stride(st_head), stride(st_page)};
  const cuuint32_t box[4] = {s8 ? (cuuint32_t)head_dim : 64u, box_tokens, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, s8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            s8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace qmm

// The tensor-core attention's fp16 instances, its tensor maps and its dispatch.
#include <cudaTypedefs.h>

#include <mutex>

#include "attn_tc_kernel.cuh"
#include "sdv.h"

namespace sdv {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace

bool attn_page_map(const void* pages, bool bf16, uint64_t rows, int dim, int box_rows, CUtensorMap* map) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)dim, rows};
  cuuint64_t strides[1] = {(cuuint64_t)dim * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(pages), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_query_map(const void* q, bool bf16, long long tokens, int heads, int group, int dim, long long stride,
                    int box_tokens, CUtensorMap* map) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t attn_tc_bf16(const AttnMaps& m, const AttnArgs& a, cudaStream_t st);

bool attn_tc_takes(int dim, int group, int page, long long cache_rows) {
  return group <= kAttnTcRows && (dim == 64 || dim == 128 || dim == 256) && page >= 8 && (page & (page - 1)) == 0 &&
         cache_rows <= INT32_MAX - 256;
}

cudaError_t launch_attn_tc(int dtype, const AttnArgs& a, cudaStream_t st) {
  AttnMaps m;
  const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page;
  const int box = a.page < a.tile ? a.page : a.tile;
  const bool bf = dtype == SDV_BF16;
  if (!attn_page_map(a.k, bf, rows, a.D, box, &m.k) || !attn_page_map(a.v, bf, rows, a.D, box, &m.v) ||
      !attn_query_map(a.q, bf, (long long)a.B * a.S, a.Hq, a.G, a.D, a.q_stride, a.tile_wrows, &m.q))
    return cudaErrorUnknown;
  return bf ? attn_tc_bf16(m, a, st) : attn_tc_dispatch<__half>(m, a, st);
}

}  // namespace sdv

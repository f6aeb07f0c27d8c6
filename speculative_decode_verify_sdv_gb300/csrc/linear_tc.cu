// The chunked linear attention's fp16 instances, its tensor maps and its dispatch.
#include <cudaTypedefs.h>

#include <mutex>

#include "linear_tc_kernel.cuh"
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

// Rows of one tensor as [B * T][heads][dim]: boxes of 64 elements x one head x a chunk's tokens.
bool token_map(const void* p, bool bf16, int dim, int heads, long long stride, long long tokens, CUtensorMap* map) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)kLinChunk};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t linear_tc_f16(const LinMaps& m, const LinArgs& a, cudaStream_t st) {
  return linear_tc_dispatch<__half>(m, a, st);
}

cudaError_t launch_linear_tc(int dtype, const LinArgs& args, cudaStream_t st) {
  LinArgs a = args;
  LinMaps m;
  const bool bf = dtype == SDV_BF16;
  const long long tokens = (long long)a.B * a.T;
  if (!token_map(a.k, bf, a.Dk, a.Hqk, a.k_stride, tokens, &m.k) ||
      !token_map(a.v, bf, a.Dv, a.H, a.v_stride, tokens, &m.v))
    return cudaErrorUnknown;
  m.q = m.k;
  if (a.o != nullptr && !token_map(a.q, bf, a.Dk, a.Hqk, a.q_stride, tokens, &m.q)) return cudaErrorUnknown;
  cudaError_t e = cudaSuccess;
  if (a.T > kLinChunk) {  // a head of one chunk is never shared
    a.pass = 0;
    e = bf ? linear_tc_bf16(m, a, st) : linear_tc_f16(m, a, st);
    if (e != cudaSuccess) return e;
  }
  a.pass = 1;
  return bf ? linear_tc_bf16(m, a, st) : linear_tc_f16(m, a, st);
}

}  // namespace sdv

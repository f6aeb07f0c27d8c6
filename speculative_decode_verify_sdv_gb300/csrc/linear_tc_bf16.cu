// The chunked linear attention's bf16 instances (a translation unit of their own: the
// two types compile side by side).
#include "linear_tc_kernel.cuh"

namespace sdv {

cudaError_t linear_tc_bf16(const LinMaps& m, const LinArgs& a, cudaStream_t st) {
  return linear_tc_dispatch<__nv_bfloat16>(m, a, st);
}

}  // namespace sdv

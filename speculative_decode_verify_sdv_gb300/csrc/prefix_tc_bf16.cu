// The tensor-core prefix attention's bf16 instances (a translation unit of their own: the
// two types compile side by side).
#include "prefix_tc_kernel.cuh"

namespace sdv {

cudaError_t prefix_tc_bf16(const PrefixMaps& m, const PrefixArgs& a, cudaStream_t st) {
  return prefix_tc_dispatch<__nv_bfloat16>(m, a, st);
}

}  // namespace sdv

// The tensor-core attention's bf16 instances (a translation unit of their own: the
// two types compile side by side).
#include "attn_tc_kernel.cuh"

namespace sdv {

cudaError_t attn_tc_bf16(const AttnMaps& m, const AttnArgs& a, cudaStream_t st) {
  return attn_tc_dispatch<__nv_bfloat16>(m, a, st);
}

}  // namespace sdv

// The tensor-core prefix attention's fp16 instances, its tensor maps and its dispatch.
#include "attn_tc.h"
#include "prefix_tc_kernel.cuh"
#include "sdv.h"

namespace sdv {

cudaError_t prefix_tc_bf16(const PrefixMaps& m, const PrefixArgs& a, cudaStream_t st);

cudaError_t launch_prefix_tc(int dtype, const PrefixArgs& a, cudaStream_t st) {
  PrefixMaps m;
  const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page;
  const int box = a.page < kPrefixTcTile ? a.page : kPrefixTcTile;
  const bool bf = dtype == SDV_BF16;
  if (!attn_page_map(a.k, bf, rows, a.D, box, &m.k) || !attn_page_map(a.v, bf, rows, a.D, box, &m.v) ||
      !attn_query_map(a.q, bf, a.tokens, a.Hq, a.G, a.D, a.q_stride, a.tile_tokens, &m.q))
    return cudaErrorUnknown;
  return bf ? prefix_tc_bf16(m, a, st) : prefix_tc_dispatch<__half>(m, a, st);
}

}  // namespace sdv

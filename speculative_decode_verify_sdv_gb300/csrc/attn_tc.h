// The tensor-core attention's interface to the entry points.
#pragma once

#include <cuda.h>

#include "attn_sched.cuh"

namespace sdv {

struct AttnMaps {
  CUtensorMap k, v, q;
};

constexpr int kAttnTcRows = 128;  // query rows per tile
// Cache positions per tile: keys and values of 64 KB (32 KB at dim 64) either way;
// at dim 256 the output takes half of tensor memory and scores the rest.
__host__ __device__ constexpr int attn_tc_tile(int dim) { return dim == 256 ? 64 : 128; }

// Head sizes with an instance, groups that fit a row tile, pages that a tile is a whole number of (or the
// reverse), and a cache whose rows the tensor map's 32-bit coordinate can name.
bool attn_tc_takes(int dim, int group, int page, long long cache_rows);
cudaError_t launch_attn_tc(int dtype, const AttnArgs& a, cudaStream_t st);

}  // namespace sdv

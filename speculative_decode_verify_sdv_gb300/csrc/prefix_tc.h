// The tensor-core attention over a shared prefix: its interface to the entry point.
#pragma once

#include <cuda.h>

#include "prefix_attn.cuh"

namespace sdv {

struct PrefixMaps {
  CUtensorMap k, v, q;
};

constexpr int kPrefixTcTile = 128;  // positions per tile
constexpr int kPrefixTcRows = 128;  // query rows per row tile, at most

// Row tiles that a unit takes side by side: two share every tile of the prefix where their
// outputs and scores fit tensor memory and there are rows for them.
constexpr int prefix_tc_streams(int dim, int row_tiles) { return dim <= 128 && row_tiles > 1 ? 2 : 1; }

cudaError_t launch_prefix_tc(int dtype, const PrefixArgs& a, cudaStream_t st);

}  // namespace sdv

// Attention of a batch's rows to each sequence's own positions, behind a shared prefix: the
// interface of its kernel to the entry point and the join.
#pragma once

#include "attn_sched.cuh"
#include "prefix_attn.cuh"

namespace sdv {

constexpr int kOwnTile = 64;        // positions that a part is a whole number of
constexpr int kOwnMaxParts = 16;

// A sequence's own positions in parts of whole tiles, a CTA each for up to 64 rows (and the prefix's).
struct OwnArgs {
  AttnArgs attn;      // tile = kOwnTile; out, lse and workspace fields of no meaning
  int warps;          // of a CTA, 1, 2 or 4: 16 rows of a kv head each
  int row_groups;     // CTAs for all rows of a kv head
  int parts;          // of a sequence, at most
  float* part_o;      // [parts][B * S][Hq][D], relative to the part's maximum
  float2* part_ml;    // [parts][B * S][Hq]: maximum (log2 domain), sum
  int* status;
  // The prefix in parts too, for few rows: all rows of a kv head in one CTA.
  int prefix_parts;   // 0: it is the tensor-core kernel's
  const int32_t *prefix_table, *prefix_length;
  int prefix_pages;
  float* prefix_o;    // [prefix_parts][B * S][Hq][D], [2]: as above
  float2* prefix_ml;
};

struct JoinArgs {
  PrefixArgs prefix;
  OwnArgs own;           // parts > 0: its partials; else attn.out32 and attn.lse hold outputs
  void* out;
  float* lse;            // or null
};

// Tiles of each part of a sequence but the last, and how many parts have any.
__device__ __forceinline__ int own_per_part(int tiles, int parts) { return (tiles + parts - 1) / parts; }
__device__ __forceinline__ int own_live_parts(int tiles, int parts) {
  const int per = own_per_part(tiles, parts);
  return (tiles + per - 1) / per;
}

// Whether the positions that a table may hold are few enough for the parts (the shapes are those of
// the tensor-core kernels, attn_tc_takes).
bool own_takes(const OwnArgs& o, int sms);
// last: the own positions, of a single part each, are joined with the prefix's partials here (heads
// of up to 128).
cudaError_t launch_prefix_own(int dtype, const JoinArgs& j, bool last, cudaStream_t st);

}  // namespace sdv

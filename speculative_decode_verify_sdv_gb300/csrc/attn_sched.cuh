// Work split of the paged attention: shared by its kernels and the join.
//
// The cache positions of every (sequence, kv head, row tile) -- a unit -- are cut
// into tiles of `tile` positions; the tiles of all units, laid end to end, are
// dealt in equal contiguous ranges to the CTAs of one wave.  A unit weighs its
// tiles and `lead` more, the time that its queries, its last tile's cleaning and its
// outputs take in tiles' time, laid before its first tile: short contexts in a batch
// would otherwise all fall to a few CTAs.  Ragged contexts are then balanced to one
// tile whatever their lengths, and one long context spreads over the whole GPU.  A unit inside one CTA's range is finished there; the others
// leave (unnormalised output, max, sum) partials that the join launch adds in CTA
// order.  The lengths live on the device, so every warp that needs the split
// computes it from them (a warp-wide scan over the sequences), and the split is a
// function of lengths and shapes alone: results do not vary from run to run.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "sdv_kernels.h"

namespace sdv {

struct AttnArgs {
  const void* q;
  long long q_stride;       // elements between window rows
  const void* k;            // [n_pages][Hkv][page][D]
  const void* v;
  const int32_t* table;     // [B][max_pages]
  const int32_t* ctx;       // [B]
  const int32_t* n_rows;    // [B] or null
  const uint32_t* mask;     // [B][S] or null
  float scale_log2;         // scale * log2(e)
  int B, S, Hq, Hkv, G, D;
  int n_pages, page, max_pages;
  int rows;                 // S * G query rows of a kv head, row r = (window row r / G, head r % G)
  int row_tiles, row_tile;  // row tiles of a kv head, rows of one (the last may hold fewer)
  int tile;                 // cache positions per tile
  int lead;                 // weight of a unit beyond its tiles
  void* out;
  float* lse;               // or null
  float* part_o;            // [2 * CTAs][row_tile][D]
  float* part_ml;           // [2 * CTAs][row_tile][2]: max (log2 domain), sum
  int* status;
  int ctas;                 // CTAs of the attention launch
  int slots, q_bufs;        // tensor-core kernel: ring slots, Q buffers
};

struct AttnSeq {
  int ctx, n;   // context positions, live window rows
  int tiles;    // tiles of each of its units (at least one: it writes the empty rows)
  bool bad;     // a length was out of range
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  AttnSeq s;
  const long long cap = (long long)a.max_pages * a.page;
  const int most = cap > 0x7fffff00ll ? 0x7fffff00 : (int)cap;
  const int c = __ldg(a.ctx + b);
  const int n = a.n_rows != nullptr ? __ldg(a.n_rows + b) : a.S;
  s.ctx = min(max(c, 0), most);
  s.n = min(min(max(n, 0), a.S), most - s.ctx);
  s.bad = s.ctx != c || s.n != n;
  s.tiles = max(1, (int)(((long long)s.ctx + s.n + a.tile - 1) / a.tile));
  return s;
}

// Weight of all units.  Warp-collective; every lane gets the result.
__device__ __forceinline__ long long attn_total(const AttnArgs& a, int lane) {
  long long sum = 0;
  for (int b = lane; b < a.B; b += 32) sum += attn_seq(a, b).tiles + a.lead;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum * a.Hkv * a.row_tiles;
}

__device__ __forceinline__ int attn_live_ctas(const AttnArgs& a, long long total) {
  return total < a.ctas ? (int)total : a.ctas;
}
// Start of CTA c's range, and the CTA whose range holds place w.
__device__ __forceinline__ long long attn_first(long long total, int live, int c) { return c * total / live; }
__device__ __forceinline__ int attn_owner(long long total, int live, long long w) {
  return (int)(((w + 1) * live - 1) / total);
}

// A CTA's way through its range, one segment (part of a unit) after another.
struct AttnWalk {
  long long at, end;  // place of the next tile, end of the CTA's range
  int b, unit, tile;  // of the next tile: sequence, unit within it, tile within the unit
  AttnSeq seq;

  // Warp-collective.  False where the CTA has nothing to do.
  __device__ __forceinline__ bool start(const AttnArgs& a, int cta, int lane) {
    const long long total = attn_total(a, lane);
    const int live = attn_live_ctas(a, total);
    if (cta >= live) return false;
    at = attn_first(total, live, cta);
    end = attn_first(total, live, cta + 1);
    const int units = a.Hkv * a.row_tiles;
    long long before = 0;  // weight of the sequences before this group of 32
    for (int b0 = 0;; b0 += 32) {
      const long long mine = b0 + lane < a.B ? ((long long)attn_seq(a, b0 + lane).tiles + a.lead) * units : 0;
      long long incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + incl > at);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        before += __shfl_sync(0xffffffffu, incl - mine, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    seq = attn_seq(a, b);
    const long long rest = at - before;
    const int weight = seq.tiles + a.lead;
    unit = (int)(rest / weight);
    const int place = (int)(rest % weight);
    tile = place > a.lead ? place - a.lead : 0;
    at += tile + a.lead - place;
    return at < end;
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  // Tiles of the segment that starts at the next tile.
  __device__ __forceinline__ int segment() const {
    const long long left = end - at;
    return left < seq.tiles - tile ? (int)left : seq.tiles - tile;
  }
  __device__ __forceinline__ void advance(const AttnArgs& a, int count) {
    at += count;
    tile += count;
    if (tile < seq.tiles) return;
    tile = 0;
    at += a.lead;
    if (++unit < a.Hkv * a.row_tiles) return;
    unit = 0;
    if (++b < a.B) seq = attn_seq(a, b);
  }
};

// Visibility word of window row i (bit j: window position j), 0 for a dead row.
__device__ __forceinline__ uint32_t attn_word(const AttnArgs& a, int b, int i, int n) {
  if (i >= n) return 0u;
  const uint32_t live = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  if (a.mask != nullptr) return __ldg(a.mask + (size_t)b * a.S + i) & live;
  return (2u << i) - 1u;  // i = 31: 2 << 31 is 0, minus 1 is all ones
}

cudaError_t launch_attn_simple(int dtype, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_join(int dtype, const AttnArgs& a, cudaStream_t st);

constexpr int kAttnSimpleRows = 8;    // rows per tile of the CUDA-core kernel
constexpr int kAttnSimpleTile = 32;   // positions per tile of it

}  // namespace sdv

// Work split of the attention over a shared prefix: its kernels and the join.
//
// The prefix's positions, cut into tiles, are the same for every unit (kv head, group of query
// rows of the whole batch).  All units' tiles, laid end to end, are dealt in equal contiguous
// ranges to the CTAs of one wave; what a CTA computes of a unit it leaves as a partial (output
// relative to its own maximum, maximum, sum), the unit's k-th CTA in place k.  The prefix's length
// lives on the device; the split is a function of it and the shapes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_sched.cuh"
#include "mixing.h"
#include "split_math.cuh"

namespace sdv {

struct PrefixArgs {
  const void* q;
  long long q_stride;         // elements between tokens
  const void *k, *v;          // [n_pages][Hkv][page][D]
  const int32_t* table;       // [max_pages] of the prefix
  const int32_t* length;      // [1]
  float scale_log2;           // scale * log2(e)
  int tokens;                 // B * S
  int Hq, Hkv, G, D;
  int n_pages, page, max_pages;
  int tile_tokens, row_tile;  // tokens and query rows (tokens * G) of a row tile, at most 128
  int row_tiles, tiles_most;  // of a kv head; and what they would be if tiles held all rows they can
  int unit_tiles, units;      // row tiles of a unit (the last unit of a head may have fewer), units in all
  int tile;                   // positions per tile
  int sharers;                // places for partials of a unit
  int ctas;
  float* part_o;              // [units][sharers][unit_tiles][row_tile][D]
  float* part_ml;             // [units][sharers][unit_tiles][row_tile][2]: maximum (log2 domain), sum
  int* status;
  unsigned* passed;           // word that passes on what the first launch has waited for, or null
  DebugFault fault;
};

// The prefix's length as it counts, and its tiles.
__device__ __forceinline__ int prefix_length(const int32_t* length, int max_pages, int page, bool& bad) {
  const int n = *length;
  const long long cap = (long long)max_pages * page;
  const int most = cap > 0x7fffff00ll ? 0x7fffff00 : (int)cap, m = min(max(n, 0), most);
  bad = m != n;
  return m;
}
__device__ __forceinline__ int prefix_length(const PrefixArgs& a, bool& bad) {
  return prefix_length(a.length, a.max_pages, a.page, bad);
}
__device__ __forceinline__ int prefix_tiles(const PrefixArgs& a, int length) {
  return (int)(((unsigned)length + a.tile - 1) / (unsigned)a.tile);
}

// A CTA's way through its range, one segment (part of a unit) after another.
struct PrefixWalk {
  long long total, at, end;
  int live, tiles, unit, tile;
  __device__ __forceinline__ bool start(const PrefixArgs& a, int length, int cta) {
    tiles = prefix_tiles(a, length);
    total = (long long)tiles * a.units;
    live = attn_live_ctas(a.ctas, total);
    if (cta >= live) return false;
    at = attn_first(total, live, cta);
    end = attn_first(total, live, cta + 1);
    unit = (int)div_fast((unsigned long long)at, (unsigned long long)tiles);
    tile = (int)(at - (long long)unit * tiles);
    return at < end;
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ int segment() const { return (int)min(end - at, (long long)(tiles - tile)); }
  __device__ __forceinline__ void advance(int count) {
    at += count;
    tile += count;
    if (tile == tiles) {
      tile = 0;
      ++unit;
    }
  }
  // The place of CTA `cta`'s partial among its unit's.
  __device__ __forceinline__ int place(int cta) const { return cta - attn_owner(total, live, (long long)unit * tiles); }
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr float kPrefixDrop = 24.f;    // bits by which weights are lowered where the type has the range for it
constexpr int kPrefixSimpleRows = 64;  // rows per tile of the kernel for any head and page size
constexpr int kPrefixSimpleTile = 32;  // positions per tile of it

}  // namespace sdv

// Work split of the paged attention: shared by its kernels and the join.
//
// The cache positions of every (sequence, kv head, row tile) -- a unit -- are cut
// into tiles of `tile` positions; the tiles of all units, laid end to end, are
// dealt in equal contiguous ranges to the CTAs of one wave.  A unit weighs its
// tiles and `lead` more, the time that its queries, its last tile's cleaning and its
// outputs take in tiles' time, laid before its first tile: short contexts in a batch
// would otherwise all fall to a few CTAs.  Ragged contexts are then balanced to one
// tile whatever their lengths, and one long context spreads over the whole GPU.  A unit
// inside one CTA's range is finished there; the others leave (unnormalised output, max,
// sum) partials that are added in CTA order, by a launch of its own or, where they are
// small, by the last of the CTAs.  The lengths live on the device, so every warp that needs the split
// computes it from them (a warp-wide scan over the sequences), and the split is a
// function of lengths and shapes alone: results do not vary from run to run.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mixing.h"
#include "split_math.cuh"
#include "tc_util.cuh"

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
  int tile_wrows;           // tensor-core kernel: window rows of a row tile (row_tile / G)
  int tile;                 // cache positions per tile
  int lead;                 // weight of a unit beyond its tiles
  void* out;
  float* out32;             // or null: outputs in fp32 here instead
  float* lse;               // or null
  float* part_o;            // [2 * CTAs][D / 4][row_tile][4]
  float* part_ml;           // [2 * CTAs][row_tile][2]: max (log2 domain), sum
  unsigned* shared;         // arrivals at the unit whose first sharer a CTA is, a byte a CTA, or null: a join follows
  int* status;
  int ctas;                 // CTAs of the attention launch
  int slots, q_bufs;        // tensor-core kernel: ring slots, Q buffers
  DebugFault fault;         // its timeout path's test hook: a tile whose keys are never asked for
};

// Bytes of arrivals in the workspace's header, which alone is zero between calls of
// different operations.
constexpr int kAttnSharedAt = 64, kAttnSharedBytes = 192;

// One more of the CTAs first .. last; how many came before.  The last one's sets the count
// back to 0.
__device__ __forceinline__ unsigned attn_arrive(unsigned* shared, int first, int last) {
  const int at = 8 * (first & 3);
  unsigned* const word = shared + (first >> 2);
  const unsigned before = (atomicAdd(word, 1u << at) >> at) & 255u;
  if (before == (unsigned)(last - first)) atomicSub(word, (before + 1) << at);
  return before;
}

struct AttnSeq {
  int ctx, n;   // context positions, live window rows
  int tiles;    // tiles of each of its units (at least one: it writes the empty rows)
  bool bad;     // a length was out of range
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int c, int n) {
  AttnSeq s;
  const long long cap = (long long)a.max_pages * a.page;
  const int most = cap > 0x7fffff00ll ? 0x7fffff00 : (int)cap;
  s.ctx = min(max(c, 0), most);
  s.n = min(min(max(n, 0), a.S), most - s.ctx);
  s.bad = s.ctx != c || s.n != n;
  s.tiles = max(1, (int)(((unsigned)s.ctx + s.n + a.tile - 1) / (unsigned)a.tile));
  return s;
}
// (By coherent loads: some kernels read lengths beside the launch in front of them.)
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  return attn_seq(a, a.ctx[b], a.n_rows != nullptr ? a.n_rows[b] : a.S);
}

__device__ __forceinline__ int attn_live_ctas(int ctas, long long total) { return total < ctas ? (int)total : ctas; }
// Start of CTA c's range, and the CTA whose range holds place w.
__device__ __forceinline__ long long attn_first(long long total, int live, int c) { return muldiv(total, c, live); }
__device__ __forceinline__ int attn_owner(long long total, int live, long long w) {
  return (int)div_fast((unsigned long long)(w + 1) * (unsigned)live - 1, total);
}

// A CTA's way through its range, one segment (part of a unit) after another.
struct AttnWalk {
  long long total, at, end;  // all weight; place of the next tile, end of the CTA's range
  int live;                  // CTAs with a range
  int b, unit, tile;  // of the next tile: sequence, unit within it, tile within the unit
  AttnSeq seq;
  int next_ctx, next_n;  // lengths of sequence b + 1, loaded ahead of their use

  // Warp-collective.  False where the CTA has nothing to do.
  __device__ __noinline__ bool start(const AttnArgs& a, int cta, int lane) {
    const int units = a.Hkv * a.row_tiles;
    // the first 32 sequences' weights serve for the total and for the search
    const long long w0 = lane < a.B ? ((long long)attn_seq(a, lane).tiles + a.lead) * units : 0;
    total = w0;
    for (int s = lane + 32; s < a.B; s += 32) total += ((long long)attn_seq(a, s).tiles + a.lead) * units;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    live = attn_live_ctas(a.ctas, total);
    if (cta >= live) return false;
    at = attn_first(total, live, cta);
    end = attn_first(total, live, cta + 1);
    long long before = 0;  // weight of the sequences before this group of 32
    for (int b0 = 0;; b0 += 32) {
      const long long mine = b0 == 0 ? w0 : b0 + lane < a.B ? ((long long)attn_seq(a, b0 + lane).tiles + a.lead) * units : 0;
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
    load_next(a);
    const long long rest = at - before;
    const int weight = seq.tiles + a.lead;
    unit = (int)muldiv(rest, 1, weight);
    const int place = (int)(rest - (long long)unit * weight);
    tile = place > a.lead ? place - a.lead : 0;
    at += tile + a.lead - place;
    return at < end;
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  // The first and the last CTA with tiles of the unit that the next tile is in.
  __device__ __forceinline__ void sharers(int& first, int& last) const {
    first = attn_owner(total, live, at - tile);
    last = attn_owner(total, live, at - tile + seq.tiles - 1);
  }
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
    if (++b < a.B) {
      seq = attn_seq(a, next_ctx, next_n);
      load_next(a);
    }
  }
  __device__ __forceinline__ void load_next(const AttnArgs& a) {
    const bool is = b + 1 < a.B;
    next_ctx = is ? a.ctx[b + 1] : 0;
    next_n = is && a.n_rows != nullptr ? a.n_rows[b + 1] : a.S;
  }
};

// What is not finite among the values of some positions: the sum of infinities and NaN is
// told by which of them there are.
constexpr uint32_t kOddPlus = 1, kOddMinus = 2, kOddNan = 4;
__device__ __forceinline__ float odd_value(uint32_t odd) {
  if ((odd & kOddNan) || (odd & (kOddPlus | kOddMinus)) == (kOddPlus | kOddMinus)) return __int_as_float(0x7fc00000);
  return odd & kOddPlus ? INFINITY : odd & kOddMinus ? -INFINITY : 0.f;
}

// x times a softmax factor.  ODD: an infinity or NaN stays what it is, as the factor is
// above 0 if not in 32 bits.
template <bool ODD>
__device__ __forceinline__ float weighted(float x, float f) {
  return !ODD || fabsf(x) < INFINITY ? x * f : x;
}

// Softmax sums of four columns, partial by partial (m: reference maximum in the log2
// domain, l and o relative to it; a partial that saw nothing is (-inf, 0)).
struct AttnSum {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <bool ODD>
  __device__ __forceinline__ void add(float m2, float l2, const float4& x) {
    if (m2 == -INFINITY && l2 == 0.f) return;
    const float mn = fmaxf(m, m2), f = exp2f(m - mn), f2 = exp2f(m2 - mn);
    m = mn;
    l = l * f + l2 * f2;
    o.x = weighted<ODD>(o.x, f) + weighted<ODD>(x.x, f2);
    o.y = weighted<ODD>(o.y, f) + weighted<ODD>(x.y, f2);
    o.z = weighted<ODD>(o.z, f) + weighted<ODD>(x.z, f2);
    o.w = weighted<ODD>(o.w, f) + weighted<ODD>(x.w, f2);
  }
  __device__ __forceinline__ bool finite() const {
    return fabsf(o.x) < INFINITY && fabsf(o.y) < INFINITY && fabsf(o.z) < INFINITY && fabsf(o.w) < INFINITY;
  }
  __device__ __forceinline__ float lse() const {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
};

// The partials of CTAs from .. to of a unit that CTA `first` begins, in their order, eight
// loads in flight; ml and po at the row (and columns) in slot 0, whose steps follow.
template <bool ODD>
__device__ __forceinline__ AttnSum attn_sum_parts(const float2* ml, const float4* po, int ml_step, size_t po_step,
                                                  int first, int from, int to) {
  AttnSum sum;
  for (int c = from; c <= to; c += 8) {
    float2 s[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s[k] = make_float2(-INFINITY, 0.f);
      if (c + k <= to) {
        const size_t slot = 2 * (size_t)(c + k) + (c + k == first);
        s[k] = __ldcg(ml + slot * ml_step);
        x[k] = __ldcg(po + slot * po_step);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum.add<ODD>(s[k].x, s[k].y, x[k]);
  }
  return sum;
}
static __device__ __noinline__ AttnSum attn_sum_odd_parts(const float2* ml, const float4* po, int ml_step,
                                                          size_t po_step, int first, int from, int to) {
  return attn_sum_parts<true>(ml, po, ml_step, po_step, first, from, to);
}

// Visibility word of window row i (bit j: window position j), 0 for a dead row.
__device__ __forceinline__ uint32_t attn_word(const AttnArgs& a, int b, int i, int n) {
  if (i >= n) return 0u;
  const uint32_t live = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  if (a.mask != nullptr) return __ldg(a.mask + (size_t)b * a.S + i) & live;
  return (2u << i) - 1u;  // i = 31: 2 << 31 is 0, minus 1 is all ones
}

// Visibility of 32 positions from p on: context positions, the window's by `word`.
__device__ __forceinline__ uint32_t attn_visible(int p, int ctx, uint32_t word) {
  const int nc = min(max(ctx - p, 0), 32);
  uint32_t bits = nc >= 32 ? 0xffffffffu : (1u << nc) - 1u;
  if (p < ctx) bits |= nc >= 32 ? 0u : word << nc;
  else bits |= p - ctx < 32 ? word >> (p - ctx) : 0u;
  return bits;
}

// Four columns of an output: as the 16-bit type, or fp32 where another launch goes on with them.
template <typename T>
__device__ __forceinline__ void attn_store4(const AttnArgs& a, long long at, float x, float y, float z, float w) {
  if (a.out32 != nullptr)
    *reinterpret_cast<float4*>(a.out32 + at) = make_float4(x, y, z, w);
  else
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at) = make_uint2(pack16<T>(x, y), pack16<T>(z, w));
}

cudaError_t launch_attn_simple(int dtype, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_join(int dtype, const AttnArgs& a, cudaStream_t st);

constexpr int kAttnSimpleRows = 8;    // rows per tile of the CUDA-core kernel
constexpr int kAttnSimpleTile = 32;   // positions per tile of it

}  // namespace sdv

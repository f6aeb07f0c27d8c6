// Attention of a verify window over a paged cache on the 5th-generation tensor
// cores (sm_103a): sdv_paged_attn for head sizes 64, 128 and 256.
//
// Per row r of a kv head's S * G query rows and cache position p:
//   s = q_r . k_p;  m = running max of scale s;  P = 2^((scale s - m) log2 e)
//   l += sum P;  O = O 2^(m_old - m) + P V;  out = O / l
// One pass over keys and values.  A unit's rows (at most 128) are one MMA tile, so
// a window reads the cache once for all its rows and heads of a group: 4 D flops
// per row and position against 4 D bytes per position, far inside the tensor
// cores' rate for any window -- reading the cache bounds it.
//
// One persistent CTA per SM walks an equal share of all tiles (attn_sched.cuh).
// Warp roles:
//   warps 0, 6  TMA producers of keys and of values: a lane per (page, 64-element
//               block) box; the tiles alternate through a ring of equal slots;
//   warp 1      allocates tensor memory, one lane issues the MMAs:
//               S = Q K^T (both K-major in shared memory), one tile ahead of
//               O += P V (P in tensor memory, V as it lies in the cache, MN-major);
//   warps 2-5   softmax, a thread per row: S from tensor memory, P back into its
//               columns; they also write the outputs;
//   warp 7      walks the units ahead of the others: stages a segment's Q (two
//               buffers of the row tile's rows) and what it is, so that short
//               contexts follow each other without a load in between.
// Few rows (single tokens, short windows) stand four times in
// the MMA's 128, and each softmax warp takes a quarter of a tile's positions for all
// of them, the other positions' weights being zero in its copy: the softmax of a tile
// then takes a quarter of the time, and the four (m, l, O) are merged at the end.
//
// The reference maximum moves only when it grows by more than 2^8 (the sum and
// output stay exact relative to it), so O in tensor memory is rescaled rarely.
// fp16's P carries a factor 2^6: with it the weights down to 2^-20 of the row's largest
// stay in the normal range, and 2^14 is the most it can reach.  bf16's, with the range of
// fp32, carries 2^-8 and never passes 1, so that values of any size overflow no sooner than
// in a plain sum with weights up to 1.  Rounding P to
// the 16-bit type is the one rounding inside the sum (the sum l takes P before
// it); it is what a matrix instruction on 16-bit values needs.
//
// Pages past the end and absent ones are boxes past the tensor map's end: the copy
// fills zeros.  In tiles that reach past the context V is cleaned in shared memory
// before P V: what the last page holds behind the end becomes zeros, and a window
// row's infinities and NaN are zeroed and noted, then added at the end to the rows
// that do see them -- 0 * inf would otherwise reach the others.  Every row sees the
// context, but in 16 bits with weights that may be 0 (spread rows: are 0 in three copies
// of four), so there too 0 * inf makes NaN what is an infinity: an output that is not
// finite makes the warp look at the segment's values themselves.
//
// Measured, a call: one token over 500,000 positions of 8 heads of 128: 291 us, 7.0 TB/s
// of cache; 48 sequences of up to 16,000: 93 us, 5.9 TB/s.  What shorter calls add is the
// start (4 us until the first tile is there: the walk, cold instructions, the first read)
// and the end.  17 rows of 8 heads a cache head of 256 over 32,768 positions: 32.1 us,
// 2.1 TB/s: 136 rows are two tiles, and a tile of 64 positions is 2100 cycles, of which
// the MMAs' issue takes 1700 (S reads Q and K from shared memory, 6 KB for 64 cycles of
// products).  One token over 613 positions: 10.9 us, all of it start and end.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "attn_sched.cuh"
#include "attn_tc.h"
#include "mixing.h"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnSmem = 232448 - kWaitLimitBytes;  // all of an SM's: one CTA, one tensor-memory allocation
constexpr uint64_t kAttnDrainNs = 100000000ull;  // 0.1 s: in-flight work at teardown
constexpr int kMaxSlots = 8;
constexpr int kSpreadRows = 32;                  // rows that can stand four times in the MMA tile
constexpr int kSpreadMost = 2048;                // and do up to this many elements of an output
// The merge buffer: 4 copies of up to 32 rows, at least 32 columns and 4 of padding.
constexpr int kMergeBytes = 4 * kSpreadRows * (32 + 4) * 4;

// What a segment is, from warp 7 to the MMA and softmax warps.
struct AttnSegment {
  int count;  // tiles; 0: no more segments
  int b, h, r0, tile, ctx, n;
  int flags;           // 1: the unit ends here; 2: a table entry of the segment cannot be followed
  int first, last;     // the CTAs that share the unit
  uint32_t words[32];  // visibility of the window rows
  int pad[2];
};

// Shared memory: the Q buffers, the ring, small things.  The MMA reads 128 rows of a
// Q buffer; what lies behind the staged ones feeds rows that nobody looks at.
template <int D, bool SPREAD>
struct AttnPlan {
  static constexpr int TK = attn_tc_tile(D);
  static constexpr int kBlocks = D / 64;
  static constexpr int kSlot = TK * D * 2;
  static constexpr int kNumBars = 2 * kMaxSlots + 2 + 2 + 2 + 2 + 1 + 1 + 1 + 1;  // the last for alignment
  static constexpr int kMerge = SPREAD ? kMergeBytes + 4 * kSpreadRows * 8 + kSpreadRows * 4 : 0;
  static constexpr int kSmall = 2 * D * 4 + kNumBars * 8 + 2 * (int)sizeof(AttnSegment) + 32 + kMerge;
  static constexpr int kS = 0;       // tensor-memory columns: two score tiles (P inside),
  static constexpr int kO = 2 * TK;  // then the output
  static_assert(kO + D <= 512, "tensor memory");
  static_assert((2 * D * 4 + kNumBars * 8) % 16 == 0 && sizeof(AttnSegment) % 16 == 0, "16-byte merge rows");
  // rows between a Q buffer's 64-element blocks, bytes between the buffers, all buffers
  __host__ __device__ static int q_rows(int row_tile) { return SPREAD ? 128 : (row_tile + 7) / 8 * 8; }
  __host__ __device__ static int q_step(int row_tile) {
    return SPREAD ? (row_tile + 7) / 8 * 1024 : q_rows(row_tile) * D * 2;
  }
  __host__ __device__ static int q_bytes(int row_tile, int q_bufs) {
    return SPREAD ? 128 * D * 2 : q_bufs * q_step(row_tile);
  }
  static int slots(int row_tile, int q_bufs) {
    const int n = (kAttnSmem - 1024 - kSmall - q_bytes(row_tile, q_bufs)) / kSlot;
    return n < kMaxSlots ? n : kMaxSlots;
  }
};

// Sum of the values that are not finite in column d of the window positions `bits`.
template <typename T>
__device__ __noinline__ float poison_of(const AttnArgs& a, const int32_t* trow, int h, int ctx, uint32_t bits, int d) {
  float sum = 0.f;
  for (; bits; bits &= bits - 1) {
    const int p = ctx + __ffs(bits) - 1;
    const int id = __ldg(trow + p / a.page);  // in range: the position's page was followed
    sum += (float)static_cast<const T*>(a.v)[(((long long)id * a.Hkv + h) * a.page + p % a.page) * a.D + d];
  }
  return sum;
}

// The infinities and NaN of positions from .. to - 1 of the context, by the whole warp in
// 16-byte loads: lane l gets columns 8 (l % (D / 8)) .. + 7, four bits each.
template <typename T, int D>
__device__ __noinline__ uint32_t odd_columns(const AttnArgs& a, const int32_t* trow, int h, int from, int to) {
  constexpr int C = D / 8;
  const int lane = threadIdx.x & 31;
  uint32_t odd = 0;
#pragma unroll 4
  for (int p = from + lane / C; p < to; p += 32 / C) {
    const int id = __ldg(trow + p / a.page);
    if (id < 0 || id >= a.n_pages) continue;
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.v) +
                          (((long long)id * a.Hkv + h) * a.page + p % a.page) * C + lane % C);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      if (!(nonfinite16<T>(xs[z >> 1]) >> (z & 1) & 1)) continue;
      const float y = z & 1 ? unpack16<T>(xs[z >> 1]).y : unpack16<T>(xs[z >> 1]).x;
      odd |= (y != y ? kOddNan : y > 0.f ? kOddPlus : kOddMinus) << (4 * z);
    }
  }
#pragma unroll
  for (int off = C; off < 32; off <<= 1) odd |= __shfl_xor_sync(0xffffffffu, odd, off);
  return odd;
}
// Whether one of N floats is not finite: 0 times it is NaN then, and so is the sum.
template <int N>
__device__ __forceinline__ bool any_odd(const uint32_t* x) {
  f32x2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = pair2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < N; e += 2)
    sum[e / 2 & 3] = fma2(pair2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), pair2(0.f, 0.f), sum[e / 2 & 3]);
  const float2 a = unpair2(sum[0]), b = unpair2(sum[1]), c = unpair2(sum[2]), d = unpair2(sum[3]);
  return ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y)) != 0.f;
}
// Of column d, from the lane that has it.
__device__ __forceinline__ uint32_t odd_of(uint32_t odd, int d) {
  return __shfl_sync(0xffffffffu, odd, d >> 3) >> (4 * (d & 7)) & 7u;
}

// Visibility of 32 positions from p on: context positions, the window's by `word`.
__device__ __forceinline__ uint32_t attn_visible(int p, int ctx, uint32_t word) {
  const int nc = min(max(ctx - p, 0), 32);
  uint32_t bits = nc >= 32 ? 0xffffffffu : (1u << nc) - 1u;
  if (p < ctx) bits |= nc >= 32 ? 0u : word << nc;
  else bits |= p - ctx < 32 ? word >> (p - ctx) : 0u;
  return bits;
}

// x / g for 0 <= x < 2^16 and 1 <= g <= 128, from 1 / g: x + 1/2 is at least 1/(2 g)
// of a quotient away from the next, more than the error of two roundings.
__device__ __forceinline__ int small_div(int x, float inv_g) { return (int)(((float)x + 0.5f) * inv_g); }

template <typename T, int D, bool SPREAD>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs a) {
  using PL = AttnPlan<D, SPREAD>;
  constexpr int TK = PL::TK;
  constexpr int CW = SPREAD ? TK / 4 : TK;  // score columns of a softmax warp
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kLift = kBf16 ? -8.f : 6.f;  // P's power of two
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const sb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NS = a.slots, q_bufs = a.q_bufs;
  const int q_block = PL::q_rows(a.row_tile) * 128, q_step = PL::q_step(a.row_tile);
  const uint32_t ring = base + PL::q_bytes(a.row_tile, q_bufs);
  const uint32_t small = ring + NS * PL::kSlot, bars = small + 2 * D * 4;
  uint8_t* const sp = sb + (small - base);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxSlots + s); };
  constexpr int kB = 2 * kMaxSlots;
  auto s_full = [&](int i) { return bars + 8u * (kB + i); };
  auto p_ready = [&](int i) { return bars + 8u * (kB + 2 + i); };
  auto q_full = [&](int i) { return bars + 8u * (kB + 4 + i); };
  auto q_free = [&](int i) { return bars + 8u * (kB + 6 + i); };
  const uint32_t pv_done = bars + 8u * (kB + 8), drain = pv_done + 8, rows_met = pv_done + 16;
  uint32_t* const poison = reinterpret_cast<uint32_t*>(sp);  // [2][D]
  AttnSegment* const segs = reinterpret_cast<AttnSegment*>(sp + 2 * D * 4 + PL::kNumBars * 8);
  // tmem base, poison seen [2], shared units: arrivals made and whether this was the last;
  // spread rows: 1 + the last segment with an output that is not finite
  volatile uint32_t* const misc = reinterpret_cast<uint32_t*>(segs + 2);
  float* const merge = const_cast<float*>(reinterpret_cast<volatile float*>(misc + 8));
  float2* const mstat = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(merge) + kMergeBytes);  // [4][32]
  uint32_t* const mword = reinterpret_cast<uint32_t*>(mstat + 4 * kSpreadRows);
  const int nq = SPREAD ? 4 : (a.row_tile + 31) / 32;  // softmax warps with rows

  if (warp == 1) {
    tmem_alloc(smem_addr(const_cast<uint32_t*>(misc)), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    set_wait_limit(a.fault);
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_ready(i), nq);
      mbar_init(q_full(i), 1);
      mbar_init(q_free(i), 1 + nq);
    }
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    mbar_init(rows_met, nq);
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  for (int e = threadIdx.x; e < 2 * D; e += kAttnThreads) poison[e] = 0;
  if (threadIdx.x < 4) misc[1 + threadIdx.x] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = misc[0];
  griddep_wait();
  griddep_launch_dependents();
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = mbar_wait_warp(bar, parity, a.status);
    return ok;
  };
  // P V products complete in tile order.  Each role that needs them waits for every
  // one, in order, and before the next can be issued: a parity wait on an older one
  // would otherwise meet the newer phase of the same parity.
  int pv_seen = 0;
  auto pv_wait = [&](int tiles) {
    for (; pv_seen < tiles; ++pv_seen)
      if (!await(pv_done, pv_seen & 1)) return false;
    return true;
  };
  // segment s is in Q buffer and note s % q_bufs
  auto seg_buf = [&](int s) { return q_bufs == 2 ? s & 1 : 0; };
  auto seg_parity = [&](int s) { return (q_bufs == 2 ? s >> 1 : s) & 1; };

  if (warp == 0 || warp == 6) {
    // ---- producers: the warp's tile i takes ring place 2i (keys) or 2i + 1 (values) ----
    AttnWalk first;
    const bool values = warp == 6;
    const int box = min(a.page, TK), chunks = TK / box;  // rows per box, pages (or page parts) per tile
    const int page_log = 31 - __clz(a.page);
    const int beyond = a.n_pages * a.Hkv * a.page;       // a row past the tensor map's end: zeros
    const uint64_t policy = a.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_normal();
    const int cb = lane % PL::kBlocks, chunk = lane / PL::kBlocks;
    const bool mine = chunk < chunks;
    const uint32_t dst = ring + cb * (TK * 128) + chunk * box * 128;
    int asked = 0;  // tiles
    int slot = values ? 1 : 0, use = 0;  // ring place: slot, and how often the ring has been passed
    bool more = first.start(a, blockIdx.x, lane);
    AttnWalk w = first;
    while (more) {
      const int count = w.segment();
      const int h = w.unit / a.row_tiles;
      const int total = w.seq.ctx + w.seq.n;
      const int32_t* const row = a.table + (size_t)w.b * a.max_pages;
      auto page_of = [&](int t) {
        const int p = t * TK + chunk * box;
        return mine && p < total ? __ldg(row + (p >> page_log)) : -1;
      };
      // table entries are loaded four tiles ahead
      const int end = w.tile + count;
      int ids[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ids[k] = w.tile + k < end ? page_of(w.tile + k) : -1;
      for (int t0 = w.tile; ok && t0 < end; t0 += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + k;
          if (t >= end) break;
          const int id = ids[k], p = t * TK + chunk * box;
          ids[k] = t + 4 < end ? page_of(t + 4) : -1;
          const int y = id >= 0 && id < a.n_pages ? (id * a.Hkv + h) * a.page + (p & (a.page - 1)) : beyond;
          if (use > 0 && !await(empty(slot), (use - 1) & 1)) break;
          if (values || ++asked != a.fault.withhold) {
            if (lane == 0) mbar_arrive_expect_tx(full(slot), PL::kSlot);
            __syncwarp();
            if (mine)
              tma_load_2d(dst + slot * PL::kSlot, values ? &maps.v : &maps.k, cb * 64, y, full(slot), policy);
          }
          asked += values;
          slot += 2;
          if (slot >= NS) {
            slot -= NS;
            ++use;
          }
        }
      }
      if (!ok) break;
      w.advance(a, count);
      more = w.more();
    }
    // The copies into places that are not taken again have to land before the CTA ends,
    // whoever else gives up waiting for them, and when: those in the ring's last NS places, or,
    // if it is this warp that gave up, any of its last (one whose place the other producer
    // has taken since had landed; the wait for it runs out).
    for (int i = max(asked - NS, 0); i < asked; ++i) {
      const int place = 2 * i + values;
      if ((ok && place < 2 * asked - NS) || (!values && i + 1 == a.fault.withhold)) continue;
      mbar_wait_bounded(full(place % NS), (place / NS) & 1, kAttnDrainNs);
    }
  } else if (warp == 7) {
    // ---- segments: Q by TMA, and what the others need to know ----
    AttnWalk start;
    const int page_log = 31 - __clz(a.page);
    const uint64_t policy = l2_policy_normal();
    constexpr int kCopies = SPREAD ? 4 : 1;
    int asked = 0;        // segments
    bool closed = false;  // the note behind the last one is out, in the buffer of one that has been read
    bool more = start.start(a, blockIdx.x, lane);
    AttnWalk w = start;
    for (int sg = 0;; ++sg) {
      const int buf = seg_buf(sg);
      if (sg >= q_bufs && !await(q_free(buf), seg_parity(sg - q_bufs))) break;
      AttnSegment& g = segs[buf];
      if (!more) {
        if (lane == 0) {
          g.count = 0;
          mbar_arrive(q_full(buf));
        }
        closed = true;
        break;
      }
      const int count = w.segment();
      const int h = w.unit / a.row_tiles, rt = w.unit - h * a.row_tiles;
      // the segment's table entries
      const int last = min((w.tile + count) * TK, w.seq.ctx + w.seq.n) - 1;  // its last position
      const int32_t* const row = a.table + (size_t)w.b * a.max_pages;
      bool absent = false;
      if (last >= 0) {
#pragma unroll 4
        for (int e = (w.tile * TK >> page_log) + lane; e <= last >> page_log; e += 32) {
          const int id = __ldg(row + e);
          absent |= id < 0 || id >= a.n_pages;
        }
      }
      if (lane < a.S) g.words[lane] = attn_word(a, w.b, lane, w.seq.n);
      absent = __any_sync(0xffffffffu, absent);
      __syncwarp();
      if (lane == 0) {
        g.count = count;
        g.b = w.b;
        g.h = h;
        g.r0 = rt * a.row_tile;
        g.tile = w.tile;
        g.ctx = w.seq.ctx;
        g.n = w.seq.n;
        g.flags = (w.tile + count == w.seq.tiles ? 1 : 0) | (absent ? 2 : 0);
        w.sharers(g.first, g.last);
        if (w.seq.bad || absent) atomicOr(a.status, kDevErrIndex);
        mbar_arrive_expect_tx(q_full(buf), kCopies * PL::kBlocks * a.row_tile * 128);
      }
      __syncwarp();
      if (lane < kCopies * PL::kBlocks)  // rows past n_rows or S: whatever lies there, for rows that give 0
        tma_load_3d(base + buf * q_step + (lane / kCopies) * q_block + lane % kCopies * 4096, &maps.q,
                    lane / kCopies * 64, h * a.G, w.b * a.S + rt * a.tile_wrows, q_full(buf), policy);
      ++asked;
      w.advance(a, count);
      more = w.more();
    }
    for (int s = max(asked - q_bufs + closed, 0); s < asked; ++s)  // as the producers do
      mbar_wait_bounded(q_full(seg_buf(s)), seg_parity(s), kAttnDrainNs);
  } else if (warp == 1) {
    // ---- MMA: every lane keeps the same state, one elected lane issues ----
    constexpr uint32_t id_pv = idesc_16_f32(kBf16, 128, D, false, true);
    // a negative scale negates Q in the product: the maximum is then over scale * s
    const uint32_t id_qk = idesc_16_f32(kBf16, 128, TK, false, false) | (a.scale_log2 < 0.f ? kIdescNegateA : 0u);
    int ks = 0, ku = 0, vs = 1, vu = 0;  // ring places of the next keys and values
    auto step2 = [&](int& s, int& u) {
      s += 2;
      if (s >= NS) {
        s -= NS;
        ++u;
      }
    };
    auto qk = [&](int i, int buf, bool last) {  // S of tile i; last: of its segment
      if (!pv_wait(i - 1)) return;              // the P that held these columns has been read
      if (!await(full(ks), ku & 1)) return;
      tc_fence_after();
      const uint64_t qd = smem_desc_sw128(base + buf * q_step, 16, 1024);
      const uint64_t kd = smem_desc_sw128(ring + ks * PL::kSlot, 16, 1024);
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        tc_mma4_ss(tm + PL::kS + (i & 1) * TK, qd + (uint32_t)(j * (q_block >> 4)), kd + j * (TK * 128 >> 4), id_qk,
                   j > 0);
      tc_commit_elect(s_full(i & 1));
      tc_commit_elect(empty(ks));
      if (last) tc_commit_elect(q_free(buf));
      step2(ks, ku);
    };
    int i = 0;
    for (int sg = 0; ok; ++sg) {
      const int buf = seg_buf(sg);
      if (!await(q_full(buf), seg_parity(sg))) break;
      const int count = __reduce_max_sync(0xffffffffu, *const_cast<volatile int*>(&segs[buf].count));
      if (count == 0) break;
      tc_fence_after();
      qk(i, buf, count == 1);
      for (int t = 0; ok && t < count; ++t, ++i) {
        if (t + 1 < count) qk(i + 1, buf, t + 2 == count);
        if (!await(full(vs), vu & 1) || !await(p_ready(i & 1), (i >> 1) & 1) || !pv_wait(i)) break;
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128(ring + vs * PL::kSlot, TK * 128, 1024);
#pragma unroll
        for (int j = 0; j < TK / 64; ++j)
          tc_mma4_ts(tm + PL::kO, tm + PL::kS + (i & 1) * TK + j * 32, vd + j * (4 * 2048 >> 4), id_pv, t > 0 || j > 0);
        tc_commit_elect(pv_done);
        tc_commit_elect(empty(vs));
        step2(vs, vu);
      }
    }
    // every MMA has ended before tensor memory is freed
    tc_commit_elect(drain);
    mbar_wait_bounded(drain, 0, kAttnDrainNs);
  } else if ((warp & 3) < nq) {
    // ---- softmax and outputs: a thread per row ----
    const int quarter = warp & 3, r = SPREAD ? lane : quarter * 32 + lane;
    const uint32_t tq = tm + ((uint32_t)(quarter * 32) << 16);
    const int box = min(a.page, TK);
    // a scale of 0 becomes one that leaves every finite score at 0 (times 0 a masked
    // score would be NaN)
    const float c = fmaxf(fabsf(a.scale_log2), 1e-36f);
    // the softmax warps meet (a bounded wait, as every one here)
    uint32_t meetings = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_met);
      return await(rows_met, meetings++ & 1);
    };
    const float inv_g = 1.f / (float)a.G;
    int i = 0, vs = 1, vu = 0;
    for (int sg = 0; ok; ++sg) {
      const int buf = seg_buf(sg);
      if (!await(q_full(buf), seg_parity(sg))) break;
      const AttnSegment& g = segs[buf];
      const int count = g.count;
      if (count == 0) break;
      const int b = g.b, tile0 = g.tile, ctx = g.ctx, n = g.n, h = g.h, r0 = g.r0, total = ctx + n;
      const bool some_absent = g.flags & 2, ends = g.flags & 1;
      const int g_first = g.first, g_last = g.last;
      const int nr = min(a.row_tile, a.rows - r0);
      const int row = r0 + r, wr = small_div(row, inv_g);
      const bool live = r < nr && wr < n;
      const uint32_t word = live ? g.words[wr] : 0u;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_free(buf));
      const int32_t* const trow = a.table + (size_t)b * a.max_pages;
      uint32_t* const pois = poison + (sg & 1) * D;
      float m = -INFINITY, l = 0.f;  // reference maximum (log2 domain), sum of P relative to it
      for (int t = tile0; t < tile0 + count; ++t, ++i) {
        const int p0 = t * TK;
        const bool edge = some_absent || p0 + TK > ctx;
        if (!await(s_full(i & 1), (i >> 1) & 1)) break;
        tc_fence_after();
        const uint32_t ts = tq + PL::kS + (i & 1) * TK;
        const int j0 = SPREAD ? quarter * CW : 0;  // the warp's first column
        uint32_t sr[CW];
        if constexpr (CW == 16) {
          tmem_ld16(ts + j0, sr);
        } else {
#pragma unroll
          for (int j = 0; j < CW; j += 32) tmem_ld32(ts + j0 + j, sr + j);
        }
        tmem_wait_ld();
        if (edge) {
          uint32_t absent = 0;  // pages of the tile that cannot be followed, a bit each
          if (some_absent) {
            const int p = p0 + lane * box;
            bool gone = false;
            if (lane * box < TK && p < total) {
              const int id = __ldg(trow + p / a.page);
              gone = id < 0 || id >= a.n_pages;
            }
            absent = __ballot_sync(0xffffffffu, gone);
          }
#pragma unroll
          for (int j = 0; j < CW; j += 32) {
            uint32_t bits = live ? attn_visible(p0 + j0 + j, ctx, word) : 0u;
            if (absent != 0) {
              for (int e = 0; e < 32; e += 8)
                if (absent >> ((j0 + j + e) / box) & 1) bits &= ~(0xffu << e);
            }
#pragma unroll
            for (int e = 0; e < (CW < 32 ? CW : 32); ++e)
              if (!(bits >> e & 1)) sr[j + e] = 0xff800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = __uint_as_float(sr[j]);
#pragma unroll
        for (int j = 4; j < CW; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(sr[j]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool grow = live && mt > m + 8.f;  // also from -inf to any number
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow && m != -INFINITY ? exp2_approx(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (t > tile0 && __any_sync(0xffffffffu, f != 1.f)) {
            if (!pv_wait(i)) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
              uint32_t o[32];
              tmem_ld32(tq + PL::kO + j, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tq + PL::kO + j, o);
            }
          }
        }
        const float ref = m == -INFINITY ? -kLift : m - kLift;
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < CW; j += 2) {
          const float e0 = exp2_approx(fmaf(__uint_as_float(sr[j]), c, -ref));
          const float e1 = exp2_approx(fmaf(__uint_as_float(sr[j + 1]), c, -ref));
          l4[j & 2] += e0;
          l4[(j & 2) + 1] += e1;
          sr[j >> 1] = pack16<T>(e0, e1);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        if constexpr (SPREAD) {  // the other positions' weights are zero in this copy of the rows
          const uint32_t zero[16] = {};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (CW == 32) {
              if (j == quarter) tmem_st16(ts + j * 16, reinterpret_cast<const uint32_t(&)[16]>(sr));
              else tmem_st16(ts + j * 16, zero);
            } else {
              tmem_st8(ts + j * 8, j == quarter ? sr : zero);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < CW / 2; j += 32) tmem_st32(ts + j, sr + j);
        }
        if (edge) {
          // clean V from the first window row to the end of the last page
          const int from = max(ctx - p0, 0), to = min(TK, (int)(((uint32_t)total + a.page - 1) / a.page * a.page - p0));
          if (from < to) {
            if (!await(full(vs), vu & 1)) break;
            const uint32_t vb = ring + vs * PL::kSlot;
            bool wrote = false;
            for (int e = from * (D / 8) + quarter * 32 + lane; e < to * (D / 8); e += 32 * nq) {
              const int j = e / (D / 8), ch = e % (D / 8), p = p0 + j;
              const uint32_t at = vb + (ch >> 3) * (TK * 128) + swz128(j, ch & 7);
              if (p >= total) {
                sts128(at, make_uint4(0, 0, 0, 0));
                wrote = true;
              } else {
                const uint4 x = lds128(at);
                uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t bad = 0;
#pragma unroll
                for (int z = 0; z < 4; ++z) bad |= nonfinite16<T>(xs[z]) << (2 * z);
                if (bad) {
#pragma unroll
                  for (int z = 0; z < 8; ++z)
                    if (bad >> z & 1) {
                      atomicOr(pois + ch * 8 + z, 1u << (p - ctx));
                      xs[z >> 1] &= z & 1 ? 0x0000ffffu : 0xffff0000u;
                    }
                  sts128(at, make_uint4(xs[0], xs[1], xs[2], xs[3]));
                  misc[1 + (sg & 1)] = 1;
                  wrote = true;
                }
              }
            }
            if (wrote) fence_proxy_async_smem();
          }
        }
        vs += 2;
        if (vs >= NS) {
          vs -= NS;
          ++vu;
        }
        if (!pv_wait(i)) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready(i & 1));
      }
      if (!ok) break;
      const bool starts = tile0 == 0, final = starts && ends;
      const size_t slot = 2 * (size_t)blockIdx.x + (starts ? 1 : 0);
      const float mm = m == -INFINITY ? -INFINITY : m - kLift;
      if (!pv_wait(i)) break;  // every warp has delivered its last P: it is past the last segment's merge
      tc_fence_after();
      const bool poisoned = misc[1 + (sg & 1)] != 0;  // noted before the P that this P V waited for
      const int ctx0 = min(tile0 * TK, ctx), ctx1 = min((tile0 + count) * TK, ctx);  // the segment's part of the context
      uint32_t odd = 0;  // what is not finite there, once looked at
      bool looked = false;
      if constexpr (SPREAD) {
        // Merge the four copies: M = max m_q, out = sum 2^(m_q - M) O_q / sum 2^(m_q - M) l_q,
        // in rounds of the columns that the merge buffer holds.
        const int cols = min(D, (kMergeBytes / 16 / a.row_tile - 4) / 32 * 32), pad = cols + 4;  // 32 at least
        if (lane < nr) mstat[quarter * kSpreadRows + lane] = live ? make_float2(mm, l) : make_float2(-INFINITY, 0.f);
        if (quarter == 0) mword[lane] = word;
        for (int j0 = 0; j0 < D; j0 += cols) {
          if (j0 > 0 && !meet()) break;  // the last round has been read
          const int now = min(cols, D - j0);
#pragma unroll 1
          for (int j = 0; j < now; j += 64) {
            uint32_t o[64];
            tmem_ld32(tq + PL::kO + j0 + j, o);
            if (j + 32 < now) tmem_ld32(tq + PL::kO + j0 + j + 32, o + 32);
            tmem_wait_ld();
            if (live && l > 0.f && (any_odd<32>(o) || (j + 32 < now && any_odd<32>(o + 32)))) misc[4] = sg + 1;
            if (lane < nr) {
              float4* const dst = reinterpret_cast<float4*>(merge + (quarter * a.row_tile + lane) * pad + j);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (e < 8 || j + 32 < now) dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
          }
          if (!meet()) break;
          if (misc[4] == sg + 1 && !looked) {
            odd = odd_columns<T, D>(a, trow, h, ctx0, ctx1);
            looked = true;
          }
          for (int e0 = quarter * 32; e0 < nr * (now / 4); e0 += 128) {
            const int e = e0 + lane, j = e % (now / 4) * 4;
            uint32_t odd4 = 0;  // of the thread's columns, which are in one lane's word
            if (looked) odd4 = __shfl_sync(0xffffffffu, odd, (j0 + j) >> 3) >> (4 * (j & 7));
            if (e >= nr * (now / 4)) continue;
            const int rr = e / (now / 4);
            float mq[4], lq = 0.f, mo = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mq[q] = mstat[q * kSpreadRows + rr].x;
              mo = fmaxf(mo, mq[q]);
            }
            const float ref = mo == -INFINITY ? 0.f : mo;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float f = exp2_approx(mq[q] - ref), lx = mstat[q * kSpreadRows + rr].y;
              lq = fmaf(f, lx, lq);
              const float4 y = *reinterpret_cast<const float4*>(merge + (q * a.row_tile + rr) * pad + j);
              // a copy that saw nothing has weights 0 only: its O is 0 (or NaN by 0 * inf)
              if (lx == 0.f) continue;
              x.x = fmaf(f, y.x, x.x);
              x.y = fmaf(f, y.y, x.y);
              x.z = fmaf(f, y.z, x.z);
              x.w = fmaf(f, y.w, x.w);
            }
            if (odd4 & 7u) x.x = odd_value(odd4);
            if (odd4 >> 4 & 7u) x.y = odd_value(odd4 >> 4);
            if (odd4 >> 8 & 7u) x.z = odd_value(odd4 >> 8);
            if (odd4 >> 12 & 7u) x.w = odd_value(odd4 >> 12);
            if (poisoned) {
              const int d = j0 + j;
              const uint32_t see = mword[rr];
              x.x += poison_of<T>(a, trow, h, ctx, pois[d] & see, d);
              x.y += poison_of<T>(a, trow, h, ctx, pois[d + 1] & see, d + 1);
              x.z += poison_of<T>(a, trow, h, ctx, pois[d + 2] & see, d + 2);
              x.w += poison_of<T>(a, trow, h, ctx, pois[d + 3] & see, d + 3);
            }
            const int rw = r0 + rr, rs = small_div(rw, inv_g);
            const long long orow = ((long long)b * a.S + rs) * a.Hq + h * a.G + (rw - rs * a.G);
            if (final) {
              const float inv = lq == 0.f ? 0.f : 1.f / lq;
              const uint2 y = lq == 0.f ? make_uint2(0u, 0u)
                                        : make_uint2(pack16<T>(x.x * inv, x.y * inv), pack16<T>(x.z * inv, x.w * inv));
              *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * D + j0 + j) = y;
              if (j0 + j == 0 && a.lse != nullptr)
                a.lse[orow] = lq == 0.f ? -INFINITY : (mo + log2f(lq)) * 0.6931471805599453f;
            } else {
              reinterpret_cast<float4*>(a.part_o)[(slot * (D / 4) + (j0 + j) / 4) * a.row_tile + rr] = x;
              if (j0 + j == 0)
                *reinterpret_cast<float2*>(a.part_ml + (slot * a.row_tile + rr) * 2) = make_float2(mo, lq);
            }
          }
        }
        if (!ok) break;
        if (a.shared != nullptr && !final) {
          // The last CTA of a shared unit to arrive adds all its partials, in CTA order
          // (the sharers' count wraps to 0 with it); a launch of its own for what one
          // SM reads in a microsecond would take longer.
          __threadfence();
          if (!meet()) break;
          const int first = g_first, last = g_last;
          if (quarter == 0 && lane == 0) {
            const unsigned before = attn_arrive(a.shared, first, last);
            misc[3] = (misc[3] & ~1u) + 2u + (before == (unsigned)(last - first) ? 1u : 0u);
          }
          if (!meet()) break;
          if (misc[3] & 1u) {
            __threadfence();
            for (int e = quarter * 32 + lane; e < nr * (D / 4); e += 128) {
              const int rr = e / (D / 4), j = e % (D / 4);
              const float2* const ml = reinterpret_cast<const float2*>(a.part_ml) + rr;
              const float4* const po = reinterpret_cast<const float4*>(a.part_o) + (size_t)j * a.row_tile + rr;
              const size_t step = (size_t)(D / 4) * a.row_tile;
              AttnSum sum = attn_sum_parts<false>(ml, po, a.row_tile, step, first, first, last);
              if (!sum.finite()) sum = attn_sum_odd_parts(ml, po, a.row_tile, step, first, first, last);
              const int rw = r0 + rr, rs = small_div(rw, inv_g);
              const long long orow = ((long long)b * a.S + rs) * a.Hq + h * a.G + (rw - rs * a.G);
              const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
              *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * D + j * 4) =
                  sum.l == 0.f ? make_uint2(0u, 0u)
                               : make_uint2(pack16<T>(sum.o.x * inv, sum.o.y * inv),
                                            pack16<T>(sum.o.z * inv, sum.o.w * inv));
              if (j == 0 && a.lse != nullptr) a.lse[orow] = sum.lse();
            }
          }
        }
      } else {
        const long long orow = ((long long)b * a.S + wr) * a.Hq + h * a.G + (row - wr * a.G);
        const bool none = !live || l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        if (poisoned) {  // into the output where it lies
#pragma unroll 1
          for (int j = 0; j < D; ++j) {
            const uint32_t bits = pois[j] & word;
            if (!__any_sync(0xffffffffu, bits != 0)) continue;
            const uint32_t x = tmem_ld1(tq + PL::kO + j);
            tmem_wait_ld();
            const float add = bits ? poison_of<T>(a, trow, h, ctx, bits, j) : 0.f;
            __syncwarp();
            tmem_st1(tq + PL::kO + j, bits ? __float_as_uint(__uint_as_float(x) + add) : x);
          }
          tmem_wait_st();
        }
        constexpr int OC = D < 128 ? D : 128;  // columns at once
#pragma unroll 1
        for (int j = 0; j < D; j += OC) {
          // written first, so that the look at them hides behind the stores; again if they were odd
#pragma unroll 1
          for (bool again = false;; again = true) {
            uint32_t o[OC];
#pragma unroll
            for (int e = 0; e < OC; e += 32) tmem_ld32(tq + PL::kO + j + e, o + e);
            tmem_wait_ld();
            if (r < nr && final) {
              uint4* const dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * D + j);
#pragma unroll
              for (int e = 0; e < OC; e += 8) {
                uint32_t y[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  y[z] = none ? 0u : pack16<T>(__uint_as_float(o[e + 2 * z]) * inv, __uint_as_float(o[e + 2 * z + 1]) * inv);
                dst[e / 8] = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else if (r < nr) {
              float4* const dst = reinterpret_cast<float4*>(a.part_o) + (slot * (D / 4) + j / 4) * a.row_tile + r;
#pragma unroll
              for (int e = 0; e < OC; e += 4)
                dst[(e / 4) * a.row_tile] = live ? make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                               __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]))
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (again || !__any_sync(0xffffffffu, live && l > 0.f && any_odd<OC>(o))) break;
            if (!looked) odd = odd_columns<T, D>(a, trow, h, ctx0, ctx1);
            looked = true;
#pragma unroll 1
            for (int d = j; d < j + OC; ++d) {
              const uint32_t kind = odd_of(odd, d);
              if (kind == 0) continue;
              const uint32_t bits = poisoned ? pois[d] & word : 0u;
              const float x = odd_value(kind) + (bits ? poison_of<T>(a, trow, h, ctx, bits, d) : 0.f);
              __syncwarp();
              tmem_st1(tq + PL::kO + d, __float_as_uint(x));
            }
            tmem_wait_st();
          }
        }
        if (r < nr) {
          if (final) {
            if (a.lse != nullptr) a.lse[orow] = none ? -INFINITY : (mm + log2f(l)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float2*>(a.part_ml + (slot * a.row_tile + r) * 2) =
                live ? make_float2(mm, l) : make_float2(-INFINITY, 0.f);
          }
        }
      }
      if (poisoned) {  // every warp has read the notes: clear them for the segment after the next
        if (!meet()) break;
        for (int e = quarter * 32 + lane; e < D; e += 32 * nq) pois[e] = 0;
        if (quarter == 0 && lane == 0) misc[1 + (sg & 1)] = 0;
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  tmem_wait_st();  // (of a role that gave up behind its stores)
  tc_fence_before();
  if (__syncthreads_or(!ok) && a.shared != nullptr && warp == 0) {
    // After a timeout: the arrivals that were not made, so that the counts are back at 0
    // when every CTA has ended.
    AttnWalk w;
    int made = misc[3] >> 1;
    for (bool more = w.start(a, blockIdx.x, lane); more; more = w.more()) {
      const int count = w.segment();
      int first, last;
      w.sharers(first, last);
      if (first != last && --made < 0 && lane == 0) attn_arrive(a.shared, first, last);
      w.advance(a, count);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

template <typename T, int D, bool SPREAD>
cudaError_t attn_tc_launch(const AttnMaps& m, AttnArgs a, cudaStream_t st) {
  using PL = AttnPlan<D, SPREAD>;
  auto kernel = attn_tc_kernel<T, D, SPREAD>;
  // two Q buffers where they cost the ring nothing (spread rows: two sets of up to 16
  // in the buffer of 128), or leave it five slots (two and a half tiles).  One buffer against
  // two, bf16, 4 cache heads, 64 sequences of 700 positions and one of 30,000: 128 rows x 128,
  // five slots left: 101.9 to 100.0 us and 25.3 to 25.6; 96 rows: 83.2 to 81.1 and 24.3 to
  // 24.5; 64 rows x 256, four slots left: 115 to 114 and 33.0 to 32.7, within the noise.
  a.q_bufs = SPREAD ? (a.row_tile <= 16 ? 2 : 1) : PL::slots(a.row_tile, 2) >= 5 ? 2 : 1;
  a.slots = PL::slots(a.row_tile, a.q_bufs);
  // more than half an SM's: one CTA and one tensor-memory allocation per SM
  const int smem = 1024 + PL::kSmall + PL::q_bytes(a.row_tile, a.q_bufs) + a.slots * PL::kSlot;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kAttnSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(a.ctas), dim3(kAttnThreads), smem, st, m, a);
}

}  // namespace

// The instance for one 16-bit type.
template <typename T>
cudaError_t attn_tc_dispatch(const AttnMaps& m, const AttnArgs& a, cudaStream_t st) {
  // Spread rows end with a merge of four outputs of rows x D.  Spread against not (us; 48
  // sequences of 4000 positions unless stated): 4 rows x 128: 138 to 143, 300 of 100: 68 to
  // 93, one of 613: 15.0 to 17.1; 8 x 256: 83 to 87; 16 x 256: 90 to 92; 32 x 128: 167 to
  // 170, but 300 of 100: 117 to 93; 32 x 256, 8 of 8000: 49 to 45, one of 30,000: 38 to 34.
  const bool spread = a.row_tile <= kSpreadRows && a.row_tile * a.D <= kSpreadMost;
  switch (a.D) {
    case 64: return spread ? attn_tc_launch<T, 64, true>(m, a, st) : attn_tc_launch<T, 64, false>(m, a, st);
    case 128: return spread ? attn_tc_launch<T, 128, true>(m, a, st) : attn_tc_launch<T, 128, false>(m, a, st);
    default: return spread ? attn_tc_launch<T, 256, true>(m, a, st) : attn_tc_launch<T, 256, false>(m, a, st);
  }
}

}  // namespace sdv

// Attention over a shared prefix on the 5th-generation tensor cores (sm_103a): sdv_prefix_attn
// for head sizes 64, 128 and 256.
//
// Per query row r and position p, as in the paged attention:
//   s = q_r . k_p;  m = running max of scale s;  P = 2^((scale s - m) log2 e)
//   l += sum P;  O = O 2^(m_old - m) + P V
// The rows are those of all sequences, 128 to an MMA tile, and every one sees every position:
// 4 D flops per row and position against 4 D bytes per position and cache head.  From some 300
// rows a head on the products bound it, below that reading the prefix does.
//
// One persistent CTA per SM walks an equal share of all tiles (prefix_attn.cuh).  Warp roles:
//   warp 0      TMA producer: a lane per (page, 64-element block) box of a ring slot of 128
//               positions x up to 128 elements, in the order in which the MMAs take them;
//   warp 1      allocates tensor memory and issues the MMAs: S = Q K^T (both K-major in shared
//               memory), O += P V (P in tensor memory, V as it lies in the cache, MN-major);
//   warp 2      a segment's queries by TMA, and whether table entries are missing;
//   warps 4-7, 8-11   softmax of a row tile each, a thread per row: S from tensor memory, P back
//               into its columns; they also write the partial outputs.
// Two row tiles (STREAMS == 2, heads up to 128) share each tile of keys and values and take turns:
// one's products run under the other's softmax.  Each has one set of score columns.  With one row
// tile the scores have two sets, and S of the next tile runs under this one's softmax.
//
// 256 windows of five rows, 32 heads over 8 of 128, 16,384 positions: 235 us, 1.46 PFLOP/s, shared
// memory's share in the products (both operands of S, one of P V) the bound; 64 rows, 32,768
// positions, 39 us, 3.4 TB/s: half of it is start, end and 13.5 tiles a CTA dealt as 14; 216 rows of 16 heads
// over 2 of 256, 8011 positions, 38 us: one row tile at a time, 128 KB of tiles for each.
//
// The reference maximum moves only when it grows by more than 2^8, so O is rescaled rarely.
// fp16's P carries a factor 2^6 (weights down to 2^-20 of the row's largest are normal numbers),
// bf16's, with the range of fp32, 2^-24: sums of 2^24 of the largest values do not overflow.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "mixing.h"
#include "prefix_attn.cuh"
#include "prefix_tc.h"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kPrefixSmem = 232448 - kWaitLimitBytes;  // all of an SM's: one CTA, one tensor-memory allocation
constexpr uint64_t kPrefixDrainNs = 100000000ull;      // 0.1 s: in-flight work at teardown
constexpr int kPrefixMaxSlots = 10;

template <int D, int STREAMS>
struct PrefixPlan {
  static constexpr int TK = kPrefixTcTile;
  static constexpr int kWide = D < 128 ? D : 128;     // elements of a ring slot's rows
  static constexpr int kHalves = D / kWide;           // slots of a tile's keys, and of its values
  static constexpr int kBlocks = kWide / 64;
  static constexpr int kSlot = TK * kWide * 2;
  static constexpr int kQ = 128 * D * 2;              // one row tile's queries
  static constexpr int kNumBars = 2 * kPrefixMaxSlots + 2 + 4 + 2 + 2 + 1 + 1 + 1 + 1;
  static constexpr int kSmall = kNumBars * 8 + 32;
  static constexpr int kFit = (kPrefixSmem - 1024 - kSmall - STREAMS * kQ) / kSlot;
  static constexpr int NS = kFit < kPrefixMaxSlots ? kFit : kPrefixMaxSlots;
  static constexpr int kThreads = 128 + 128 * STREAMS;
  static constexpr int kO = 256;                      // tensor-memory columns: two sets of scores, then outputs
  static constexpr int kSmem = 1024 + STREAMS * kQ + NS * kSlot + kSmall;
  static_assert(kO + STREAMS * D <= 512, "tensor memory");
  static_assert(NS >= 2 * kHalves + 1 && kSmem * 2 > kPrefixSmem, "a tile ahead; one CTA per SM");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Lane q of four has y[0 .. 3] of its row; afterwards y[q] of rows 0 .. 3.
__device__ __forceinline__ void quad_transpose(float (&y)[4][4], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float give = up ? y[i][z] : y[i | bit][z], got = __shfl_xor_sync(0xffffffffu, give, bit);
        if (up) y[i][z] = got;
        else y[i | bit][z] = got;
      }
    }
  }
}

template <typename T, int D>
__device__ __noinline__ uint32_t prefix_odd_columns(const PrefixArgs& a, int h, int from, int to) {
  // lane l gets columns 8 (l % (D / 8)) .. + 7, four bits each
  constexpr int C = D / 8;
  const int lane = threadIdx.x & 31;
  uint32_t odd = 0;
#pragma unroll 4
  for (int p = from + lane / C; p < to; p += 32 / C) {
    const int id = __ldg(a.table + p / a.page);
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

template <typename T, int D, int STREAMS>
__global__ void __launch_bounds__(128 + 128 * STREAMS, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixMaps maps, const __grid_constant__ PrefixArgs a) {
  using PL = PrefixPlan<D, STREAMS>;
  constexpr int TK = PL::TK, NS = PL::NS, KH = PL::kHalves;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kLift = kBf16 ? -kPrefixDrop : 6.f;  // P's power of two
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const sb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = base + STREAMS * PL::kQ, bars = ring + NS * PL::kSlot;
  volatile uint32_t* const misc = reinterpret_cast<uint32_t*>(sb + (bars - base) + PL::kNumBars * 8);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kPrefixMaxSlots + s); };
  constexpr int kB = 2 * kPrefixMaxSlots;
  auto s_full = [&](int i) { return bars + 8u * (kB + i); };       // a set of scores is there
  auto p_ready = [&](int i, int half) { return bars + 8u * (kB + 2 + 2 * i + half); };  // the weights of its 64 positions are
  auto pv_done = [&](int q) { return bars + 8u * (kB + 6 + q); };  // a row tile's P V has ended
  auto o_free = [&](int q) { return bars + 8u * (kB + 8 + q); };   // its outputs have been read
  const uint32_t q_full = bars + 8u * (kB + 10), q_free = q_full + 8, drain = q_full + 16;
  const int nq = (a.row_tile + 31) / 32;  // softmax warps of a row tile with rows

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
      mbar_init(p_ready(i, 0), nq);
      mbar_init(p_ready(i, 1), nq);
      mbar_init(pv_done(i), 1);
      mbar_init(o_free(i), nq);
    }
    mbar_init(q_full, 2);
    mbar_init(q_free, 1 + STREAMS * nq);
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = misc[0];
  griddep_wait();
  // the launch behind may start when the word is there: the last block's idle warp sees to it
  if (a.passed == nullptr || blockIdx.x + 1 < gridDim.x) {
    griddep_launch_dependents();
  } else if (warp == 3) {
    if (lane == 0) pass_on(a.passed);
    __syncwarp();
    griddep_launch_dependents();
  }
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = mbar_wait_warp(bar, parity, a.status);
    return ok;
  };
  bool bad_length;
  const int length = prefix_length(a, bad_length);
  if (bad_length && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, kDevErrIndex);
  const int per_head = (a.row_tiles + STREAMS - 1) / STREAMS;
  PrefixWalk w;
  bool more = w.start(a, length, blockIdx.x);
  const int page_log = 31 - __clz(a.page), box = min(a.page, TK);
  // Ring places of tile t's keys and values in a segment of c tiles, from the segment's first
  // place on: the order in which the MMAs take them.
  auto place_k = [](int t, int) { return STREAMS == 2 ? 2 * t * KH : t == 0 ? 0 : (2 * t - 1) * KH; };
  auto place_v = [](int t, int c) { return (STREAMS == 2 ? 2 * t + 1 : t == c - 1 ? 2 * t + 1 : 2 * t + 2) * KH; };

  if (warp == 0) {
    // ---- producer ----
    const int chunks = TK / box;                         // pages (or one page's part) of a tile
    const int beyond = a.n_pages * a.Hkv * a.page;       // a row past the tensor map's end: zeros
    const uint64_t policy = per_head == 1 ? l2_policy_evict_first() : l2_policy_normal();
    const int cb = lane % PL::kBlocks, chunk = lane / PL::kBlocks;
    const bool mine = chunk < chunks;
    const uint32_t dst = ring + cb * (TK * 128) + chunk * box * 128;
    int slot = 0, use = 0, issued = 0, asked = 0, withheld = -1;
    for (; ok && more; more = w.more()) {
      const int count = w.segment(), h = w.unit / per_head;
      auto page_of = [&](int t) {
        const int p = t * TK + chunk * box;
        return mine && p < length ? __ldg(a.table + (p >> page_log)) : -1;
      };
      auto row_of = [&](int t, int id) {
        return id >= 0 && id < a.n_pages ? (id * a.Hkv + h) * a.page + ((t * TK + chunk * box) & (a.page - 1)) : beyond;
      };
      auto put = [&](const CUtensorMap* map, int y, bool skip) {
#pragma unroll
        for (int half = 0; half < KH; ++half) {
          if (use > 0 && !await(empty(slot), (use - 1) & 1)) return;
          if (skip && half == 0) {
            withheld = issued;
          } else {
            if (lane == 0) mbar_arrive_expect_tx(full(slot), PL::kSlot);
            __syncwarp();
            if (mine) tma_load_2d(dst + slot * PL::kSlot, map, half * 128 + cb * 64, y, full(slot), policy);
          }
          ++issued;
          if (++slot == NS) {
            slot = 0;
            ++use;
          }
        }
      };
      const int end = w.tile + count;
      // table entries are loaded four tiles ahead
      int ids[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) ids[k] = w.tile + k < end ? page_of(w.tile + k) : -1;
      int last = 0;  // one row tile: the row of the tile before, whose values come behind this one's keys
      for (int t0 = w.tile; ok && t0 < end; t0 += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + k;
          if (t >= end || !ok) break;
          const int y = row_of(t, ids[k]);
          ids[k] = t + 4 < end ? page_of(t + 4) : -1;
          put(&maps.k, y, ++asked == a.fault.withhold);
          if constexpr (STREAMS == 2) {
            if (ok) put(&maps.v, y, false);
          } else {
            if (ok && t > w.tile) put(&maps.v, last, false);
            last = y;
          }
        }
      }
      if (STREAMS == 1 && ok) put(&maps.v, last, false);
      w.advance(count);
    }
    // copies into places that are not taken again have to land before the CTA ends
    for (int i = max(issued - NS, 0); i < issued; ++i)
      if (i != withheld) mbar_wait_bounded(full(i % NS), (i / NS) & 1, kPrefixDrainNs);
  } else if (warp == 2) {
    // ---- a segment's queries ----
    const uint64_t policy = l2_policy_normal();
    int sg = 0;
    for (; more; more = w.more(), ++sg) {
      if (sg > 0 && !await(q_free, (sg - 1) & 1)) break;
      const int count = w.segment(), h = w.unit / per_head, rt = (w.unit - h * per_head) * STREAMS;
      const int streams = min(STREAMS, a.row_tiles - rt);
      if (lane == 0) mbar_arrive_expect_tx(q_full, streams * (D / 64) * a.row_tile * 128);
      __syncwarp();
      if (lane < streams * (D / 64)) {
        const int q = lane / (D / 64), cb = lane % (D / 64);  // rows past the batch's end: zeros
        tma_load_3d(base + q * PL::kQ + cb * (128 * 128), &maps.q, cb * 64, h * a.G, (rt + q) * a.tile_tokens, q_full,
                    policy);
      }
      const int last = min((w.tile + count) * TK, length) - 1;
      bool absent = false;
#pragma unroll 4
      for (int e = (w.tile * TK >> page_log) + lane; e <= last >> page_log; e += 32) {
        const int id = __ldg(a.table + e);
        absent |= id < 0 || id >= a.n_pages;
      }
      absent = __any_sync(0xffffffffu, absent);
      if (lane == 0) {
        misc[1] = absent;
        if (absent) atomicOr(a.status, kDevErrIndex);
        mbar_arrive(q_full);
      }
      __syncwarp();
      w.advance(count);
    }
    if (sg > 0) mbar_wait_bounded(q_full, (sg - 1) & 1, kPrefixDrainNs);
  } else if (warp == 1) {
    // ---- MMA: every lane keeps the same state, one elected lane issues ----
    constexpr uint32_t id_pv = idesc_16_f32(kBf16, 128, PL::kWide, false, true);
    // a negative scale negates Q in the product: the maximum is then over scale * s
    const uint32_t id_qk = idesc_16_f32(kBf16, 128, TK, false, false) | (a.scale_log2 < 0.f ? kIdescNegateA : 0u);
    int first = 0, tiles = 0;            // ring place and tile number of the segment's start
    int done[2] = {0, 0}, begun[2] = {0, 0}, sent[2] = {0, 0};  // per row tile: P V waited for, segments, P V issued
    auto wait_full = [&](int place) { return await(full(place % NS), (place / NS) & 1); };
    auto pv_wait = [&](int q, int n) {   // the first n P V of row tile q have ended
      for (; done[q] < n; ++done[q])
        if (!await(pv_done(q), done[q] & 1)) return false;
      return true;
    };
    // S of a tile into score set `set`, from row tile q's queries
    auto qk = [&](int q, int set, int place) {
#pragma unroll
      for (int half = 0; half < KH; ++half) {
        const uint64_t qd = smem_desc_sw128(base + q * PL::kQ + half * (2 * 128 * 128), 16, 1024);
        const uint64_t kd = smem_desc_sw128(ring + (place + half) % NS * PL::kSlot, 16, 1024);
#pragma unroll
        for (int j = 0; j < PL::kBlocks; ++j)
          tc_mma4_ss(tm + set * TK, qd + j * (128 * 128 >> 4), kd + j * (TK * 128 >> 4), id_qk, half > 0 || j > 0);
      }
      tc_commit_elect(s_full(set));
    };
    // O += P V in two steps of 64 positions, each as soon as its weights are there
    auto pv = [&](int q, int set, int place, bool add, uint32_t parity) {
#pragma unroll
      for (int j = 0; j < TK / 64; ++j) {
        if (!await(p_ready(set, j), parity)) return false;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < KH; ++half) {
          const uint64_t vd = smem_desc_sw128(ring + (place + half) % NS * PL::kSlot, TK * 128, 1024);
          tc_mma4_ts(tm + PL::kO + q * D + half * 128, tm + set * TK + j * 32, vd + j * (4 * 2048 >> 4), id_pv,
                     add || j > 0);
        }
      }
      tc_commit_elect(pv_done(q));
      ++sent[q];
      return true;
    };
    auto release = [&](int place) {
#pragma unroll
      for (int half = 0; half < KH; ++half) tc_commit_elect(empty((place + half) % NS));
    };
    auto wait_tile = [&](int place) {
      for (int half = 0; half < KH; ++half)
        if (!wait_full(place + half)) return false;
      return true;
    };
    for (int sg = 0; more && ok; more = w.more(), ++sg) {
      const int count = w.segment();
      const int rt = w.unit % per_head * STREAMS, streams = min(STREAMS, a.row_tiles - rt);
      if (!await(q_full, sg & 1) || !wait_tile(first + place_k(0, count))) break;
      tc_fence_after();
      if constexpr (STREAMS == 2) {
        // the last P of either set has been read: its P V was waited for before the segment's end
        for (int q = 0; q < streams; ++q) {
          if (!pv_wait(q, sent[q])) break;
          qk(q, q, first);
        }
        if (!ok) break;
        release(first);
        if (count == 1) tc_commit_elect(q_free);
        for (int t = 0; ok && t < count; ++t) {
          const int v = first + place_v(t, count), k = first + place_k(t + 1, count);
          if (!wait_tile(v)) break;
          for (int q = 0; q < streams; ++q) {
            if (t == 0 && begun[q] > 0 && !await(o_free(q), (begun[q] - 1) & 1)) break;
            if (!pv(q, q, v, t > 0, sent[q] & 1)) break;
            if (q == streams - 1) release(v);
            if (t + 1 < count) {
              if (q == 0 && !wait_tile(k)) break;
              if (!pv_wait(q, sent[q])) break;
              tc_fence_after();
              qk(q, q, k);
              if (q == streams - 1) {
                release(k);
                if (t + 2 == count) tc_commit_elect(q_free);
              }
            }
          }
        }
      } else {
        if (!pv_wait(0, max(tiles - 1, 0))) break;
        qk(0, tiles & 1, first);
        release(first);
        if (count == 1) tc_commit_elect(q_free);
        for (int t = 0; ok && t < count; ++t) {
          const int i = tiles + t;
          if (t + 1 < count) {
            const int k = first + place_k(t + 1, count);
            if (!pv_wait(0, i) || !wait_tile(k)) break;  // P of tile i - 1 stood in these columns
            tc_fence_after();
            qk(0, (i + 1) & 1, k);
            release(k);
            if (t + 2 == count) tc_commit_elect(q_free);
          }
          const int v = first + place_v(t, count);
          if (!wait_tile(v)) break;
          if (t == 0 && begun[0] > 0 && !await(o_free(0), (begun[0] - 1) & 1)) break;
          if (!pv_wait(0, i) || !pv(0, i & 1, v, t > 0, (i >> 1) & 1)) break;
          release(v);
        }
      }
      for (int q = 0; q < streams; ++q) ++begun[q];
      first += 2 * KH * count;
      tiles += count;
      w.advance(count);
    }
    // every MMA has ended before tensor memory is freed
    tc_commit_elect(drain);
    mbar_wait_bounded(drain, 0, kPrefixDrainNs);
  } else if (warp >= 4 && (warp & 3) < nq) {
    // ---- softmax and partial outputs: a thread per row ----
    const int q = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tm + ((uint32_t)(quarter * 32) << 16);
    // a scale of 0 becomes one that leaves every finite score at 0 (times 0 a masked score
    // would be NaN)
    const float c = fmaxf(fabsf(a.scale_log2), 1e-36f);
    int first = 0, i = 0;  // ring place of the segment's start; tiles of this row tile so far
    int seen = 0;          // P V waited for
    auto pv_wait = [&](int n) {
      for (; seen < n; ++seen)
        if (!await(pv_done(q), seen & 1)) return false;
      return true;
    };
    for (int sg = 0; more && ok; more = w.more(), ++sg) {
      const int count = w.segment(), h = w.unit / per_head, rt = (w.unit - h * per_head) * STREAMS + q;
      const int tile0 = w.tile, place = w.place(blockIdx.x), unit = w.unit;
      if (!await(q_full, sg & 1)) break;
      const bool some_absent = misc[1] != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_free);
      w.advance(count);
      const int seg_first = first;
      first += 2 * KH * count;
      if (rt >= a.row_tiles) continue;  // an odd number of row tiles: nothing for the second
      float m = -INFINITY, l = 0.f;     // reference maximum (log2 domain), sum of P relative to it
      for (int t = 0; t < count; ++t, ++i) {
        const int p0 = (tile0 + t) * TK, set = STREAMS == 2 ? q : i & 1;
        const bool edge = some_absent || p0 + TK > length;
        if (!await(s_full(set), (STREAMS == 2 ? i : i >> 1) & 1)) break;
        tc_fence_after();
        const uint32_t ts = tq + set * TK;
        uint32_t sr[TK];
#pragma unroll
        for (int j = 0; j < TK; j += 32) tmem_ld32(ts + j, sr + j);
        tmem_wait_ld();
        uint32_t absent = 0;  // pages of the tile that cannot be followed, a bit each
        if (some_absent) {
          const int p = p0 + lane * box;
          bool gone = false;
          if (lane * box < TK && p < length) {
            const int id = __ldg(a.table + (p >> page_log));
            gone = id < 0 || id >= a.n_pages;
          }
          absent = __ballot_sync(0xffffffffu, gone);
        }
        auto mask32 = [&](uint32_t* x, int j) {  // of 32 columns from j on
          const int n = min(max(length - p0 - j, 0), 32);
          uint32_t bits = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
          if (absent != 0) {
            for (int e = 0; e < 32; e += 8)
              if (absent >> ((j + e) / box) & 1) bits &= ~(0xffu << e);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(bits >> e & 1)) x[e] = 0xff800000u;
        };
        if (edge) {
#pragma unroll
          for (int j = 0; j < TK; j += 32) mask32(sr + j, j);
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = __uint_as_float(sr[j]);
#pragma unroll
        for (int j = 4; j < TK - 4; j += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(sr[j + e]), __uint_as_float(sr[j + 4 + e]));
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(sr[TK - 4 + e]));
        const float mt = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c;
        const bool grow = mt > m + 8.f;  // also from -inf to any number
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow && m != -INFINITY ? exp2_approx(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (t > 0 && __any_sync(0xffffffffu, f != 1.f)) {
            if (!pv_wait(i)) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D; j += 16) {
              uint32_t o[16];
              tmem_ld16(tq + PL::kO + q * D + j, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tq + PL::kO + q * D + j, o);
            }
          }
        }
        const float ref = m == -INFINITY ? -kLift : m - kLift;
        const f32x2 c2 = pair2(c, c), ref2 = pair2(-ref, -ref);
        f32x2 l2[2] = {pair2(0.f, 0.f), pair2(0.f, 0.f)};
        if (p0 + TK > length && q == 0) {
          // what the last page holds behind the end must not meet its zero weights
          const int from = length - p0, to = min(TK, (int)(((uint32_t)length + a.page - 1) / a.page * a.page - p0));
          const int v = seg_first + place_v(t, count);
          for (int half = 0; half < KH && from < to; ++half) {
            if (!await(full((v + half) % NS), ((v + half) / NS) & 1)) break;
            const uint32_t vb = ring + (v + half) % NS * PL::kSlot;
            for (int e = from * (PL::kWide / 8) + quarter * 32 + lane; e < to * (PL::kWide / 8); e += 32 * nq) {
              const int j = e / (PL::kWide / 8), ch = e % (PL::kWide / 8);
              sts128(vb + (ch >> 3) * (TK * 128) + swz128(j, ch & 7), make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
          }
        }
        if (!ok) break;
        // The weights, in two halves: the products with the first run under the second, whose scores
        // are read again rather than kept in registers.  (2^x of a part of them by a polynomial, beside
        // the special function unit, made every tile longer: 245 to 260 us for 20,480 tiles of two row
        // tiles, and so did two threads a row, 281; 239 as it is.)
        uint32_t again[2][32];
#pragma unroll
        for (int j = 0; ok && j < TK / 32; ++j) {
          uint32_t* const x = j < 2 ? sr + 32 * j : again[j & 1];
          if (j >= 2) {
            tmem_wait_ld();
            if (edge) mask32(x, 32 * j);
          }
          if (j == 1 || j == 2) tmem_ld32(ts + 32 * (j + 1), again[(j + 1) & 1]);
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 z = unpair2(fma2(pair2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, ref2));
            const f32x2 y = pair2(exp2_approx(z.x), exp2_approx(z.y));
            l2[e & 1] = add2(l2[e & 1], y);
            p[e] = pack16<T>(y);
          }
          tmem_st16(ts + j * 16, p);
          if (j == 0 || j == 2) continue;
          if (j == 3 && !pv_wait(i)) break;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready(set, j / 2));
        }
        if (!ok) break;
        const float2 la = unpair2(l2[0]), lb = unpair2(l2[1]);
        l += (la.x + la.y) + (lb.x + lb.y);
      }
      if (!ok) break;
      if (!pv_wait(i)) break;
      tc_fence_after();
      const int nr = min(a.row_tile, a.tokens * a.G - rt * a.row_tile);
      const size_t at = ((size_t)unit * a.sharers + place) * a.unit_tiles + q;
      const bool live = r < nr;
      bool looked = false;
      uint32_t odd = 0;
#pragma unroll 1
      for (int j = 0; j < D; j += 32) {
        uint32_t o[32];
        tmem_ld32(tq + PL::kO + q * D + j, o);
        tmem_wait_ld();
        // an infinity among the values has met weights of 0 in 16 bits: an output that is not
        // finite is told from the values themselves
        float zero = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) zero = fmaf(__uint_as_float(o[e]), 0.f, zero);
        if (__any_sync(0xffffffffu, live && l > 0.f && zero != 0.f)) {
          if (!looked) odd = prefix_odd_columns<T, D>(a, h, tile0 * TK, min((tile0 + count) * TK, length));
          looked = true;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t kind = __shfl_sync(0xffffffffu, odd, (j + e) >> 3) >> (4 * (e & 7)) & 7u;
            if (kind && l > 0.f) o[e] = __float_as_uint(odd_value(kind));
          }
        }
        // four lanes pass 16-byte pieces round so that they write 64 bytes of one row side by side
        float* const dst = a.part_o + (at * a.row_tile + (r & ~3)) * D + j + (lane & 3) * 4;
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          float y[4][4];
#pragma unroll
          for (int z = 0; z < 16; ++z) y[z >> 2][z & 3] = __uint_as_float(o[e + z]);
          quad_transpose(y, lane);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            if ((r & ~3) + z < nr) *reinterpret_cast<float4*>(dst + z * D + e) = make_float4(y[z][0], y[z][1], y[z][2], y[z][3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free(q));
      if (live)
        *reinterpret_cast<float2*>(a.part_ml + (at * a.row_tile + r) * 2) =
            make_float2(m == -INFINITY ? -INFINITY : m - kLift, l);
    }
  }
  __syncwarp();
  tmem_wait_st();  // (of a role that gave up behind its stores)
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

template <typename T, int D, int STREAMS>
cudaError_t prefix_tc_launch(const PrefixMaps& m, const PrefixArgs& a, cudaStream_t st) {
  using PL = PrefixPlan<D, STREAMS>;
  auto kernel = prefix_tc_kernel<T, D, STREAMS>;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPrefixSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(a.ctas), dim3(PL::kThreads), PL::kSmem, st, m, a);
}

}  // namespace

// The instance for one 16-bit type.
template <typename T>
cudaError_t prefix_tc_dispatch(const PrefixMaps& m, const PrefixArgs& a, cudaStream_t st) {
  const bool two = a.unit_tiles == 2;
  switch (a.D) {
    case 64: return two ? prefix_tc_launch<T, 64, 2>(m, a, st) : prefix_tc_launch<T, 64, 1>(m, a, st);
    case 128: return two ? prefix_tc_launch<T, 128, 2>(m, a, st) : prefix_tc_launch<T, 128, 1>(m, a, st);
    default: return prefix_tc_launch<T, 256, 1>(m, a, st);
  }
}

}  // namespace sdv

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
//   warp 0      TMA producer: a lane per (page, 64-element block) box; tiles of keys
//               and values alternate through a ring of equal slots;
//   warp 1      allocates tensor memory, one lane issues the MMAs:
//               S = Q K^T (both K-major in shared memory), one tile ahead of
//               O += P V (P in tensor memory, V as it lies in the cache, MN-major);
//   warps 2-5   softmax, a thread per row: S from tensor memory, P back into its
//               columns; they also stage Q, and write the outputs.
// The reference maximum moves only when it grows by more than 2^8 (the sum and
// output stay exact relative to it), so O in tensor memory is rescaled rarely.
// P carries a factor 2^6: with it the weights down to 2^-20 of the row's largest
// stay in fp16's normal range, and 2^14 is the most it can reach.  Rounding P to
// the 16-bit type is the one rounding inside the sum (the sum l takes P before
// it); it is what a matrix instruction on 16-bit values needs.
//
// Tiles that reach past the context (window rows, the end, absent pages) are
// cleaned in shared memory before P V: rows that nobody may see become zeros, and
// a window row's infinities and NaN are zeroed and noted, then added to the rows
// that do see them at the end -- 0 * inf would otherwise reach the others.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "attn_sched.cuh"
#include "attn_tc.h"
#include "host_util.h"
#include "sdv.h"
#include "sdv_kernels.h"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kAttnThreads = 192;
constexpr uint64_t kAttnDrainNs = 100000000ull;  // 0.1 s: in-flight work at teardown

template <int D>
struct AttnPlan {
  static constexpr int TK = attn_tc_tile(D);
  static constexpr int kBlocks = D / 64;
  static constexpr int kSlot = TK * D * 2;
  static constexpr int kQ = 128 * D * 2;
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 6 : 5;
  static constexpr int kRing = kQ;
  static constexpr int kPoison = kRing + kSlots * kSlot;
  static constexpr int kBars = kPoison + D * 4;
  static constexpr int kNumBars = 2 * kSlots + 2 + 2 + 1 + 1 + 1 + 1;
  static constexpr int kMisc = kBars + kNumBars * 8;
  static constexpr int kTotal = kMisc + 32 + 1024;  // the base is aligned to 1024
  static constexpr int kS = 0;                      // tensor-memory columns: two score tiles (P inside),
  static constexpr int kO = 2 * TK;                 // then the output
  static_assert(kO + D <= 512, "tensor memory");
  static_assert(kTotal <= 232448, "shared memory");
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

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const AttnArgs a) {
  using PL = AttnPlan<D>;
  constexpr int TK = PL::TK, NS = PL::kSlots;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const sb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + PL::kBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (NS + s); };
  auto s_full = [&](int i) { return bars + 8u * (2 * NS + i); };
  auto p_ready = [&](int i) { return bars + 8u * (2 * NS + 2 + i); };
  const uint32_t pv_done = bars + 8u * (2 * NS + 4), q_full = pv_done + 8, drain = pv_done + 16,
                 rows_met = pv_done + 24;
  uint32_t* const poison = reinterpret_cast<uint32_t*>(sb + PL::kPoison);
  volatile uint32_t* const misc = reinterpret_cast<uint32_t*>(sb + PL::kMisc);  // tmem base, poison seen
  const int nq = (a.row_tile + 31) / 32;  // softmax warps with rows

  if (warp == 1) {
    tmem_alloc(base + PL::kMisc, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_ready(i), nq);
    }
    mbar_init(pv_done, 1);
    mbar_init(q_full, nq);
    mbar_init(drain, 1);
    mbar_init(rows_met, nq);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = misc[0];
  griddep_wait();
  AttnWalk w;
  const bool work = w.start(a, blockIdx.x, lane);
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity))) {
      ok = false;
      if (lane == 0) atomicOr(a.status, kDevErrTimeout);
    }
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
  griddep_launch_dependents();

  if (work && warp == 0) {
    // ---- producer ----
    const int box = min(a.page, TK), chunks = TK / box;  // rows per box, pages (or page parts) per tile
    const uint64_t policy = a.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_normal();
    const int cb = lane % PL::kBlocks, chunk = lane / PL::kBlocks;
    const uint32_t dst = cb * (TK * 128) + chunk * box * 128;
    int slot = 0, use = 0;  // ring position and how often the ring has been passed
    uint32_t issued = 0;    // slots that ever got a copy
    while (ok && w.more()) {
      const int count = w.segment();
      const int h = w.unit / a.row_tiles;
      const int total = w.seq.ctx + w.seq.n;
      const int32_t* const row = a.table + (size_t)w.b * a.max_pages;
      auto page_of = [&](int t) {
        const int p = t * TK + chunk * box;
        return chunk < chunks && p < total ? __ldg(row + p / a.page) : -1;
      };
      int next = page_of(w.tile);
      for (int t = w.tile; ok && t < w.tile + count; ++t) {
        const int id = next;
        if (t + 1 < w.tile + count) next = page_of(t + 1);
        const bool there = id >= 0 && id < a.n_pages;
        const int y = there ? (id * a.Hkv + h) * a.page + (t * TK + chunk * box) % a.page : 0;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, there)) * box * 128;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (use > 0 && !await(empty(slot), (use - 1) & 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(full(slot), bytes);
          __syncwarp();
          if (there) tma_load_2d(base + PL::kRing + slot * PL::kSlot + dst, kv ? &tm_v : &tm_k, cb * 64, y, full(slot), policy);
          issued |= 1u << slot;
          if (++slot == NS) {
            slot = 0;
            ++use;
          }
        }
      }
      w.advance(a, count);
    }
    // every copy has landed before the CTA may end (after a timeout; otherwise its
    // consumers have seen it): slots from `slot` on were last used in the pass before
    if (!ok)
      for (int s = 0; s < NS; ++s)
        if (issued >> s & 1) mbar_wait_bounded(full(s), (s < slot ? use : use - 1) & 1, kAttnDrainNs);
  } else if (work && warp == 1) {
    // ---- MMA ----
    constexpr uint32_t id_qk = idesc_16_f32(kBf16, 128, TK, false, false);
    constexpr uint32_t id_pv = idesc_16_f32(kBf16, 128, D, false, true);
    // K and V tiles alternate: tile i uses ring positions 2i and 2i + 1
    int ks = 0, ku = 0, vs = 1, vu = 0;
    auto step2 = [&](int& s, int& u) {
      s += 2;
      if (s >= NS) {
        s -= NS;
        ++u;
      }
    };
    int segs = 0;
    auto qk = [&](int i, bool first) {  // S tile i; the first of a segment waits for its Q
      if (first && !await(q_full, segs & 1)) return;
      if (first) ++segs;
      if (!pv_wait(i - 1)) return;  // the P that held these columns has been read
      if (!await(full(ks), ku & 1)) return;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t kb = base + PL::kRing + ks * PL::kSlot;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t off = (j & 3) * 32;
          tc_mma_ss(tm + PL::kS + (i & 1) * TK, smem_desc_sw128(base + (j >> 2) * 16384 + off, 16, 1024),
                    smem_desc_sw128(kb + (j >> 2) * (TK * 128) + off, 16, 1024), id_qk, j > 0);
        }
        tc_commit(s_full(i & 1));
        tc_commit(empty(ks));
      }
      __syncwarp();
      step2(ks, ku);
    };
    int i = 0;
    qk(0, true);
    while (ok && w.more()) {
      const int count = w.segment();
      for (int t = 0; ok && t < count; ++t, ++i) {
        if (t + 1 < count) qk(i + 1, false);
        if (!await(full(vs), vu & 1) || !await(p_ready(i & 1), (i >> 1) & 1) || !pv_wait(i)) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t vb = base + PL::kRing + vs * PL::kSlot;
#pragma unroll
          for (int j = 0; j < TK / 16; ++j)
            tc_mma_ts(tm + PL::kO, tm + PL::kS + (i & 1) * TK + j * 8,
                      smem_desc_sw128(vb + j * 2048, TK * 128, 1024), id_pv, t > 0 || j > 0);
          tc_commit(pv_done);
          tc_commit(empty(vs));
        }
        __syncwarp();
        step2(vs, vu);
      }
      w.advance(a, count);
      if (ok && w.more()) qk(i, true);
    }
    // every MMA has ended before tensor memory is freed
    if (lane == 0) tc_commit(drain);
    __syncwarp();
    mbar_wait_bounded(drain, 0, kAttnDrainNs);
  } else if (work && warp >= 2 && (warp & 3) < nq) {
    // ---- softmax, Q and outputs: a thread per row ----
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tm + ((uint32_t)(quarter * 32) << 16);
    const int box = min(a.page, TK), chunks = TK / box;
    const bool flip = a.scale_log2 < 0.f, flat = a.scale_log2 == 0.f;  // in Q: the scale is taken as > 0
    const float c = flat ? 1.f : fabsf(a.scale_log2);
    const uint4* const qg = static_cast<const uint4*>(a.q);
    // Q of the unit the walk stands at, this warp's rows
    auto stage_q = [&](const AttnWalk& u) {
      const int h = u.unit / a.row_tiles, r0 = (u.unit % a.row_tiles) * a.row_tile;
      const int nr = min(a.row_tile, a.rows - r0);
      for (int e = lane; e < 32 * (D / 8); e += 32) {
        const int rr = quarter * 32 + e / (D / 8), ch = e % (D / 8), row = r0 + rr;
        if (rr >= nr) break;
        const int s = row / a.G, g = row - s * a.G;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (s < u.seq.n && !flat)
          x = __ldg(qg + ((((long long)u.b * a.S + s) * a.q_stride + (long long)(h * a.G + g) * D) >> 3) + ch);
        if (flip) {
          x.x ^= 0x80008000u;
          x.y ^= 0x80008000u;
          x.z ^= 0x80008000u;
          x.w ^= 0x80008000u;
        }
        sts128(base + (ch >> 3) * 16384 + swz128(rr, ch & 7), x);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    // the softmax warps meet (a bounded wait, as every one here)
    uint32_t meetings = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_met);
      return await(rows_met, meetings++ & 1);
    };
    stage_q(w);
    int i = 0;
    while (ok && w.more()) {
      const int count = w.segment();
      const int h = w.unit / a.row_tiles, r0 = (w.unit % a.row_tiles) * a.row_tile;
      const int nr = min(a.row_tile, a.rows - r0);
      const int row = r0 + r, wr = row / a.G;
      const bool live = r < nr && wr < w.seq.n;
      const uint32_t word = live ? attn_word(a, w.b, wr, w.seq.n) : 0u;
      const int ctx = w.seq.ctx, total = ctx + w.seq.n;
      const int32_t* const trow = a.table + (size_t)w.b * a.max_pages;
      if (w.seq.bad && lane == 0) atomicOr(a.status, kDevErrIndex);
      // the tiles that reach past the context may note poison (infinities, NaN in window rows)
      const bool edges = (w.tile + count) * (long long)TK > ctx;
      if (edges) {
        if (!meet()) break;  // the last segment's readers are done
        for (int e = quarter * 32 + lane; e < D; e += 32 * nq) poison[e] = 0;
        if (quarter == 0 && lane == 0) misc[1] = 0;
        if (!meet()) break;
      }
      auto absent_of = [&](int t) {  // pages of tile t that cannot be followed, a bit each
        const int p = t * TK + lane * box;
        bool gone = false;
        if (lane < chunks && p < total) {
          const int id = __ldg(trow + p / a.page);
          gone = id < 0 || id >= a.n_pages;
        }
        return gone;
      };
      float m = -INFINITY, l = 0.f;  // reference maximum (log2 domain), sum of P relative to it
      bool gone_next = absent_of(w.tile);
      for (int t = w.tile; ok && t < w.tile + count; ++t, ++i) {
        const uint32_t absent = __ballot_sync(0xffffffffu, gone_next);
        if (t + 1 < w.tile + count) gone_next = absent_of(t + 1);
        const int p0 = t * TK;
        const bool edge = p0 + TK > ctx || absent != 0;
        if (!await(s_full(i & 1), (i >> 1) & 1)) break;
        tc_fence_after();
        const uint32_t ts = tq + PL::kS + (i & 1) * TK;
        uint32_t sr[TK];
#pragma unroll
        for (int j = 0; j < TK; j += 32) tmem_ld32(ts + j, sr + j);
        tmem_wait_ld();
        if (edge) {
          if (absent != 0 && lane == 0) atomicOr(a.status, kDevErrIndex);
#pragma unroll
          for (int j = 0; j < TK; j += 32) {
            const int p = p0 + j, nc = min(max(ctx - p, 0), 32);
            uint32_t bits = nc >= 32 ? 0xffffffffu : ((1u << nc) - 1u);
            if (p < ctx) bits |= nc >= 32 ? 0u : word << nc;
            else bits |= p - ctx < 32 ? word >> (p - ctx) : 0u;
            if (!live) bits = 0u;
            if (absent != 0) {
              for (int e = 0; e < 32; e += 8)
                if (absent >> ((j + e) / box) & 1) bits &= ~(0xffu << e);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1)) sr[j + e] = 0xff800000u;
          }
        }
        float mx0 = __uint_as_float(sr[0]), mx1 = __uint_as_float(sr[1]);
#pragma unroll
        for (int j = 2; j < TK; j += 2) {
          mx0 = fmaxf(mx0, __uint_as_float(sr[j]));
          mx1 = fmaxf(mx1, __uint_as_float(sr[j + 1]));
        }
        const float mt = fmaxf(mx0, mx1) * c;
        const bool grow = live && mt > m + 8.f;  // also from -inf to any number
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow && m != -INFINITY ? exp2_approx(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (t > w.tile && __any_sync(0xffffffffu, f != 1.f)) {
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
        const float ref = m == -INFINITY ? -6.f : m - 6.f;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int j = 0; j < TK; j += 2) {
          const float e0 = exp2_approx(fmaf(__uint_as_float(sr[j]), c, -ref));
          const float e1 = exp2_approx(fmaf(__uint_as_float(sr[j + 1]), c, -ref));
          l0 += e0;
          l1 += e1;
          sr[j >> 1] = pack16<T>(e0, e1);
        }
        l += l0 + l1;
#pragma unroll
        for (int j = 0; j < TK / 2; j += 32) tmem_st32(ts + j, sr + j);
        if (edge) {
          // clean V: rows nobody may see, and what a window row holds that is not finite
          const int vslot = (2 * i + 1) % NS, vuse = (2 * i + 1) / NS;
          if (!await(full(vslot), vuse & 1)) break;
          const uint32_t vb = base + PL::kRing + vslot * PL::kSlot;
          const int from = absent != 0 ? 0 : max(ctx - p0, 0);
          for (int e = from * (D / 8) + quarter * 32 + lane; e < TK * (D / 8); e += 32 * nq) {
            const int j = e / (D / 8), ch = e % (D / 8), p = p0 + j;
            const uint32_t at = vb + (ch >> 3) * (TK * 128) + swz128(j, ch & 7);
            if (p >= total || (absent >> (j / box) & 1)) {
              sts128(at, make_uint4(0, 0, 0, 0));
            } else if (p >= ctx) {
              uint4 x = lds128(at);
              uint32_t* const xs = &x.x;
              uint32_t bad = 0;
#pragma unroll
              for (int z = 0; z < 4; ++z) bad |= nonfinite16<T>(xs[z]) << (2 * z);
              if (bad) {
#pragma unroll
                for (int z = 0; z < 8; ++z)
                  if (bad >> z & 1) {
                    atomicOr(poison + ch * 8 + z, 1u << (p - ctx));
                    xs[z >> 1] &= z & 1 ? 0x0000ffffu : 0xffff0000u;
                  }
                sts128(at, x);
                misc[1] = 1;
              }
            }
          }
          fence_proxy_async_smem();
        }
        if (!pv_wait(i)) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready(i & 1));
      }
      if (!ok) break;
      // the next unit's Q: this segment's score MMAs have all ended
      const bool starts = w.tile == 0, ends = w.tile + count == w.seq.tiles;
      const int b = w.b;
      w.advance(a, count);
      if (w.more()) stage_q(w);
      if (!pv_wait(i)) break;
      tc_fence_after();
      if (edges && !meet()) break;
      const bool poisoned = edges && misc[1] != 0;
      const bool final = starts && ends;
      const size_t slot = 2 * (size_t)blockIdx.x + (starts ? 1 : 0);
      const long long orow = ((long long)b * a.S + wr) * a.Hq + h * a.G + (row - wr * a.G);
      const bool none = !live || l == 0.f;
      const float inv = final ? (none ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
      for (int j = 0; j < D; j += 32) {
        uint32_t o[32];
        tmem_ld32(tq + PL::kO + j, o);
        tmem_wait_ld();
        if (poisoned) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t bits = poison[j + e] & word;
            if (bits) o[e] = __float_as_uint(__uint_as_float(o[e]) + poison_of<T>(a, trow, h, ctx, bits, j + e));
          }
        }
        if (final) {
          if (r < nr) {
            uint4* const dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * D + j);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t y[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                y[z] = none ? 0u : pack16<T>(__uint_as_float(o[e + 2 * z]) * inv, __uint_as_float(o[e + 2 * z + 1]) * inv);
              dst[e / 8] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        } else if (r < nr) {
          float4* const dst = reinterpret_cast<float4*>(a.part_o) + (slot * (D / 4) + j / 4) * a.row_tile + r;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            dst[(e / 4) * a.row_tile] = live ? make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                           __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      const float mm = m == -INFINITY ? -INFINITY : m - 6.f;
      if (r < nr) {
        if (final) {
          if (a.lse != nullptr) a.lse[orow] = none ? -INFINITY : (mm + log2f(l)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float2*>(a.part_ml + (slot * a.row_tile + r) * 2) =
              live ? make_float2(mm, l) : make_float2(-INFINITY, 0.f);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The cache as rows of dim elements: boxes of 64 elements x one page's rows of a
// tile, 128-byte swizzle.
bool page_map(const void* pages, bool bf16, uint64_t rows, int dim, int box_rows, CUtensorMap* map) {
  auto enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)dim, rows};
  cuuint64_t strides[1] = {(cuuint64_t)dim * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(pages), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, cudaStream_t st) {
  auto kernel = attn_tc_kernel<T, D>;
  constexpr int smem = AttnPlan<D>::kTotal;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.ctas), dim3(kAttnThreads), smem, st, k, v, a);
}

}  // namespace

bool attn_tc_takes(int dim, int page, long long cache_rows) {
  return (dim == 64 || dim == 128 || dim == 256) && page >= 8 && (page & (page - 1)) == 0 && cache_rows < (1ll << 31);
}

cudaError_t launch_attn_tc(int dtype, const AttnArgs& a, cudaStream_t st) {
  CUtensorMap k, v;
  const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page;
  const int box = a.page < a.tile ? a.page : a.tile;
  const bool bf = dtype == SDV_BF16;
  if (!page_map(a.k, bf, rows, a.D, box, &k) || !page_map(a.v, bf, rows, a.D, box, &v)) return cudaErrorUnknown;
  switch (a.D) {
    case 64: return bf ? launch<__nv_bfloat16, 64>(k, v, a, st) : launch<__half, 64>(k, v, a, st);
    case 128: return bf ? launch<__nv_bfloat16, 128>(k, v, a, st) : launch<__half, 128>(k, v, a, st);
    default: return bf ? launch<__nv_bfloat16, 256>(k, v, a, st) : launch<__half, 256>(k, v, a, st);
  }
}

}  // namespace sdv

// Linear attention in chunks of 128 tokens on the 5th-generation tensor cores
// (sm_103a): sdv_linear_attn for prompts and windows, key and value sizes 64 and 128.
//
// With G the cumulative log decay inside a chunk and M the state before it, per head:
//   O_t  = scale (e^{G_t} q_t M + sum_{s <= t} (q_t . k_s) e^{G_t - G_s} v_s)
//   M'   = e^{G_C} M + sum_s e^{G_C - G_s} k_s v_s^T
// as four products of 128 x 128 tiles: Q K^T, Q M, P V (P the decayed scores) and
// U = K~^T V (K~ the decayed keys).  Scores, outputs (Q M, scaled row by row, then P V on
// top), U and the state are fp32 in tensor memory (128 + 3 Dv columns).  The state takes
// U with rounded fp32 operations: added up inside the tensor cores over a long prompt it
// was 5 times less exact.
//
// Precision.  M is a sum over all tokens, so its terms are kept to 22 (fp16) or 24
// (bf16) bits: K~ goes into the product as high and low part, of bf16 as three parts
// (two left the state 3e-6 off where sums of fp32 are 4e-7).  P and the copy of M
// that Q multiplies are rounded to the 16-bit type once, as the values of a matrix
// instruction have to be.  fp16 has neither the range of scores nor of states nor of
// decayed keys, so each carries a power of two: P one per row, M's copy one per chunk,
// K~ one per chunk.  G is summed in pairs of floats and used as differences, so a token
// far behind a reset loses nothing.
//
// The chunks of all heads are dealt to the CTAs in equal contiguous ranges.  A head
// that several CTAs share needs its state at the start of each part: a first launch
// computes each part's own contribution (keys and values alone), and in the second
// one each CTA sums those before it, decayed, on its way in.
//
// Warp roles: 0 TMA; 1 MMA; 2 the decays; 3 the values' end and their largest; then the
// state's (key rows of M: U, decay, 16-bit copy for Q M; four, or eight with outputs,
// where the copy is waited for), the keys' (K~'s parts, then the decay of Q M; eight,
// or four with outputs), four for scores to P and four for outputs.  All of it runs in
// rolled loops: sixteen warps of unrolled code were bound by the instruction cache (three
// times as slow).
//
// A zero weight must not meet an infinite value (0 * inf): keys or values that are not
// finite make U so, its head is noted, its state left unwritten, and the recurrent
// kernel, launched behind, recomputes noted heads by the definition.
//
// Measured: 8192 tokens, 32 heads of 128 x 128 (16 of queries and keys), fp16: 132 us a
// call, 1.6 TB/s of what has to move; of it the first launch 48 us, the second 90, 4 for
// the recurrent kernel that finds nothing to do (each alone, nothing in L2).  Six
// prompts of up to 3001 tokens, 24 heads of 64 x 128, bf16: 102 us, 2.3 TB/s (32, 76, 4).
// bf16's third part is 7 % of that (95 without it), 19 % at 128 x 128 (140 against 118 for
// 8192 tokens): the keys' warps write half as much again, and the room for it is the second
// buffer of keys.
// The memory and the tensor cores (12 to 19 %) wait for a chain of roles: a chunk of the
// second launch is 7 to 8 thousand cycles from U through the state's copy (3 thousand),
// Q M, its decay and P V to the output, at 38 % of the issue slots; 680 KB of shared
// memory traffic a chunk keep that at 5 thousand.  768 threads leave 80 registers each: the
// instances with outputs spill, 28 to 64 bytes a thread.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "linear_args.h"
#include "mixing.h"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kLC = kLinChunk;
constexpr uint64_t kLinDrainNs = 100000000ull;  // 0.1 s: in-flight work at teardown

// x under a decay; one of 0 drops x whatever it holds.
__device__ __forceinline__ float keep(float x, float dec) { return dec == 0.f ? 0.f : x * dec; }

__device__ __forceinline__ uint32_t abs_max2(const uint4& x) {  // of 16-bit magnitudes, per half
  return __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

// A pair of fp16 times f = fh + fl (each in both halves) as the type's nearest (in place)
// and the rest: k fh rounds to h, the rest k fh - h is a value of the type and exact
// (twice the type's bits less those of h), and k fl goes on top: 22 bits.
__device__ __forceinline__ void split16(uint32_t& x, uint32_t fh, uint32_t fl, uint32_t& lo) {
  asm("{\n\t.reg .b32 h, n, r;\n\t"
      "mul.rn.f16x2 h, %0, %2;\n\tneg.f16x2 n, h;\n\t"
      "fma.rn.f16x2 r, %0, %2, n;\n\tfma.rn.f16x2 %1, %0, %3, r;\n\tmov.b32 %0, h;\n\t}"
      : "+r"(x), "=&r"(lo)
      : "r"(fh), "r"(fl));
}

// A pair of bf16 times f in fp32 as three pairs of bf16, the first in place: each takes the
// leading 8 bits of what is left, so the three are the product to its last bit, without a
// conversion.
__device__ __forceinline__ uint32_t upper_halves(f32x2 x) {
  return __byte_perm((uint32_t)x, (uint32_t)(x >> 32), 0x7632);
}
__device__ __forceinline__ f32x2 without_upper(f32x2 x) {
  return fma2(x & 0xffff0000ffff0000ull, pair2(-1.f, -1.f), x);
}
__device__ __forceinline__ void split3(uint32_t& x, f32x2 f, uint32_t& lo, uint32_t& third) {
  const float2 k = unpack16<__nv_bfloat16>(x);
  const f32x2 p = mul2(pair2(k.x, k.y), f), r = without_upper(p);
  x = upper_halves(p);
  lo = upper_halves(r);
  third = upper_halves(without_upper(r));
}

__device__ __forceinline__ uint32_t mul16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// The decays of a chunk, G_t in log2 units.
struct LinTables {
  float hi[kLC], lo[kLC];
  __device__ __forceinline__ DecaySum at(int t) const { return DecaySum{hi[t], lo[t]}; }
};

template <int DK, int DV, bool OUT, bool THIRD>
struct LinPlan {
  // Two buffers of keys, whose place K~'s high part then takes (one where its third part
  // leaves room for no more); the first launch, without queries, state copy and outputs, has
  // room for two of values too, and of the lower parts but where those are three of 128 wide.
  static constexpr int kBufs = OUT ? 1 : 2;  // values
  static constexpr int kLoBufs = OUT || (THIRD && DK == 128) ? 1 : 2;
  static constexpr int kKeyBufs = OUT && THIRD && DK == 128 && DV == 128 ? 1 : 2;
  static constexpr int kThreads = OUT ? 768 : 512;
  static constexpr int kK = kLC * DK * 2, kV = kLC * DV * 2;
  static constexpr int oK = 0, oLo = oK + kKeyBufs * kK, o3 = oLo + kLoBufs * kK;
  static constexpr int oZero = o3 + (THIRD ? kLoBufs * kK : 0);  // Dk = 64: the third part's lower half
  static constexpr int oV = oZero + (THIRD && DK == 64 ? kK : 0), oQ = oV + kBufs * kV;
  static constexpr int oSt = oQ + (OUT ? kK : 0), oOut = oSt + (OUT ? 128 * DV * 2 : 0);
  static constexpr int oEx = oOut + (OUT ? 4 * 4096 : 0);  // Dk = 64: the state's low rows on their way to the high ones
  static constexpr int oTab = oEx + (DK == 64 ? (OUT ? 2 : 1) * 64 * 33 * 4 : 0);
  static constexpr int oFac = oTab + 2 * (int)sizeof(LinTables);  // the scores' warps' factors [4][128]
  static constexpr int oRing = oFac + (OUT ? 4 * kLC * 4 : 0);  // four chunks' decays
  static constexpr int oBars = oRing + 4 * kLC * 4;
  static constexpr int kNumBars = 36;
  static constexpr int oMisc = oBars + kNumBars * 8;
  static constexpr int oUp = oMisc + 256;         // the rows' powers of two [2][128]
  static constexpr int kTotal = oUp + 2 * kLC * 4 + 1024;  // the base is aligned to 1024
  static constexpr int cS = 0, cO = 128, cU = 256, cM = 384;  // tensor-memory columns
  static_assert(kTotal <= 232448 - kWaitLimitBytes, "shared memory");
};

// A CTA's way through its range of chunks; all lanes of a warp keep the same.  The host
// takes this form only where chunks times CTAs stay below 2^31.
struct LinWalk {
  int total, at, end;
  int live, b, h, chunk, n, chunks;

  static __device__ __forceinline__ int chunks_of(int n) { return n <= kLC ? 1 : (n + kLC - 1) / kLC; }
  __device__ __forceinline__ void sequence(const LinArgs& a) {
    n = lin_tokens(a, b);
    chunks = chunks_of(n);
  }
  __device__ __noinline__ bool start(const LinArgs& a, int cta, int lane) {
    // the first 32 sequences' chunks serve for the total and for the search
    const int c0 = lane < a.B ? chunks_of(lin_tokens(a, lane)) : 0;
    int sum = c0;
    for (int s = lane + 32; s < a.B; s += 32) sum += chunks_of(lin_tokens(a, s));
    total = __reduce_add_sync(0xffffffffu, sum) * a.H;
    const long long most = (long long)kLinRuns * a.B * a.H;
    live = min(a.ctas, total);
    if (live > most) live = (int)most;
    if (cta >= live) return false;
    at = (int)((unsigned)(total * cta) / (unsigned)live);
    end = (int)((unsigned)(total * (cta + 1)) / (unsigned)live);
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int mine = (b0 == 0 ? c0 : b0 + lane < a.B ? chunks_of(lin_tokens(a, b0 + lane)) : 0) * a.H;
      int incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
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
    sequence(a);
    const unsigned rest = (unsigned)(at - before);
    h = (int)(rest / (unsigned)chunks);
    chunk = (int)(rest - (unsigned)h * (unsigned)chunks);
    // the first launch takes the range's last part alone, and that only if the head goes on
    if (a.pass == 0) {
      while (more() && chunk + count() == chunks) advance(a, count());
    }
    return more();
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  // chunks of the part that starts here
  __device__ __forceinline__ int count() const { return min(end - at, chunks - chunk); }
  __device__ __noinline__ void advance(const LinArgs& a, int c) {
    at += c;
    chunk += c;
    if (chunk < chunks) return;
    chunk = 0;
    if (++h < a.H) return;
    h = 0;
    if (++b < a.B) sequence(a);
  }
  // The first CTA with chunks of the head.
  __device__ __forceinline__ int first_cta() const {
    return (int)((unsigned)((at - chunk + 1) * live - 1) / (unsigned)total);
  }
};

template <typename T, int DK, int DV, bool OUT>
using LinPlanOf = LinPlan<DK, DV, OUT, std::is_same<T, __nv_bfloat16>::value>;

template <typename T, int DK, int DV, bool OUT>
__global__ void __launch_bounds__(LinPlanOf<T, DK, DV, OUT>::kThreads, 1)
    linear_tc_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs a) {
  using PL = LinPlanOf<T, DK, DV, OUT>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr bool kThird = kBf16;         // three parts of 8 bits make K~ as exact as fp32
  constexpr bool kScaled = !kBf16;       // powers of two beside fp16 operands
  constexpr bool kBound = OUT && kScaled;  // the largest value of a chunk bounds what it adds to M
  constexpr int kStateWarps = OUT ? 8 : 4, kKeyWarps = OUT ? 4 : 8;
  constexpr int kKeys0 = 4 + kStateWarps, kScores0 = kKeys0 + 4, kOut0 = kScores0 + 4;  // the roles' first warps
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const sb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  LinTables* const tabs = reinterpret_cast<LinTables*>(sb + PL::oTab);
  const uint32_t bars = base + PL::oBars;
  auto bar = [&](int i) { return bars + 8u * i; };
  const uint32_t q_full = bar(4), s_full = bar(6), qm_done = bar(7),
                 pv_done = bar(9), p_ready = bar(12), o_free = bar(13),
                 met = bar(14), met_m = bar(15), drain = bar(16), q_read = bar(23);
  // values and lower parts per buffer; a barrier of two takes turns, another one's phase is the chunk
  auto buf = [&](int i) { return PL::kBufs == 2 ? i & 1 : 0; };
  auto lo_at = [&](int i) { return base + PL::oLo + (PL::kLoBufs == 2 ? i & 1 : 0) * PL::kK; };
  auto third_at = [&](int i) { return base + PL::o3 + (PL::kLoBufs == 2 ? i & 1 : 0) * PL::kK; };
  auto u_col = [&](int i) { return !OUT && (i & 1) ? PL::cO : PL::cU; };
  auto phase = [&](int i) { return (uint32_t)(PL::kBufs == 2 ? i >> 1 : i) & 1u; };
  auto k_buf = [&](int i) { return base + PL::oK + (PL::kKeyBufs == 2 ? i & 1 : 0) * PL::kK; };
  auto k_full = [&](int i) { return bar(24 + (i & 1)); };
  auto v_full = [&](int i) { return bar(26 + buf(i)); };
  auto v_free = [&](int i) { return bar(30 + buf(i)); };
  auto upd_done = [&](int i) { return i & 1 ? bar(8) : bar(32); };
  auto m_ready = [&](int i) { return i & 1 ? bar(10) : bar(33); };
  auto kv_ready = [&](int i) { return i & 1 ? bar(11) : bar(34); };
  auto v_seen = [&](int i) { return i & 1 ? bar(5) : bar(17); };
  auto tab_full = [&](int i) { return bar(2 + (i & 1)); };
  auto tab_free = [&](int i) { return bar(18 + (i & 1)); };
  auto up_ready = [&](int i) { return i & 1 ? bar(1) : bar(22); };
  auto ek_ready = [&](int i) { return bar(20 + (i & 1)); };
  volatile int* const misc = reinterpret_cast<int*>(sb + PL::oMisc);
  // misc: 0 tmem base; 2, 3 a part whose values are not all finite; 4, 5 exponent of K~;
  // 6, 7 M's copy's power of two undone; 16-23 the warps' maxima of the state; 24, 25 the
  // chunk's largest value; 32-47 the warps' maxima of the keys
  volatile float* const fmisc = reinterpret_cast<volatile float*>(misc);
  volatile float* const ups = reinterpret_cast<volatile float*>(sb + PL::oUp);

  if (warp == 1) {
    tmem_alloc(base + PL::oMisc, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    set_wait_limit(a.fault);
    for (int i = 0; i < 10; ++i)
      if (i != 1) mbar_init(bar(i), 1);
    mbar_init(upd_done(0), 1);
    mbar_init(o_free, 4);
    mbar_init(met_m, kStateWarps);
    mbar_init(q_read, 4);
    mbar_init(drain, 1);
    mbar_init(v_seen(0), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(24 + i), 1);
      mbar_init(bar(26 + i), 1);
      mbar_init(bar(30 + i), kBound ? 2 + kStateWarps : kScaled ? 1 + kStateWarps : 1);
      mbar_init(m_ready(i), kStateWarps);
      mbar_init(kv_ready(i), kKeyWarps + 1);
    }
    mbar_init(met, kKeyWarps);
    mbar_init(p_ready, 8);
    mbar_init(up_ready(0), 4);
    mbar_init(up_ready(1), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(18 + i), kStateWarps + kKeyWarps + (OUT ? 4 : 0));
      mbar_init(bar(20 + i), 1);
    }
    fence_barrier_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    if (OUT) tma_prefetch_desc(&maps.q);
  }
  if (threadIdx.x >= 32 && threadIdx.x < 34) misc[2 + threadIdx.x - 32] = 0;
  if (kThird && DK == 64) {
    for (int e = threadIdx.x; e < PL::kK / 16; e += PL::kThreads) sts128(base + PL::oZero + 16 * e, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = misc[0];
  // The second launch needs nothing of the first but the parts, and that one has waited for
  // what came before both.
  const bool second = a.pass == 1 && a.T > kLC;
  if (!second) griddep_wait();
  griddep_launch_dependents();
  bool ok = true;
  auto await = [&](uint32_t b, uint32_t parity) {
    if (ok) ok = mbar_wait_warp(b, parity, a.status);
    return ok;
  };
  auto arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  // Barriers that complete once a chunk: a role waits for every phase, in order, before
  // the next can complete.
  int upd_seen = 0, pv_seen = 0;
  auto upd_wait = [&](int chunks) {
    for (; upd_seen < chunks; ++upd_seen)
      if (!await(upd_done(upd_seen), (upd_seen >> 1) & 1)) return false;
    return true;
  };
  auto pv_wait = [&](int chunks) {
    for (; pv_seen < chunks; ++pv_seen)
      if (!await(pv_done, pv_seen & 1)) return false;
    return true;
  };
  LinWalk from;
  const bool any = from.start(a, blockIdx.x, lane);
  LinWalk w = from;
  int i = 0;  // the CTA's chunk number

  if (warp == 0) {
    // ---- TMA ----
    const uint64_t normal = l2_policy_normal();
    const uint64_t v_policy = OUT ? l2_policy_evict_first() : normal;  // the second launch reads values last
    const int shared = a.H / a.Hqk;
    int asked_k = 0, asked_q = 0, asked_v = 0;
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count(), hk = w.h / shared;
      const int z0 = w.b * a.T + w.chunk * kLC;
      for (int c = 0; c < count; ++c, ++i) {
        const int z = z0 + c * kLC;
        // the product with K~ that took the place of the keys before in this buffer
        if (OUT ? !upd_wait(i + 1 - PL::kKeyBufs) : i >= 2 && !await(v_free(i), phase(i - 2))) break;
        if (++asked_k != a.fault.withhold) {
          if (lane == 0) mbar_arrive_expect_tx(k_full(i), PL::kK);
          __syncwarp();
          if (lane < DK / 64)
            tma_load_3d(k_buf(i) + lane * 16384, &maps.k, lane * 64, hk, z, k_full(i), normal);
        }
        if (OUT) {
          if (i > 0 && (!await(qm_done, (i - 1) & 1) || (kScaled && !await(q_read, (i - 1) & 1)))) break;
          if (lane == 0) mbar_arrive_expect_tx(q_full, PL::kK);
          __syncwarp();
          if (lane < DK / 64) tma_load_3d(base + PL::oQ + lane * 16384, &maps.q, lane * 64, hk, z, q_full, normal);
          ++asked_q;
        }
        // the values before in this buffer: read by the products and by their check
        if (OUT && i > 0 && !await(v_free(i), (i - 1) & 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(v_full(i), PL::kV);
        __syncwarp();
        if (lane < DV / 64)
          tma_load_3d(base + PL::oV + buf(i) * PL::kV + lane * 16384, &maps.v, lane * 64, w.h, z, v_full(i), v_policy);
        ++asked_v;
      }
      if (!ok) break;
      w.advance(a, count);
    }
    // The last copies have to land before the CTA ends, whoever else gives up waiting for
    // them, and when.  (The same behind the block's barrier, for dead CTAs alone, made a
    // prompt 3 % slower.)
    for (int e = max(asked_k - 2, 0); e < asked_k; ++e)
      if (e + 1 != a.fault.withhold) mbar_wait_bounded(k_full(e), (e >> 1) & 1, kLinDrainNs);
    for (int e = max(asked_v - PL::kBufs, 0); e < asked_v; ++e) mbar_wait_bounded(v_full(e), phase(e), kLinDrainNs);
    if (asked_q > 0) mbar_wait_bounded(q_full, (asked_q - 1) & 1, kLinDrainNs);
  } else if (warp == 1) {
    // ---- MMA: every lane keeps the same state, one elected lane issues ----
    constexpr uint32_t id_qk = idesc_16_f32(kBf16, 128, kLC, false, false);
    constexpr uint32_t id_kb = idesc_16_f32(kBf16, 128, DV, false, true);  // Q M and P V
    constexpr uint32_t id_up = idesc_16_f32(kBf16, 128, DV, true, true);
    const uint64_t qd = smem_desc_sw128(base + PL::oQ, 16, 1024);
    const uint64_t md = smem_desc_sw128(base + PL::oSt, 16384, 1024);
    // the chunks of all parts follow each other alike; a uniform count keeps the operands
    // in uniform registers
    const int total = __reduce_max_sync(0xffffffffu, any ? (int)(w.end - w.at) : 0);
    for (; ok && i < total; ++i) {
      const uint64_t vd = smem_desc_sw128(base + PL::oV + buf(i) * PL::kV, 16384, 1024);
      if (OUT) {
        // scores; P of the chunk before has been read
        if (!pv_wait(i) || !await(q_full, i & 1) || !await(k_full(i), (i >> 1) & 1)) break;
        tc_fence_after();
        const uint64_t kd = smem_desc_sw128(k_buf(i), 16, 1024);
#pragma unroll 1
        for (int j = 0; j < DK / 64; ++j)
          tc_mma4_ss<2, 2>(tm + PL::cS, qd + j * 1024, kd + j * 1024, id_qk, j > 0);
        tc_commit_elect(s_full);
      }
      // M's copy; the first launch, with two buffers of U, wants U's before taken
      if (OUT ? !await(m_ready(i), (i >> 1) & 1) : i > 0 && !await(m_ready(i - 1), ((i - 1) >> 1) & 1)) break;
      if (OUT) {
        // Q M over M's copy: 128 rows (at Dk = 64 the state's high and low part, both by Q)
        if (i > 0 && !await(o_free, (i - 1) & 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < 2; ++j)
          tc_mma4_ss<2, 128>(tm + PL::cO, qd + (DK == 128 ? j * 1024 : 0), md + j * 512, id_kb, j > 0);
        tc_commit_elect(qm_done);
      }
      if (!await(kv_ready(i), (i >> 1) & 1)) break;
      tc_fence_after();
      // K~^T V: the lowest parts first; at Dk = 64 high and low at once (rows 0-63 from the
      // high, 64-127 from the low part), and before them the third part over zeros
      const uint32_t lo = lo_at(i), third = third_at(i);
      if constexpr (DK == 128) {
        const uint64_t hd = smem_desc_sw128(k_buf(i), 16384, 1024), ld = smem_desc_sw128(lo, 16384, 1024);
        const uint64_t td = smem_desc_sw128(third, 16384, 1024);
#pragma unroll 1
        for (int j = kThird ? -2 : 0; j < 4; ++j)
          tc_mma4_ss<128, 128>(tm + u_col(i), (j < 0 ? td : j < 2 ? ld : hd) + (j & 1) * 512, vd + (j & 1) * 512, id_up,
                               j > (kThird ? -2 : 0));
      } else {
        const uint64_t bd = smem_desc_sw128(k_buf(i), lo - k_buf(i), 1024);
        const uint64_t td = smem_desc_sw128(third, base + PL::oZero - third, 1024);
#pragma unroll 1
        for (int j = kThird ? -2 : 0; j < 2; ++j)
          tc_mma4_ss<128, 128>(tm + u_col(i), (j < 0 ? td : bd) + (j & 1) * 512, vd + (j & 1) * 512, id_up,
                               j > (kThird ? -2 : 0));
      }
      tc_commit_elect(upd_done(i));
      if (!OUT) tc_commit_elect(v_free(i));
      if (OUT) {
        if (!await(p_ready, i & 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < 2; ++j) tc_mma4_ts(tm + PL::cO, tm + PL::cS + j * 32, vd + j * 512, id_kb, 1);
        tc_commit_elect(pv_done);
        tc_commit_elect(v_free(i));
      }
    }
    tc_commit_elect(drain);  // every MMA has ended before tensor memory is freed
    mbar_wait_bounded(drain, 0, kLinDrainNs);
  } else if (warp == 2) {
    // ---- decays: four tokens a lane, sums in pairs of floats ----
    DecaySum run;  // log2 decay of the part so far
    // natural log decays, asked for three chunks ahead of their use (a chunk takes less than
    // memory under this load does) into a ring of shared memory; a lane reads its own
    const uint32_t ring = base + PL::oRing + 16 * lane;
    auto ask = [&](int c, int count) {
      if (c < count) {
        const int t = (w.chunk + c) * kLC + 4 * lane;
        const float* const from = a.g + (a.g_token ? ((long long)w.b * a.T + t) * a.H + w.h : w.h);
        const int step = a.g_token ? a.H : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          cp_async4(ring + (c & 3) * (kLC * 4) + 4 * e, t + e < w.n ? from + e * step : a.g, t + e < w.n);
      }
      cp_async_commit();
    };
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
#pragma unroll 1
      for (int c = -3; c < count; ++c) {
        ask(c + 3, count);
        if (c < 0) continue;
        cp_async_wait<3>();
        const uint4 x = lds128(ring + (c & 3) * (kLC * 4));
        const uint32_t given[4] = {x.x, x.y, x.z, x.w};
        DecaySum g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = DecaySum::log2_of(lin_clamp_decay(__uint_as_float(given[e])));
#pragma unroll
        for (int e = 1; e < 4; ++e) g[e].add(g[e - 1]);
        DecaySum incl = g[3];
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
          const DecaySum o{__shfl_up_sync(0xffffffffu, incl.hi, off), __shfl_up_sync(0xffffffffu, incl.lo, off)};
          if (lane >= off) incl.add(o);
        }
        DecaySum before{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
        if (lane == 0) before = DecaySum();
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e].add(before);
        if (i >= 2 && !await(tab_free(i), ((i - 2) >> 1) & 1)) break;
        LinTables& tb = tabs[i & 1];
        reinterpret_cast<float4*>(tb.hi)[lane] = make_float4(g[0].hi, g[1].hi, g[2].hi, g[3].hi);
        reinterpret_cast<float4*>(tb.lo)[lane] = make_float4(g[0].lo, g[1].lo, g[2].lo, g[3].lo);
        if (a.pass == 0) run.add(DecaySum{__shfl_sync(0xffffffffu, g[3].hi, 31), __shfl_sync(0xffffffffu, g[3].lo, 31)});
        arrive(tab_full(i));
        ++i;
      }
      if (!ok) break;
      if (a.pass == 0 && lane == 0) a.parts[blockIdx.x].decay = run;
      w.advance(a, count);
    }
    cp_async_wait<0>();
  } else if (warp == 3) {
    // ---- the values: zeros behind the end, the largest ----
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
      for (int c = 0; c < count; ++c, ++i) {
        const int nv = w.n - (w.chunk + c) * kLC;  // tokens of the chunk
        if (!await(v_full(i), phase(i))) break;
        const uint32_t vb = base + PL::oV + buf(i) * PL::kV;
        if (nv < kLC) {
          for (int e = max(nv, 0) * 8 + lane; e < kLC * 8; e += 32)
#pragma unroll
            for (int h = 0; h < DV / 64; ++h) sts128(vb + h * 16384 + swz128(e >> 3, e & 7), make_uint4(0, 0, 0, 0));
          fence_proxy_async_smem();
        }
        arrive(kv_ready(i));  // the search reads beside the products
        if (!kBound) continue;
        uint32_t mx = 0;
#pragma unroll 1
        for (int e = 0; e < DV / 16; ++e) {  // rows 32 (e % 4) + lane, 64 columns
          const uint32_t row = vb + (e >> 2) * 16384;
          const int r = 32 * (e & 3) + lane;
          uint4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = lds128(row + swz128(r, k));
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = __vmaxu2(mx, abs_max2(x[k]));
        }
        mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
        if (lane == 0) fmisc[24 + (i & 1)] = __half2float(__ushort_as_half((unsigned short)min(mx, 0x7bffu)));
        arrive(v_seen(i));
        if (lane == 0) mbar_arrive(v_free(i));
      }
      if (!ok) break;
      w.advance(a, count);
    }
  } else if (warp < kKeys0) {
    // ---- the state: thread = key row of M, or half of one (at Dk = 64: rows 64-127 hold the low part) ----
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tq = tm + ((uint32_t)(quarter * 32) << 16);
    const int half = (warp - 4) >> 2;  // at eight warps a thread has half of the columns
    const int col0 = half * (DV / 2), col1 = kStateWarps == 8 ? col0 + DV / 2 : DV;
    const bool owner = r < DK;  // rows with a place in the state's array
    uint32_t meetings = 0;
    int part = 0;
    if (second) griddep_wait();
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
      const long long unit = (long long)w.b * a.H + w.h;
      // the state before the part: what was given, then the parts before this one, in order
      float bound = 0.f;  // of M's finite entries: what they start at, then what a chunk can add
      const int first = a.pass == 1 && w.chunk > 0 ? w.first_cta() : (int)blockIdx.x;
      // Another CTA writes a shared head's final state, perhaps over the given one: the
      // second launch takes the first one's copy of that.
      const bool ends = w.chunk + count == w.chunks, whole = w.chunk == 0 && ends;
      if (a.pass == 0 && w.chunk == 0 && a.s_in != nullptr) {
        const float4* const from4 = reinterpret_cast<const float4*>(a.s_in + unit * DK * DV);
        float4* const to4 = reinterpret_cast<float4*>(a.part_in + (long long)blockIdx.x * DK * DV);
#pragma unroll 4
        for (int e = threadIdx.x - 128; e < DK * DV / 4; e += 32 * kStateWarps) to4[e] = from4[e];
      }
#pragma unroll 1
      for (int j = col0; j < col1; j += 32) {
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0.f;
        if (owner && a.pass == 1) {
#pragma unroll 1
          for (int c = first - 1; c < (int)blockIdx.x; ++c) {
            if (c < first && a.s_in == nullptr) continue;
            // a row of the given state; the parts' lie column by column, as this reads them
            const float* const src = c >= first ? a.part + (long long)c * DK * DV + (j * DK + r * 4)
                                     : whole    ? a.s_in + (unit * DK + r) * DV + j
                                                : a.part_in + ((long long)first * DK + r) * DV + j;
            const int step = c < first ? 4 : DK * 4;
            float dec = 0.f;
            if (c >= first) dec = exp2f(a.parts[c].decay.hi + a.parts[c].decay.lo);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = *reinterpret_cast<const float4*>(src + e / 4 * step);
              x[e] = keep(x[e], dec) + y.x;
              x[e + 1] = keep(x[e + 1], dec) + y.y;
              x[e + 2] = keep(x[e + 2], dec) + y.z;
              x[e + 3] = keep(x[e + 3], dec) + y.w;
            }
          }
        }
        tmem_st32(tq + PL::cM + j, reinterpret_cast<const uint32_t*>(x));
        if (OUT && kScaled) {
#pragma unroll
          for (int e = 0; e < 32; ++e) bound = fmaxf(bound, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.f);
        }
      }
      tmem_wait_st();
      if (OUT && kScaled) {
        const uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(bound));
        if (lane == 0) misc[warp + 12] = (int)mx;
        arrive(met_m);
        if (!await(met_m, meetings++ & 1)) break;
        int top = 0;
#pragma unroll
        for (int e = 0; e < kStateWarps; ++e) top = max(top, misc[16 + e]);
        bound = __int_as_float(top);
      }
      auto take_u = [&](int chunks) {  // the last chunk's U is there, and its largest value
        if (!upd_wait(chunks)) return false;
        if (kBound) {
          if (!await(v_seen(chunks - 1), ((chunks - 1) >> 1) & 1)) return false;
          if (lane == 0) mbar_arrive(v_free(chunks - 1));
        }
        tc_fence_after();
        return true;
      };
      float dec = 0.f, dn = 1.f;  // of the last chunk: M = dec M + dn U
      // 0 times U, summed: NaN once a key or value of the part is not finite, which makes
      // a row or column of U so (0 times it is NaN)
      f32x2 odd = pair2(0.f, 0.f);
      auto state_of = [&](int j, uint32_t (&x)[32], bool take) {  // 32 columns of M behind the last chunk
        tmem_ld32(tq + PL::cM + j, x);
        if (!take) {
          tmem_wait_ld();
          return;
        }
        uint32_t u[32];
        tmem_ld32(tq + u_col(i - 1) + j, u);
        tmem_wait_ld();
        if (dec == 0.f) {  // drops M whatever it holds
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0u;
        }
        const f32x2 dec2 = pair2(dec, dec), dn2 = pair2(dn, dn);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const f32x2 u2 = pair2(__uint_as_float(u[e]), __uint_as_float(u[e + 1]));
          odd = fma2(u2, pair2(0.f, 0.f), odd);
          const float2 y = unpair2(fma2(u2, dn2, mul2(pair2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), dec2)));
          x[e] = __float_as_uint(y.x);
          x[e + 1] = __float_as_uint(y.y);
        }
      };
      auto copy_out = [&](int j, const uint32_t (&x)[32], float cs) {  // M's copy for Q M
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            y[z] = pack16<T>(mul2(pair2(__uint_as_float(x[e + 2 * z]), __uint_as_float(x[e + 2 * z + 1])), pair2(cs, cs)));
          sts128(base + PL::oSt + (j >> 6) * 16384 + swz128(r, ((j & 32) + e) >> 3), make_uint4(y[0], y[1], y[2], y[3]));
        }
      };
      for (int c = 0; c < count; ++c, ++i) {
        if (c > 0 && !take_u(i)) break;
        if (OUT || c > 0) {
          float cs = 1.f;  // what M's copy carries
          if (OUT && kScaled) {
            // |U| is at most 128 times the largest |k~| (below 2^15 in U's units) times the
            // largest value: the bound is loose by the square root of what it counts, far
            // within what fp16's 30 octaves leave
            if (c > 0) bound = bound * dec + 4194304.f * dn * fmisc[24 + ((i - 1) & 1)];
            const int ex = min(max((int)(__float_as_uint(bound) >> 23) - 127, -100), 120);
            cs = exp2f((float)(14 - ex));  // the bound to [2^14, 2^15)
            if (warp == 4 && lane == 0) fmisc[6 + (i & 1)] = exp2f((float)(ex - 14));
          }
#pragma unroll 1
          for (int j = col0; j < col1; j += 32) {
            uint32_t x[32];
            state_of(j, x, c > 0);
            if (c > 0) tmem_st32(tq + PL::cM + j, x);
            if (OUT) copy_out(j, x, cs);
          }
          if (OUT) fence_proxy_async_smem();
          tmem_wait_st();
        }
        // this chunk's factors, before the product may go on (the next but one's come after it)
        if (!await(tab_full(i), (i >> 1) & 1)) break;
        dec = exp2_approx(tabs[i & 1].hi[kLC - 1] + tabs[i & 1].lo[kLC - 1]);
        arrive(tab_free(i));
        if (kScaled) {
          if (!await(ek_ready(i), (i >> 1) & 1)) break;
          dn = exp2f((float)-misc[4 + (i & 1)]);
          // without outputs the product does not wait for this: the next keys here do
          if (!OUT) {
            __syncwarp();
            if (lane == 0) mbar_arrive(v_free(i));
          }
        }
        tc_fence_before();
        arrive(m_ready(i));
      }
      if (!ok || !take_u(i)) break;
      // into the array if the head ends here, else this CTA's contribution
#pragma unroll 1
      for (int j = col0; j < col1; j += 32) {  // the last U
        uint32_t u[32];
        tmem_ld32(tq + u_col(i - 1) + j, u);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          odd = fma2(pair2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), pair2(0.f, 0.f), odd);
      }
      if (unpair2(odd).x != 0.f || unpair2(odd).y != 0.f) misc[2 + (part & 1)] = part + 1;
      arrive(met_m);
      if (!await(met_m, meetings++ & 1)) break;
      float* dst = nullptr;
      int bad = misc[2 + (part & 1)] == part + 1;
      if (a.pass == 0) {
        dst = a.part + (long long)blockIdx.x * DK * DV;
        if (threadIdx.x == 128) a.parts[blockIdx.x].bad = bad;
      } else if (ends) {
        for (int c = first; c < (int)blockIdx.x; ++c) bad |= a.parts[c].bad;
        if (threadIdx.x == 128) a.repair[unit] = bad;
        if (!bad) dst = a.s_out != nullptr ? a.s_out + unit * DK * DV : nullptr;
      }
#pragma unroll 1
      for (int j = col0; j < col1; j += 32) {
        uint32_t x[32];
        state_of(j, x, true);
        if constexpr (DK == 64) {
          // rows 64-127 add theirs to rows 0-63
          float* const ex = reinterpret_cast<float*>(sb + PL::oEx) + half * 64 * 33;
          if (!owner) {
#pragma unroll
            for (int e = 0; e < 32; ++e) ex[(r - 64) * 33 + e] = __uint_as_float(x[e]);
          }
          arrive(met_m);
          if (!await(met_m, meetings++ & 1)) break;
          if (owner) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) + ex[r * 33 + e]);
          }
          arrive(met_m);
          if (!await(met_m, meetings++ & 1)) break;
        }
        if (owner && dst != nullptr) {
          float4* const p = reinterpret_cast<float4*>(a.pass == 0 ? dst + j * DK + r * 4 : dst + (long long)r * DV + j);
          const int step = a.pass == 0 ? DK : 1;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            p[e * step] = make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]), __uint_as_float(x[4 * e + 2]),
                               __uint_as_float(x[4 * e + 3]));
        }
      }
      if (!ok) break;
      tc_fence_before();
      ++part;
      w.advance(a, count);
    }
  } else if (warp < kKeys0 + kKeyWarps) {
    // ---- keys: thread = token, at eight warps half of its elements ----
    const int quarter = warp & 3, r = quarter * 32 + lane;
    constexpr int kUnits = DK / 8 / (kKeyWarps / 4);  // a thread's 16-byte units
    const int u0 = (warp - kKeys0) / 4 * kUnits;
    uint32_t meetings = 0;
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
      for (int c = 0; c < count; ++c, ++i) {
        const int nv = w.n - (w.chunk + c) * kLC;  // tokens of the chunk
        const uint32_t kb = k_buf(i);
        if (!await(k_full(i), (i >> 1) & 1)) break;
        float up = 1.f;
        int pre = 0;
        if (kScaled) {
          // the largest key of the chunk sets its power of two
          uint32_t mx = 0;
          if (r < nv) {
#pragma unroll 1
            for (int h = u0; h < u0 + kUnits; h += 4) {
              uint4 x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = lds128(kb + (h >> 3) * 16384 + swz128(r, (h & 7) + k));
#pragma unroll
              for (int k = 0; k < 4; ++k) mx = __vmaxu2(mx, abs_max2(x[k]));
            }
            mx = max(mx & 0xffffu, mx >> 16);
          }
          mx = __reduce_max_sync(0xffffffffu, mx);
          if (lane == 0) misc[32 + 8 * (i & 1) + warp - kKeys0] = (int)mx;
          arrive(met);
          if (!await(met, meetings++ & 1)) break;
          int bits = 0;
#pragma unroll
          for (int e = 0; e < kKeyWarps; ++e) bits = max(bits, misc[32 + 8 * (i & 1) + e]);
          const float top = __half2float(__ushort_as_half((unsigned short)min(bits, 0x7bff)));
          const int ex = top == 0.f ? 0 : (int)(__float_as_uint(top) >> 23) - 127;
          // the largest to [2^14, 2^15): low parts then end at 2^-39 of it.  2^15 of it goes
          // into the factor (times a decay it has to be a fp16 value), the rest of small
          // keys' into the keys, exactly.
          const int ek = min(14 - ex, 30);  // -1 .. 30
          pre = max(ek - 15, 0);
          up = exp2f((float)(ek - pre));
          if (warp == kKeys0 && lane == 0) {
            misc[4 + (i & 1)] = ek;
            mbar_arrive(ek_ready(i));
          }
        }
        if (!await(tab_full(i), (i >> 1) & 1)) break;
        const float f = r < nv ? exp2_approx(tabs[i & 1].at(kLC - 1).minus(tabs[i & 1].at(r))) * up : 0.f;  // e^{G_C - G_s}
        const uint32_t fh = pack16<T>(f, f);
        const float eg = OUT ? exp2_approx(tabs[i & 1].hi[r] + tabs[i & 1].lo[r]) : 0.f;  // e^{G_t}
        const float fr = f - unpack16<T>(fh).x;
        const uint32_t fl = pack16<T>(fr, fr);
        const float pw = exp2f((float)pre);
        const uint32_t up2 = pack16<T>(pw, pw);
        arrive(tab_free(i));
        // the last product has read K~'s lower parts, Q K^T the keys
        if ((PL::kLoBufs == 1 && !upd_wait(i)) || (OUT && !await(s_full, i & 1))) break;
#pragma unroll 1
        for (int h = u0; h < u0 + kUnits; h += 4) {  // four 16-byte units in flight
          const uint32_t blk = (h >> 3) * 16384;
          uint4 x[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = lds128(kb + blk + swz128(r, (h & 7) + k));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (r >= nv) x[k] = make_uint4(0, 0, 0, 0);
            if (pre > 0) {
              x[k].x = mul16x2(x[k].x, up2);
              x[k].y = mul16x2(x[k].y, up2);
              x[k].z = mul16x2(x[k].z, up2);
              x[k].w = mul16x2(x[k].w, up2);
            }
            if constexpr (kThird) {
              const f32x2 f2 = pair2(f, f);
              uint4 third;
              split3(x[k].x, f2, lo[k].x, third.x);
              split3(x[k].y, f2, lo[k].y, third.y);
              split3(x[k].z, f2, lo[k].z, third.z);
              split3(x[k].w, f2, lo[k].w, third.w);
              sts128(third_at(i) + blk + swz128(r, (h & 7) + k), third);
              continue;
            }
            split16(x[k].x, fh, fl, lo[k].x);
            split16(x[k].y, fh, fl, lo[k].y);
            split16(x[k].z, fh, fl, lo[k].z);
            split16(x[k].w, fh, fl, lo[k].w);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sts128(kb + blk + swz128(r, (h & 7) + k), x[k]);
            sts128(lo_at(i) + blk + swz128(r, (h & 7) + k), lo[k]);
          }
        }
        fence_proxy_async_smem();
        arrive(kv_ready(i));
        if (OUT) {
          // the state's part of the output, in the units of P V: by e^{G_t}, M's copy's power
          // of two and the row's
          float rise = 1.f;
          if (kScaled) {
            if (!await(up_ready(i), (i >> 1) & 1)) break;
            rise = ups[(i & 1) * kLC + r];
          }
          if (!await(qm_done, i & 1)) break;
          tc_fence_after();
          const float by = eg * (kScaled ? fmisc[6 + (i & 1)] : 1.f) * rise;
          const f32x2 by2 = pair2(by, by);
          const bool drop = eg == 0.f;  // whatever the state holds
          const uint32_t to = tm + PL::cO + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
          for (int j = 0; j < DV; j += 32) {
            uint32_t x[32];
            tmem_ld32(to + j, x);
            tmem_wait_ld();
            if (__any_sync(0xffffffffu, drop)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (drop) x[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = unpair2(mul2(pair2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), by2));
              x[e] = __float_as_uint(y.x);
              x[e + 1] = __float_as_uint(y.y);
            }
            tmem_st32(to + j, x);
          }
          tmem_wait_st();
          tc_fence_before();
          arrive(p_ready);
        }
      }
      if (!ok) break;
      w.advance(a, count);
    }
  } else if (OUT && warp < kOut0) {
    // ---- scores: thread = token ----
    const int quarter = warp & 3, t = quarter * 32 + lane;
    const uint32_t tq = tm + ((uint32_t)(quarter * 32) << 16);
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
      for (int c = 0; c < count; ++c, ++i) {
        if (!await(tab_full(i), (i >> 1) & 1)) break;
        const LinTables& tb = tabs[i & 1];
        // e^{G_t - G_s} = e^{G_t - G_r} e^{G_r - G_s}, r the last token before the warp's
        // block of 32 (G_r = 0 in the first): exact enough for s <= r, and inside the block
        // where that decays by less than 2^-60
        const DecaySum gt = tb.at(t), gr = quarter > 0 ? tb.at(quarter * 32 - 1) : DecaySum();
        const bool mild = tb.at(quarter * 32 + 31).minus(gr) > -60.f;
        float* const fac = reinterpret_cast<float*>(sb + PL::oFac) + quarter * kLC;
        __syncwarp();  // the last chunk's have been read
        for (int j = 0; j <= quarter; ++j)
          if (j < quarter || mild) fac[32 * j + lane] = exp2_approx(gr.minus(tb.at(32 * j + lane)));
        __syncwarp();
        // fp16: a bound of the row's scores sets its power of two: Dk times the row's largest
        // query times the chunk's largest key
        float up = 1.f;
        if (kScaled) {
          if (!await(q_full, i & 1)) break;
          uint32_t mx = 0;
#pragma unroll 1
          for (int h = 0; h < DK / 8; h += 4) {
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = lds128(base + PL::oQ + (h >> 3) * 16384 + swz128(t, (h & 7) + k));
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = __vmaxu2(mx, abs_max2(x[k]));
          }
          arrive(q_read);
          mx = min(max(mx & 0xffffu, mx >> 16), 0x7bffu);
          const float top = __half2float(__ushort_as_half((unsigned short)mx));
          if (!await(ek_ready(i), (i >> 1) & 1)) break;
          // |q| below 2^(eq + 1), |k| below 2^(15 - ek), 2^7 products at most
          const int eq = (int)(__float_as_uint(top) >> 23) - 127;
          const int eu = min(14 - (eq + 1 + 15 - misc[4 + (i & 1)] + 7), 40);
          up = exp2f((float)eu);
          ups[(i & 1) * kLC + t] = up;
          arrive(up_ready(i));
        }
        if (!await(s_full, i & 1)) break;
        tc_fence_after();
        const uint32_t ts = tq + PL::cS;
        const float rf = exp2_approx(gt.minus(gr)) * up;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          uint32_t y[16];
          if (j <= quarter) {
            uint32_t x[32];
            tmem_ld32(ts + 32 * j, x);
            tmem_wait_ld();
            if (j < quarter || mild) {
              const float4* const cf = reinterpret_cast<const float4*>(fac + 32 * j);
              const f32x2 r2 = pair2(rf, rf);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 f = cf[e];
                y[2 * e] = pack16<T>(mul2(pair2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])),
                                          mul2(pair2(f.x, f.y), r2)));
                y[2 * e + 1] = pack16<T>(mul2(pair2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])),
                                              mul2(pair2(f.z, f.w), r2)));
              }
              if (j == quarter) {  // tokens behind t
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] &= 2 * e + 1 <= lane ? 0xffffffffu : 2 * e <= lane ? 0x0000ffffu : 0u;
              }
            } else {
              const float4* const h4 = reinterpret_cast<const float4*>(tb.hi + 32 * j);
              const float4* const l4 = reinterpret_cast<const float4*>(tb.lo + 32 * j);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 hs = h4[e], ls = l4[e];
                const float d0 = (gt.hi - hs.x) + (gt.lo - ls.x), d1 = (gt.hi - hs.y) + (gt.lo - ls.y);
                const float d2 = (gt.hi - hs.z) + (gt.lo - ls.z), d3 = (gt.hi - hs.w) + (gt.lo - ls.w);
                const float p0 = 4 * e <= lane ? __uint_as_float(x[4 * e]) * (up * exp2_approx(d0)) : 0.f;
                const float p1 = 4 * e + 1 <= lane ? __uint_as_float(x[4 * e + 1]) * (up * exp2_approx(d1)) : 0.f;
                const float p2 = 4 * e + 2 <= lane ? __uint_as_float(x[4 * e + 2]) * (up * exp2_approx(d2)) : 0.f;
                const float p3 = 4 * e + 3 <= lane ? __uint_as_float(x[4 * e + 3]) * (up * exp2_approx(d3)) : 0.f;
                y[2 * e] = pack16<T>(p0, p1);
                y[2 * e + 1] = pack16<T>(p2, p3);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = 0u;
          }
          tmem_st16(ts + 16 * j, y);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(p_ready);
        arrive(tab_free(i));
      }
      if (!ok) break;
      w.advance(a, count);
    }
  } else if (OUT) {
    // ---- outputs: thread = token, then rows as 128-byte lines ----
    // first the zeros behind the sequences' ends, whole chunks (heads dealt to the CTAs)
    if (a.n_tokens != nullptr) {
#pragma unroll 1
      for (int u = blockIdx.x; u < a.B * a.H; u += gridDim.x) {
        const int b = u / a.H, h = u - b * a.H;
        constexpr int per = DV / 8;  // 16-byte units of a row
        const int e = (warp - kOut0) * 32 + lane;
        int t = LinWalk::chunks_of(lin_tokens(a, b)) * kLC + e / per;
        uint4* p = reinterpret_cast<uint4*>(a.o) + (((long long)b * a.T + t) * a.H + h) * per + e % per;
#pragma unroll 1
        for (; t < a.T; t += 128 / per, p += 128 / per * a.H * per) *p = make_uint4(0, 0, 0, 0);
      }
    }
    const int quarter = warp & 3, t = quarter * 32 + lane;
    const uint32_t tq = tm + PL::cO + ((uint32_t)(quarter * 32) << 16);
    const uint32_t stage = base + PL::oOut + quarter * 4096;
    for (bool more = any; ok && more; more = w.more()) {
      const int count = w.count();
      for (int c = 0; c < count; ++c, ++i) {
        if (!pv_wait(i + 1)) break;
        tc_fence_after();
        // (a power of two; the scores' warps have left it long ago)
        const float f = kScaled ? a.scale / ups[(i & 1) * kLC + t] : a.scale;
        const int row = (w.chunk + c) * kLC + quarter * 32 + (lane >> 3);
        T* const dst = static_cast<T*>(a.o) + (((long long)w.b * a.T + row) * a.H + w.h) * DV + (lane & 7) * 8;
        // 64 columns at a time through shared memory; all of them leave tensor memory first
        uint32_t y[32];
        auto take = [&](int j) {
#pragma unroll
          for (int hf = 0; hf < 64; hf += 32) {
            uint32_t x[32];
            tmem_ld32(tq + j + hf, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              y[(hf + e) / 2] = pack16<T>(mul2(pair2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), pair2(f, f)));
          }
        };
        take(0);
#pragma unroll 1
        for (int j = 0; j < DV; j += 64) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sts128(stage + swz128(lane, e), make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
          if (j + 64 < DV) take(j + 64);
          if (j == 0) {
            tc_fence_before();
            arrive(o_free);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint4 v = lds128(stage + swz128(4 * k + (lane >> 3), lane & 7));
            if (row + 4 * k >= w.n) v = make_uint4(0, 0, 0, 0);  // behind the sequence's end
            if (row + 4 * k < a.T) *reinterpret_cast<uint4*>(dst + (long long)4 * k * a.H * DV + j) = v;
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      w.advance(a, count);
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

template <typename T, int DK, int DV, bool OUT>
cudaError_t linear_tc_launch(const LinMaps& m, const LinArgs& a, cudaStream_t st) {
  auto kernel = linear_tc_kernel<T, DK, DV, OUT>;
  // more than half an SM's: one CTA and one tensor-memory allocation per SM
  constexpr int half = 232448 / 2 + 1024;
  using PL = LinPlanOf<T, DK, DV, OUT>;
  constexpr int smem = PL::kTotal > half ? PL::kTotal : half;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(a.ctas), dim3(PL::kThreads), smem, st, m, a);
}

}  // namespace

template <typename T>
cudaError_t linear_tc_dispatch(const LinMaps& m, const LinArgs& a, cudaStream_t st) {
  const bool out = a.pass == 1 && a.o != nullptr;
  if (a.Dk == 128 && a.Dv == 128)
    return out ? linear_tc_launch<T, 128, 128, true>(m, a, st) : linear_tc_launch<T, 128, 128, false>(m, a, st);
  if (a.Dk == 128)
    return out ? linear_tc_launch<T, 128, 64, true>(m, a, st) : linear_tc_launch<T, 128, 64, false>(m, a, st);
  if (a.Dv == 128)
    return out ? linear_tc_launch<T, 64, 128, true>(m, a, st) : linear_tc_launch<T, 64, 128, false>(m, a, st);
  return out ? linear_tc_launch<T, 64, 64, true>(m, a, st) : linear_tc_launch<T, 64, 64, false>(m, a, st);
}

}  // namespace sdv

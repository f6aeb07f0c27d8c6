// Verification of drafted tokens against the target's probabilities, and the draw of the next
// token, from given random numbers (sdv_verify_drafts).
//
//   p_i = softmax(logits_i / T);  draft d_i is kept while u_i q_i(d_i) < p_i(d_i);  at the first
//   one that is not, the next token is drawn from max(p_i - q_i, 0), else from p_n:
//   the lowest v whose running weight exceeds u_S-1 of the total.
//
// Two launches.  The first reads every row once: per chunk of 1024 logits the maximum m and
// sum 2^(x c - K), c = log2(e) / T, K = ceil(m c) (or, greedy, the place of the maximum).  The
// second joins the rows' sums, runs the tests and draws: from a row of the target by the chunks'
// sums and one more look at one chunk; from what a drafter's probabilities leave of a row by a
// pass over it with a cluster of CTAs per sequence.
//
// A draw compares running sums of up to 10^5 weights with a random number, so an error of e of
// the total gives another token with a chance of 10^5 e: 32-bit weights, whose errors of 2^-24
// add up to 10^-9 of the total or more, would miss one draw in some thousands.  The weights
// are therefore pairs of floats, exact to some 2^-30 of each while logits over temperatures stay below
// 10^5 (2^x by a table of 2^(k/32) and a short polynomial: Tang, "Table-driven implementation of the
// exponential function", ACM TOMS 1989), and their sums carry the rounding of every addition along
// (Knuth's two-sum); the first launch takes each weight apart at 2^-17 instead, adds the upper parts
// exactly and the rest, a hundredth at most, in 32 bits: a chunk's sum to 2^-32 (in the mean of random
// logits; 2^-29 the worst of 1800).  No sum is of 64-bit numbers: this GPU adds those at a fiftieth of the rate.
//
// 25 instructions a logit bound the first launch, not its read: 32 windows, 226 rows of 151,936
// fp32 logits in all (137 MB), 47 us, 60 % of the issue slots; 200 rows of 50,257 in bf16 16 us.  A warp
// takes one chunk and ends: looping with the next chunk's loads ahead took 88 registers for 80 and
// 65 us for 48, and loading a chunk again for its sum 75 to 77 us a call for 71.  The second launch is a
// chain of latencies: 10 us where a row of the target is drawn from, 28 where a cluster looks
// through the drafter's probabilities (eight CTAs of a sequence).  Both together 71, 20 and, one window
// of five rows, 10.8 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "mixing.h"
#include "sdv.h"
#include "sdv_device.cuh"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kStatChunk = 1024;   // logits of a warp's unit of work in the first launch
constexpr int kDrawChunk = 512;    // and of its pass in the second
constexpr int kStatThreads = 128;
constexpr int kDrawThreads = 256;
constexpr int kDrawWarps = kDrawThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kShares = kMaxCluster * kDrawWarps;  // warps of a sequence, at most
constexpr int kMaxDrafts = 31;

struct DraftArgs {
  const void* logits;
  long long stride;           // elements between rows
  const float* temperature;   // [B]
  const int32_t *drafts, *n_drafts;
  const float *probs, *uniforms;
  int32_t *accepted, *next;
  int B, S, V, chunks, draws;  // chunks of a row in the two launches
  int share;                   // chunks of a warp in the second
  float4* stats;              // [B * S][chunks]: maximum, sum in two floats (greedy: the bits of its place)
};

__device__ const float kPowHi[32] = {
    0x1.000000p+0f, 0x1.059b0ep+0f, 0x1.0b5586p+0f, 0x1.11301ep+0f, 0x1.172b84p+0f, 0x1.1d4874p+0f, 0x1.2387a6p+0f,
    0x1.29e9e0p+0f, 0x1.306fe0p+0f, 0x1.371a74p+0f, 0x1.3dea64p+0f, 0x1.44e086p+0f, 0x1.4bfdaep+0f, 0x1.5342b6p+0f,
    0x1.5ab07ep+0f, 0x1.6247ecp+0f, 0x1.6a09e6p+0f, 0x1.71f75ep+0f, 0x1.7a1148p+0f, 0x1.82589ap+0f, 0x1.8ace54p+0f,
    0x1.93737cp+0f, 0x1.9c4918p+0f, 0x1.a5503cp+0f, 0x1.ae89fap+0f, 0x1.b7f770p+0f, 0x1.c199bep+0f, 0x1.cb720ep+0f,
    0x1.d5818ep+0f, 0x1.dfc974p+0f, 0x1.ea4afap+0f, 0x1.f50766p+0f};
__device__ const float kPowLo[32] = {  // 2^(k/32) - kPowHi[k]
    0x0.000000p+0f,   -0x1.9d4f52p-25f, 0x1.9f3122p-25f,  -0x1.fdb496p-25f, -0x1.c15742p-27f, -0x1.d2e8cap-25f,
    0x1.ceac48p-25f,  -0x1.5c0424p-25f, 0x1.4636e2p-25f,  -0x1.18aac6p-25f, 0x1.824684p-25f,  0x1.8624b4p-30f,
    -0x1.593abcp-25f, -0x1.2c5610p-25f, -0x1.5bd5ecp-27f, -0x1.f8b550p-25f, 0x1.9fcef4p-26f,  0x1.1d8beep-25f,
    -0x1.829fd0p-25f, -0x1.accc7cp-26f, 0x1.15506ep-27f,  -0x1.e64744p-25f, 0x1.51f848p-27f,  -0x1.b83b54p-25f,
    -0x1.a94b14p-26f, -0x1.a09438p-25f, -0x1.3d56b2p-27f, -0x1.8837ccp-27f, -0x1.822dbcp-27f, -0x1.908c94p-25f,
    0x1.52486cp-27f,  -0x1.246eb0p-26f};

// A logit as it counts: NaN as one that is never drawn, +inf as the largest number.
__device__ __forceinline__ float counted_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <typename T>
__device__ __forceinline__ float logit(const T* p) {
  return counted_logit((float)*p);
}

__device__ __forceinline__ void group_floats(const uint4& x, float (&f)[4], float) {
  f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y), f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
}
template <typename T>
__device__ __forceinline__ void group_floats(const uint4& x, float (&f)[8], T) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = unpack16<T>(w[i]);
    f[2 * i] = y.x;
    f[2 * i + 1] = y.y;
  }
}

// Row r's logits in groups of 16 bytes from an aligned address on, the first `shift` elements of
// which lie before the row; a chunk is CHUNK elements of groups, 32 groups (one a lane) a step.
template <typename T, int CHUNK>
struct Row {
  static constexpr int kPer = 16 / sizeof(T);            // elements of a group
  static constexpr int kSteps = CHUNK / kPer / 32;       // groups of a lane in a chunk
  const T* p;
  int V, shift;
  __device__ __forceinline__ Row(const DraftArgs& a, long long row)
      : p(static_cast<const T*>(a.logits) + row * a.stride), V(a.V) {
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  }
  __device__ __forceinline__ int first(int chunk, int step, int lane) const {  // element of a group's start
    return (chunk * (CHUNK / kPer) + step * 32 + lane) * kPer - shift;
  }
  __device__ __forceinline__ bool whole(int v) const { return v >= 0 && v + kPer <= V; }
  __device__ __forceinline__ uint4 load(int v) const { return __ldg(reinterpret_cast<const uint4*>(p + v)); }
  // Element v + e as it counts; outside the row -inf.
  __device__ __forceinline__ float at(int v) const {
    return v >= 0 && v < V ? counted_logit((float)__ldg(p + v)) : -INFINITY;
  }
  __device__ __forceinline__ void load_chunk(int n, int lane, uint4 (&raw)[kSteps]) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int v = first(n, s, lane);
      if (whole(v)) raw[s] = load(v);
    }
  }
  // Elements of a loaded chunk's step as they lie; outside the row -inf.
  __device__ __forceinline__ void step(int n, int s, int lane, const uint4& raw, float (&x)[kPer]) const {
    const int v = first(n, s, lane);
    if (whole(v)) {
      group_floats(raw, x, T());
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] = at(v + e);
    }
  }
  __device__ __forceinline__ float largest(int n, int lane, const uint4 (&raw)[kSteps]) const {
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float x[kPer];
      step(n, s, lane, raw[s], x);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) m = max3(m, x[e], x[e + 1]);  // (of a number and NaN the number)
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return fminf(m, FLT_MAX);
  }
  // The lowest place of a chunk's maximum.
  __device__ __forceinline__ int place_of(int n, int lane, const uint4 (&raw)[kSteps], float m) const {
    int best = INT_MAX;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float x[kPer];
      step(n, s, lane, raw[s], x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = first(n, s, lane) + e;
        if (counted_logit(x[e]) == m && v >= 0 && v < V) best = min(best, v);
      }
    }
    return __reduce_min_sync(0xffffffffu, best);
  }
};

// log2(e) / T as a pair; greedy where T is 0, below, NaN, or so small that it overflows.
struct Warmth {
  float hi, lo;
  bool greedy;
  __device__ __forceinline__ explicit Warmth(float t) {
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0c0p-26f;  // log2(e)
    hi = kHi / t;
    lo = (fmaf(-hi, t, kHi) + kLo) / t;
    greedy = !(t > 0.f) || !(hi < INFINITY);
    if (!(hi >= 1e-37f)) {  // where the rest is no number any more; an infinite T: all equal, and 0 times -inf nowhere
      hi = fmaxf(hi, 1e-44f);
      lo = 0.f;
    }
  }
};

// ---- precise weights -------------------------------------------------------------------

struct Pair {  // two numbers, each the sum of two floats
  f32x2 hi, lo;
};
__device__ __forceinline__ f32x2 both(float x) { return pair2(x, x); }
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, both(-1.f), a); }  // (one instruction)
// s = fl(a + b) and what the rounding took.
__device__ __forceinline__ f32x2 two_sum(f32x2 a, f32x2 b, f32x2& err) {
  const f32x2 s = add2(a, b), t = sub2(s, a);
  err = add2(sub2(a, sub2(s, t)), sub2(b, t));
  return s;
}

// One number as the sum of two floats, the second far below the first.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add_two(Two a, Two b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  return Two{s, __fadd_rn(err, __fadd_rn(a.lo, b.lo))};
}
__device__ __forceinline__ Two shfl_up(Two a, int off) {
  return Two{__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
}
__device__ __forceinline__ Two shfl_at(Two a, int lane) {
  return Two{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
__device__ __forceinline__ bool exceeds(Two a, Two b) {
  return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) > 0.f;
}
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    x = add_two(x, Two{__shfl_xor_sync(0xffffffffu, x.hi, off), __shfl_xor_sync(0xffffffffu, x.lo, off)});
  return x;
}
// The sum up to and with this lane's.
__device__ __forceinline__ Two warp_scan(Two x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Two o = shfl_up(x, off);
    if (lane >= off) x = add_two(o, x);
  }
  return x;
}

// 2^(x c - K) for the two x of a pair, K = ceil(m c) for the largest x: exact to some 2^-30 of
// each, or to 2^-48 |x c|, that of x c itself, where this is more; 0 where it is below 2^-124 and where x is -inf.  For all lanes of a warp: lane k holds
// 2^(k/32).  x c is taken apart as it is, K being a whole number; where it is so large that its
// last bits are no fraction any more, K is taken off first (exact: the two are close).  Past 2^24,
// where neighbouring logits are a power of two and more apart, K is m c itself.
struct Weigher {
  float M, c_hi, c_lo, pow_hi, pow_lo, least, K, K_lo;
  uint32_t bias;
  bool off, far;
  __device__ __forceinline__ Weigher(float m, const Warmth& c, int lane)
      : M(m), c_hi(c.hi), c_lo(c.lo), pow_hi(kPowHi[lane]), pow_lo(kPowLo[lane]) {
    least = fmaxf(m - 124.f / c.hi, -FLT_MAX);
    K = ceilf(m * c.hi);
    K_lo = 0.f;
    if (!(fabsf(K) < 0x1p100f)) {  // nothing but the largest has a weight, nor has it at this c
      c_hi = 0x1p40f / fabsf(m);
      c_lo = 0.f;
      K = ceilf(m * c_hi);
      least = fmaxf(m - 124.f / c_hi, -FLT_MAX);
    }
    off = fabsf(K) >= 65536.f;
    far = fabsf(K) >= 16777216.f;
    if (far) K_lo = fmaf(m, c_lo, fmaf(m, c_hi, -K));
    bias = ((uint32_t)(127 - (off ? 0 : (int)K)) << 23) - (0x4b400000u << 18);
  }
  // The weight of a sum that is relative to the K of its own largest x, mk.
  __device__ __forceinline__ float of_chunk(float mk) const {
    if (!(mk >= least)) return 0.f;
    if (far) {
      const float d = mk - M, t = d * c_hi, tl = fmaf(d, c_lo, fmaf(d, c_hi, -t));
      return exp2f(t) * fmaf(tl, 0.6931472f, 1.f);
    }
    return __uint_as_float((uint32_t)(127 + (int)(ceilf(mk * c_hi) - K)) << 23);
  }
  // What 2^(x c - K) of two finite x is made of: (th + tlo) (1 + s) times a power of two.
  struct Made {
    f32x2 th, tlo, s;
    float scale0, scale1;
  };
  __device__ __forceinline__ Made made(float x0, float x1) const {
    const f32x2 x = pair2(x0, x1);
    f32x2 t = mul2(x, both(-c_hi));  // - x c
    f32x2 tl = fma2(x, both(c_lo), fma2(x, both(c_hi), t));
    if (off) {
      f32x2 err;
      t = two_sum(add2(t, both(K)), sub2(both(K_lo), tl), err);
      tl = sub2(both(0.f), err);
    }
    // x c = k / 32 - r, |r| <= 1 / 64: k in the low bits of a number of 1.5 2^23
    const f32x2 magic = both(12582912.f), kk = fma2(t, both(-32.f), magic);
    const f32x2 r = fma2(sub2(kk, magic), both(0.03125f), t);
    const float2 kf = unpair2(kk);
    const uint32_t k0 = __float_as_uint(kf.x), k1 = __float_as_uint(kf.y);
    Made w;
    w.th = pair2(__shfl_sync(0xffffffffu, pow_hi, k0), __shfl_sync(0xffffffffu, pow_hi, k1));
    w.tlo = pair2(__shfl_sync(0xffffffffu, pow_lo, k0), __shfl_sync(0xffffffffu, pow_lo, k1));
    // 2^-r = 1 + s, |s| < 0.011
    f32x2 p = fma2(r, both(0.009618129f), both(-0.05550411f));
    p = fma2(r, p, both(0.24022651f));
    p = fma2(r, p, both(-0x1.62e430p-1f));
    w.s = fma2(r, p, fma2(tl, both(0x1.62e430p-1f), mul2(r, both(0x1.05c610p-29f))));
    w.scale0 = __uint_as_float(((k0 & ~31u) << 18) + bias);
    w.scale1 = __uint_as_float(((k1 & ~31u) << 18) + bias);
    return w;
  }
  // Two weights; 0 for an x that does not count.
  __device__ __forceinline__ Pair operator()(float x0, float x1) const {
    // (NaN and -inf become the least)
    const Made w = made(fminf(fmaxf(x0, least), M), fminf(fmaxf(x1, least), M));
    const f32x2 scale = pair2(x0 >= least ? w.scale0 : 0.f, x1 >= least ? w.scale1 : 0.f);
    return Pair{mul2(w.th, scale), mul2(fma2(w.th, w.s, w.tlo), scale)};
  }
  // Whether `add` may be used: an x that does not count then adds some 2^-124, which a sum whose
  // largest weight is 1/2 or more does not notice.
  __device__ __forceinline__ bool plain() const { return least > -FLT_MAX && !far && M < FLT_MAX; }
  // Two weights of up to 1 to a sum of up to 64 of them: to sum.hi (its negative) what of them is a
  // multiple of 2^-17, exactly, and to sum.lo the rest.
  __device__ __forceinline__ void add(Pair& sum, float x0, float x1) const {
    const Made w = made(fmaxf(x0, least), fmaxf(x1, least));
    const f32x2 scale = pair2(w.scale0, w.scale1), grid = both(96.f);  // 1.5 2^6: the last place is 2^-17
    const f32x2 down = sub2(grid, fma2(w.th, scale, grid));
    sum.hi = add2(sum.hi, down);
    sum.lo = add2(sum.lo, fma2(fma2(w.th, w.s, w.tlo), scale, fma2(w.th, scale, down)));
  }
};

__device__ __forceinline__ void add_pair(Pair& sum, const Pair& w) {
  f32x2 err;
  sum.hi = two_sum(sum.hi, w.hi, err);
  sum.lo = add2(sum.lo, add2(err, w.lo));
}
__device__ __forceinline__ Two lanes_sum(const Pair& sum) {
  const float2 h = unpair2(sum.hi), l = unpair2(sum.lo);
  return warp_sum(add_two(Two{h.x, l.x}, Two{h.y, l.y}));
}

template <typename T>
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(const DraftArgs a) {
  using R = Row<T, kStatChunk>;
  constexpr int W = kStatThreads / 32;
  const int lane = threadIdx.x & 31, blocks = (a.chunks + W - 1) / W;
  const int row = blockIdx.x / blocks;
  const int chunk = (blockIdx.x - row * blocks) * W + (threadIdx.x >> 5);
  const int b = row / a.S, i = row - b * a.S;
  griddep_wait();
  griddep_launch_dependents();
  const int n = a.n_drafts != nullptr ? min(max(__ldg(a.n_drafts + b), 0), a.S - 1) : a.S - 1;
  if (chunk >= a.chunks || i > n) return;
  const R r(a, row);
  const float t = __ldg(a.temperature + b);
  uint4 raw[R::kSteps];
  r.load_chunk(chunk, lane, raw);
  const float m = r.largest(chunk, lane, raw);
  const Warmth c(t);
  float4 out = make_float4(m, 0.f, 0.f, 0.f);
  if (c.greedy) {
    out.y = __int_as_float(r.place_of(chunk, lane, raw, m));
  } else if (m != -INFINITY) {
    const Weigher weigh(m, c, lane);
    Pair sum{0, 0};
    if (weigh.plain()) {
#pragma unroll
      for (int s = 0; s < R::kSteps; ++s) {
        float x[R::kPer];
        r.step(chunk, s, lane, raw[s], x);
#pragma unroll
        for (int e = 0; e < R::kPer; e += 2) weigh.add(sum, x[e], x[e + 1]);
      }
      sum.hi = sub2(both(0.f), sum.hi);
    } else {
#pragma unroll 1
      for (int s = 0; s < R::kSteps; ++s) {
        float x[R::kPer];
#pragma unroll
        for (int e = 0; e < R::kPer; ++e) x[e] = r.at(r.first(chunk, s, lane) + e);
#pragma unroll
        for (int e = 0; e < R::kPer; e += 2) add_pair(sum, weigh(x[e], x[e + 1]));
      }
    }
    const Two all = lanes_sum(sum);
    out.y = all.hi;
    out.z = all.lo;
  }
  if (lane == 0) a.stats[(long long)row * a.chunks + chunk] = out;
}

// What max(w - q Z, 0) leaves, Z = z.hi + z.lo.
__device__ __forceinline__ Pair rest_of(const Pair& w, float q0, float q1, Two z) {
  const f32x2 q = pair2(q0 > 0.f ? q0 : 0.f, q1 > 0.f ? q1 : 0.f);
  const f32x2 a = mul2(q, both(-z.hi));  // - q Z
  const f32x2 al = fma2(q, both(z.lo), fma2(q, both(z.hi), a));
  f32x2 err;
  const f32x2 d = two_sum(w.hi, a, err);
  const f32x2 l = add2(err, sub2(w.lo, al));
  const float2 sum = unpair2(add2(d, l)), dh = unpair2(d), dl = unpair2(l);
  return Pair{pair2(sum.x > 0.f ? dh.x : 0.f, sum.y > 0.f ? dh.y : 0.f),
              pair2(sum.x > 0.f ? dl.x : 0.f, sum.y > 0.f ? dl.y : 0.f)};
}

// To a lane's sum what q leaves of the weights of its part of a chunk.
template <typename R>
__device__ __forceinline__ void add_rest(Pair& sum, const R& r, const Weigher& weigh, int n, int lane, const float* q,
                                         Two z) {
  uint4 raw[R::kSteps];
  r.load_chunk(n, lane, raw);
#pragma unroll
  for (int s = 0; s < R::kSteps; ++s) {
    const int v = r.first(n, s, lane);
    float x[R::kPer], qs[R::kPer];
    if (r.whole(v) && (reinterpret_cast<uintptr_t>(q + v) & 15u) == 0) {
#pragma unroll
      for (int e = 0; e < R::kPer; e += 4) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(q + v + e));
        qs[e] = y.x, qs[e + 1] = y.y, qs[e + 2] = y.z, qs[e + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) qs[e] = v + e >= 0 && v + e < r.V ? __ldg(q + v + e) : 0.f;
    }
    r.step(n, s, lane, raw[s], x);
#pragma unroll
    for (int e = 0; e < R::kPer; e += 2) add_pair(sum, rest_of(weigh(x[e], x[e + 1]), qs[e], qs[e + 1], z));
  }
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive();
  cluster_wait();
}

// Writes y to place `at` of the same list in every CTA of the cluster, a lane each.
__device__ __forceinline__ void tell(float2* list, int at, float2 y, int lane, int size) {
  if (lane >= size) return;
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(list + at)), "r"(lane));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(y.x), "f"(y.y) : "memory");
}

// A list of sums, by one warp, a lane a stretch of it in order; `entry(i)` gives one.  The first
// kHeld of each lane are read once.
template <typename F>
struct Listed {
  static constexpr int kHeld = 5;
  F entry;
  int n, lane, from, to;
  Two held[kHeld], upto;  // and all up to the end of this lane's
  __device__ __forceinline__ Listed(int count, int l, F f) : entry(f), n(count), lane(l) {
    const int per = (n + 31) / 32;
    from = min(lane * per, n);
    to = min(from + per, n);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = from + i < to ? entry(from + i) : Two{0.f, 0.f};
    Two mine = held[0];
#pragma unroll
    for (int i = 1; i < kHeld; ++i) mine = add_two(mine, held[i]);
#pragma unroll 4
    for (int i = from + kHeld; i < to; ++i) mine = add_two(mine, entry(i));
    upto = warp_scan(mine, lane);
  }
  __device__ __forceinline__ Two total() const { return shfl_at(upto, 31); }
  // The entry in which the running sum first exceeds `want`, and the sum in front of it; the last
  // entry with any weight and no bound where none does.
  __device__ __forceinline__ int find(Two& want, Two& before) const {
    const Two up = shfl_up(upto, 1);
    Two run = lane > 0 ? up : Two{0.f, 0.f};
    int hit = INT_MAX, last = -1;
    before = run;
    auto look = [&](int i, Two x) {
      const Two next = add_two(run, x);
      if (x.hi > 0.f) {
        last = i;
        if (hit == INT_MAX && exceeds(next, want)) {
          hit = i;
          before = run;
        }
      }
      run = next;
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) look(from + i, held[i]);
#pragma unroll 4
    for (int i = from + kHeld; i < to; ++i) look(i, entry(i));
    const int at = __reduce_min_sync(0xffffffffu, hit);
    if (at != INT_MAX) {
      before = shfl_at(before, __ffs(__ballot_sync(0xffffffffu, hit == at)) - 1);
      return at;
    }
    want = Two{INFINITY, 0.f};
    return __reduce_max_sync(0xffffffffu, last);
  }
};
template <typename F>
__device__ __forceinline__ Listed<F> listed(int n, int lane, F f) {
  return Listed<F>(n, lane, f);
}

template <typename T>
__global__ void __launch_bounds__(kDrawThreads, 3) verify_draw_kernel(const DraftArgs a) {
  using R = Row<T, kDrawChunk>;
  constexpr int W = kDrawWarps;
  __shared__ float2 s_rests[kShares];
  __shared__ float s_max[kMaxDrafts + 1];
  __shared__ Two s_total[kMaxDrafts + 1], s_part[W], s_want, s_before;
  __shared__ int s_best[kMaxDrafts + 1], s_token, s_last, s_at;
  __shared__ bool s_ok[kMaxDrafts + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = cluster_size(), rank = cluster_rank(), b = blockIdx.x / size;
  if (tid == 0) {
    s_token = INT_MAX;
    s_last = -1;
  }
  cluster_arrive();
  // Logits, drafts and counts may be what launches in front of this call have written: like the sums,
  // they are only sure to be seen behind the wait.
  griddep_wait();
  const float t = __ldg(a.temperature + b);
  const int n = a.n_drafts != nullptr ? min(max(__ldg(a.n_drafts + b), 0), a.S - 1) : a.S - 1;
  const float u = __ldg(a.uniforms + (long long)b * a.S + a.S - 1);
  struct Test {
    bool real;
    float x, q, u;  // the draft's logit and probability, its random number
  };
  auto test_of = [&](int i) {
    const long long row = (long long)b * a.S + i;
    const int d = i < a.S - 1 ? __ldg(a.drafts + (long long)b * (a.S - 1) + i) : -1;  // (not behind the load of n)
    Test v;
    v.real = i < n && d >= 0 && d < a.V;
    v.u = __ldg(a.uniforms + row);
    v.x = v.real ? logit(static_cast<const T*>(a.logits) + row * a.stride + d) : -INFINITY;
    v.q = a.probs != nullptr && v.real ? __ldg(a.probs + ((long long)b * (a.S - 1) + i) * a.V + d) : 1.f;
    v.q = v.q > 0.f ? v.q : 0.f;
    return v;
  };
  Test test{};
  if (warp < a.S) test = test_of(warp);
  const Warmth c(t);
  cluster_wait();  // every CTA has begun: its shared memory can be written
  // every row's sum, and its draft's test
  for (int i = warp; i <= n; i += W) {
    const long long row = (long long)b * a.S + i;
    const float4* const st = a.stats + row * a.chunks;
    constexpr int kHeld = 5;  // entries of a lane that are read once
    float4 e[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      e[k] = lane + 32 * k < a.chunks ? __ldcg(st + lane + 32 * k) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (i != warp) test = test_of(i);
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) m = fmaxf(m, e[k].x);
#pragma unroll 4
    for (int k = lane + 32 * kHeld; k < a.chunks; k += 32) m = fmaxf(m, __ldcg(&st[k].x));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    Two z{0.f, 0.f};
    float p = 0.f;
    int best = INT_MAX;
    if (c.greedy) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (e[k].x == m && lane + 32 * k < a.chunks) best = min(best, __float_as_int(e[k].y));
      for (int k = lane + 32 * kHeld; k < a.chunks; k += 32) {
        const float4 s = __ldcg(st + k);
        if (s.x == m) best = min(best, __float_as_int(s.y));
      }
      best = __reduce_min_sync(0xffffffffu, best);
      z.hi = 1.f;
      if (m == -INFINITY) best = INT_MAX;
      p = test.real && test.x == m && m != -INFINITY && __ldg(a.drafts + (long long)b * (a.S - 1) + i) == best ? 1.f : 0.f;
    } else if (m != -INFINITY) {
      const Weigher weigh(m, c, lane);
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const float f = weigh.of_chunk(e[k].x);
        z = add_two(z, Two{e[k].y * f, e[k].z * f});
      }
#pragma unroll 4
      for (int k = lane + 32 * kHeld; k < a.chunks; k += 32) {
        const float4 s = __ldcg(st + k);
        const float f = weigh.of_chunk(s.x);
        z = add_two(z, Two{s.y * f, s.z * f});
      }
      z = warp_sum(z);
      const Pair w = weigh(test.x, test.x);
      p = unpair2(add2(w.hi, w.lo)).x;
    }
    if (lane == 0) {
      s_ok[i] = i < n && test.real && test.u * test.q * z.hi < p;
      s_max[i] = m;
      s_best[i] = best;
      s_total[i] = z;
    }
  }
  __syncthreads();
  int j = 0;
  while (j < n && s_ok[j]) ++j;
  const bool missed = j < n;
  const float m = s_max[j];
  if (rank == 0 && tid == 0) a.accepted[b] = j;
  if (c.greedy || m == -INFINITY) {  // the same in the whole cluster
    // what a drafter's probabilities leave of a single token is that token
    if (rank == 0 && tid == 0) a.next[b] = m == -INFINITY ? -1 : s_best[j];
    return;
  }
  const R r(a, (long long)b * a.S + j);
  const Weigher weigh(m, c, lane);
  const bool rest = missed && a.probs != nullptr;
  const int d = missed ? __ldg(a.drafts + (long long)b * (a.S - 1) + j) : -1;
  const int gone = !rest && d >= 0 && d < a.V ? d : INT_MIN;  // the token that is not drawn
  const float* const q = rest ? a.probs + ((long long)b * (a.S - 1) + j) * a.V : nullptr;
  const Two z = s_total[j];
  auto bound = [&](Two all) {
    const float p = __fmul_rn(u, all.hi);
    return Two{p, fmaf(u, all.lo, fmaf(u, all.hi, -p))};
  };
  bool left = false;    // whether the drafter's probabilities leave anything
  int at, from, each;   // the entry of the list that the draw falls into; its first element, elements per thread
  Two want, run;
  if (rest) {
    const int share = rank * W + warp, k1 = min((share + 1) * a.share, a.draws);
    Pair sum{0, 0};
    for (int k = share * a.share; k < k1; ++k) add_rest(sum, r, weigh, k, lane, q, z);
    const Two s = lanes_sum(sum);
    tell(s_rests, share, make_float2(s.hi, s.lo), lane, size);
    cluster_meet();
    const auto list = listed(size * W, lane, [&](int i) { return Two{s_rests[i].x, s_rests[i].y}; });
    const Two all = list.total();
    left = all.hi > 0.f;
    if (left) {
      want = bound(all);
      at = list.find(want, run);
      if (at / W != rank) return;
      from = at * a.share * kDrawChunk - r.shift;
      each = kDrawChunk / kDrawThreads * a.share;
    }
  }
  auto pair_at = [&](int v) {
    Pair w = weigh(v == gone ? -INFINITY : r.at(v), v + 1 == gone ? -INFINITY : r.at(v + 1));
    if (left)
      w = rest_of(w, v >= 0 && v < a.V ? __ldg(q + v) : 0.f, v + 1 >= 0 && v + 1 < a.V ? __ldg(q + v + 1) : 0.f, z);
    return w;
  };
  // The sum of a thread's stretch of elements, in order, and of all threads' in front of it.
  auto stretch = [&](Two& before) {
    Two mine{0.f, 0.f};
    for (int e = 0; e < each; e += 2) {
      const Pair w = pair_at(from + each * tid + e);
      const float2 h = unpair2(w.hi), l = unpair2(w.lo);
      mine = add_two(mine, add_two(Two{h.x, l.x}, Two{h.y, l.y}));
    }
    const Two incl = warp_scan(mine, lane);
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    Two all{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (k == warp) before = all;
      all = add_two(all, s_part[k]);
    }
    const Two up = shfl_up(incl, 1);
    if (lane > 0) before = add_two(before, up);
    return all;
  };
  if (!left) {  // from the row itself, by the first launch's sums
    if (rank != 0) return;
    const int gone_chunk = gone >= 0 ? (gone + r.shift) / kStatChunk : -1;
    each = kStatChunk / kDrawThreads;
    Two without{0.f, 0.f}, front;
    if (gone_chunk >= 0) {  // that chunk's sum without the token
      from = gone_chunk * kStatChunk - r.shift;
      without = stretch(front);
    }
    if (warp == 0) {
      const float4* const st = a.stats + ((long long)b * a.S + j) * a.chunks;
      const auto list = listed(a.chunks, lane, [&](int i) {
        if (i == gone_chunk) return without;
        const float4 s = __ldcg(st + i);
        const float f = weigh.of_chunk(s.x);
        return Two{s.y * f, s.z * f};
      });
      want = bound(list.total());
      at = list.find(want, run);
      if (lane == 0) {
        s_at = at;
        s_want = want;
        s_before = run;
      }
    }
    __syncthreads();
    at = s_at;
    want = s_want;
    run = s_before;
    if (at < 0) {  // all weight was the draft's that was not kept
      if (tid == 0) a.next[b] = gone;
      return;
    }
    from = at * kStatChunk - r.shift;
  }
  Two front;
  stretch(front);
  run = add_two(run, front);
  int token = INT_MAX, last = -1;
  for (int e = 0; e < each; e += 2) {
    const int v = from + each * tid + e;
    const Pair w = pair_at(v);
    const float2 h = unpair2(w.hi), l = unpair2(w.lo);
    run = add_two(run, Two{h.x, l.x});
    if (h.x > 0.f) {
      last = v;
      if (exceeds(run, want)) token = min(token, v);
    }
    run = add_two(run, Two{h.y, l.y});
    if (h.y > 0.f) {
      last = v + 1;
      if (exceeds(run, want)) token = min(token, v + 1);
    }
  }
  token = __reduce_min_sync(0xffffffffu, token);
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane == 0) {
    if (token != INT_MAX) atomicMin(&s_token, token);
    if (last >= 0) atomicMax(&s_last, last);
  }
  __syncthreads();
  if (tid == 0) a.next[b] = s_token != INT_MAX ? s_token : s_last;
}

int chunks_of(int V, int chunk) { return (int)(((long long)V + 7 + chunk - 1) / chunk); }

size_t drafts_need(int B, int S, int V) {
  if (B < 1 || S < 1 || S > kMaxDrafts + 1 || V < 1 || V > (1 << 24) || B > (1 << 24)) return 0;
  if ((unsigned long long)B * S * ((chunks_of(V, kStatChunk) + 3) / 4) > INT_MAX) return 0;
  return kHeaderBytes + round_256((size_t)B * S * chunks_of(V, kStatChunk) * 16);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T>
cudaError_t drafts_launch(DraftArgs a, int sms, cudaStream_t st) {
  constexpr int W = kStatThreads / 32;
  const unsigned grid = (unsigned)((long long)a.B * a.S * ((a.chunks + W - 1) / W));
  const cudaError_t e = launch_pdl(verify_stats_kernel<T>, dim3(grid), dim3(kStatThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  // CTAs of a sequence: one, or where there are drafter's probabilities to look at eight at most,
  // a chunk for every warp, and not more than run at once
  int cluster = 1;
  while (a.probs != nullptr && cluster < kMaxCluster && cluster * kDrawWarps < a.draws &&
         2ll * cluster * a.B <= 3ll * sms)
    cluster *= 2;
  a.share = (a.draws + cluster * kDrawWarps - 1) / (cluster * kDrawWarps);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster * a.B);
  cfg.blockDim = dim3(kDrawThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return counted(cudaLaunchKernelEx(&cfg, verify_draw_kernel<T>, a));
}

}  // namespace

}  // namespace sdv

extern "C" {

size_t sdv_verify_drafts_workspace_bytes(int32_t B, int32_t S, int32_t V) { return sdv::drafts_need(B, S, V); }

sdv_status sdv_verify_drafts(int32_t dtype, const void* logits, int64_t row_stride, int32_t B, int32_t S, int32_t V,
                             const float* temperature, const int32_t* drafts_or_null,
                             const int32_t* n_drafts_or_null, const float* draft_probs_or_null,
                             const float* uniforms, int32_t* accepted, int32_t* next_token, void* ws, size_t ws_bytes,
                             sdv_stream_t stream) {
  if (dtype != SDV_F16 && dtype != SDV_BF16 && dtype != SDV_F32) return SDV_ERR_INVALID_ARG;
  const uintptr_t odd = reinterpret_cast<uintptr_t>(logits) & (dtype == SDV_F32 ? 3u : 1u);
  if (logits == nullptr || odd != 0 || B < 1 || S < 1 || V < 1 || row_stride < V) return SDV_ERR_INVALID_ARG;
  if (temperature == nullptr || uniforms == nullptr || accepted == nullptr || next_token == nullptr ||
      (S > 1 && drafts_or_null == nullptr))
    return SDV_ERR_INVALID_ARG;
  for (const void* p : {(const void*)temperature, (const void*)drafts_or_null, (const void*)n_drafts_or_null,
                        (const void*)draft_probs_or_null, (const void*)uniforms, (const void*)accepted,
                        (const void*)next_token})
    if (!sdv::aligned4(p)) return SDV_ERR_INVALID_ARG;
  const size_t need = sdv::drafts_need(B, S, V);
  if (need == 0) return SDV_ERR_UNSUPPORTED;
  if (ws == nullptr || !sdv::is_aligned16(ws) || ws_bytes < need) return SDV_ERR_WORKSPACE;
  sdv::DraftArgs a{};
  a.logits = logits;
  a.stride = row_stride;
  a.temperature = temperature;
  a.drafts = drafts_or_null;
  a.n_drafts = n_drafts_or_null;
  a.probs = S > 1 ? draft_probs_or_null : nullptr;
  a.uniforms = uniforms;
  a.accepted = accepted;
  a.next = next_token;
  a.B = B;
  a.S = S;
  a.V = V;
  a.chunks = sdv::chunks_of(V, sdv::kStatChunk);
  a.draws = sdv::chunks_of(V, sdv::kDrawChunk);
  a.stats = reinterpret_cast<float4*>(static_cast<char*>(ws) + sdv::kHeaderBytes);
  const int sms = sdv::sm_count();
  if (sms <= 0) return SDV_ERR_CUDA;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return sdv::status_of(dtype == SDV_F32   ? sdv::drafts_launch<float>(a, sms, st)
                        : dtype == SDV_F16 ? sdv::drafts_launch<__half>(a, sms, st)
                                           : sdv::drafts_launch<__nv_bfloat16>(a, sms, st));
}

}  // extern "C"

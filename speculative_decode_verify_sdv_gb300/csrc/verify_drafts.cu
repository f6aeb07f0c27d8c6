// Verification of drafted tokens against the target's probabilities, and the draw of the next
// token, from given random numbers (sdv_verify_drafts).
//
//   p_i = softmax(logits_i / T);  draft d_i is kept while u_i q_i(d_i) < p_i(d_i);  at the first
//   one that is not, the next token is drawn from max(p_i - q_i, 0), else from p_n:
//   the lowest v whose running weight exceeds u_S-1 of the total.
//
// Two launches.  The first reads every row once: per chunk of 2048 logits the maximum m and
// sum 2^((x - m) c), c = log2(e) / T (or, greedy, the place of the maximum).  Reading the logits
// bounds it.  The second has a cluster per sequence: it joins the rows' sums, runs the tests and
// draws from the one row left.  Without drafts the second does it all.
//
// A draw compares running sums of up to 10^5 weights with a random number, so an error of e of
// the total gives another token with a chance of 10^5 e: 32-bit weights, whose errors of 2^-24
// add up to 10^-9 of the total or more, would miss one draw in some thousands.  The row's weights
// are therefore pairs of floats, exact to some 2^-30 of each (2^x by a table of 2^(k/32) and a
// short polynomial: Tang, "Table-driven implementation of the exponential function", ACM TOMS
// 1989), and their sums carry the rounding of every addition along (Knuth's two-sum).  No sum is
// of 64-bit numbers: this GPU adds those at a fiftieth of the rate.
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

constexpr int kStatChunk = 2048;   // logits of a warp's unit of work in the first launch
constexpr int kDrawChunk = 1024;   // and in the second: two for each thread of a CTA
constexpr int kStatThreads = 128;
constexpr int kDrawThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kMaxDrafts = 31;

struct DraftArgs {
  const void* logits;
  long long stride;           // elements between rows
  const float* temperature;   // [B]
  const int32_t *drafts, *n_drafts;
  const float *probs, *uniforms;
  int32_t *accepted, *next;
  int B, S, V, chunks, draws;  // chunks of a row in the two launches
  float2* stats;              // [B * S][chunks] (no drafts: [B][draws]): maximum, sum (greedy: the bits of its place)
  float2 *sums, *rests;       // [B][draws]: the drawn row's weights, and what the drafter's leave of them
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

template <typename T>
__device__ __forceinline__ float logit(const T* p) {
  return counted_logit((float)*p);
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
  // A chunk's elements as they count, of this lane; their maximum over the warp.
  __device__ __forceinline__ float chunk(int n, int lane, float (&x)[kSteps][kPer]) const;
};

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

template <typename T, int CHUNK>
__device__ __forceinline__ float Row<T, CHUNK>::chunk(int n, int lane, float (&x)[kSteps][kPer]) const {
  uint4 raw[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int v = first(n, s, lane);
    if (whole(v)) raw[s] = load(v);
  }
  float m = -INFINITY;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int v = first(n, s, lane);
    if (whole(v)) {
      group_floats(raw[s], x[s], T());
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[s][e] = counted_logit(x[s][e]);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[s][e] = at(v + e);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) m = fmaxf(m, x[s][e]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// The lowest place of a chunk's maximum.
template <typename R>
__device__ __forceinline__ int place_of(const R& r, int n, int lane, const float (&x)[R::kSteps][R::kPer], float m) {
  int best = INT_MAX;
#pragma unroll
  for (int s = 0; s < R::kSteps; ++s)
#pragma unroll
    for (int e = 0; e < R::kPer; ++e) {
      const int v = r.first(n, s, lane) + e;
      if (x[s][e] == m && v >= 0 && v < r.V) best = min(best, v);
    }
  return __reduce_min_sync(0xffffffffu, best);
}

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
  float x[R::kSteps][R::kPer];
  const float m = r.chunk(chunk, lane, x);
  const Warmth c(t);
  float2 out = make_float2(m, 0.f);
  if (c.greedy) {
    out.y = __int_as_float(place_of(r, chunk, lane, x, m));
  } else if (m != -INFINITY) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < R::kSteps; ++s)
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) sum[e & 3] += exp2_approx((x[s][e] - m) * c.hi);
    float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    out.y = all;
  }
  if (lane == 0) a.stats[(long long)row * a.chunks + chunk] = out;
}

// ---- precise weights -------------------------------------------------------------------

struct Pair {  // two numbers, each the sum of two floats
  f32x2 hi, lo;
};
__device__ __forceinline__ f32x2 neg2(f32x2 a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return add2(a, neg2(b)); }
__device__ __forceinline__ f32x2 both(float x) { return pair2(x, x); }
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

// 2^(x c - K) for the two x of a pair, K the exponent of the row's largest weight: exact to some
// 2^-30 of each; 0 where it is below 2^-124 and where x is -inf.  For all lanes of a warp: lane k
// holds 2^(k/32).  x c is taken apart as it is, K being a whole number; where it is so large that
// its last bits are no fraction any more, the row's maximum is taken off x first.
struct Weigher {
  float M, c_hi, c_lo, pow_hi, pow_lo, least;
  uint32_t bias;
  bool off;
  __device__ __forceinline__ Weigher(float m, const Warmth& c, int lane)
      : M(m), c_hi(c.hi), c_lo(c.lo), pow_hi(kPowHi[lane]), pow_lo(kPowLo[lane]) {
    least = fmaxf(m - 124.f / c.hi, -FLT_MAX);
    off = fabsf(m) * c.hi >= 16384.f;
    const int K = off ? 0 : (int)ceilf(m * c.hi);
    bias = ((uint32_t)(127 - K) << 23) - ((0x4b400000u >> 5) << 23);
  }
  __device__ __forceinline__ Pair operator()(float x0, float x1) const {
    const bool in0 = x0 >= least, in1 = x1 >= least;
    f32x2 x = pair2(in0 ? x0 : M, in1 ? x1 : M), x_lo = 0;
    if (off) x = two_sum(x, both(-M), x_lo);
    const f32x2 ch = both(c_hi), t = mul2(x, ch);
    f32x2 tl = fma2(x, both(c_lo), fma2(x, ch, neg2(t)));
    if (off) tl = fma2(x_lo, ch, tl);
    // t = k / 32 + r, |r| <= 1 / 64: k in the low bits of a number of 1.5 2^23
    const f32x2 magic = both(12582912.f), kk = fma2(t, both(32.f), magic);
    const f32x2 r = fma2(sub2(kk, magic), both(-0.03125f), t);
    const float2 kf = unpair2(kk);
    const uint32_t k0 = __float_as_uint(kf.x), k1 = __float_as_uint(kf.y);
    const f32x2 th = pair2(__shfl_sync(0xffffffffu, pow_hi, k0), __shfl_sync(0xffffffffu, pow_hi, k1));
    const f32x2 tlo = pair2(__shfl_sync(0xffffffffu, pow_lo, k0), __shfl_sync(0xffffffffu, pow_lo, k1));
    // 2^r = 1 + s, |s| < 0.011
    f32x2 p = fma2(r, both(0.009618129f), both(0.05550411f));
    p = fma2(r, p, both(0.24022651f));
    p = fma2(r, p, both(0x1.62e430p-1f));
    f32x2 s = fma2(tl, both(0x1.62e430p-1f), mul2(r, both(-0x1.05c610p-29f)));
    s = fma2(r, p, s);
    const f32x2 scale = pair2(in0 ? __uint_as_float(((k0 >> 5) << 23) + bias) : 0.f,
                              in1 ? __uint_as_float(((k1 >> 5) << 23) + bias) : 0.f);
    return Pair{mul2(th, scale), mul2(fma2(th, s, tlo), scale)};
  }
};

// What max(w - q Z, 0) leaves, Z = z.hi + z.lo.
__device__ __forceinline__ Pair rest_of(const Pair& w, float q0, float q1, Two z) {
  const f32x2 q = pair2(q0 > 0.f ? q0 : 0.f, q1 > 0.f ? q1 : 0.f);
  const f32x2 a = mul2(q, both(z.hi));
  const f32x2 al = fma2(q, both(z.lo), fma2(q, both(z.hi), neg2(a)));
  f32x2 err;
  const f32x2 d = two_sum(w.hi, neg2(a), err);
  const f32x2 l = add2(err, sub2(w.lo, al));
  const float2 sum = unpair2(add2(d, l)), dh = unpair2(d), dl = unpair2(l);
  return Pair{pair2(sum.x > 0.f ? dh.x : 0.f, sum.y > 0.f ? dh.y : 0.f),
              pair2(sum.x > 0.f ? dl.x : 0.f, sum.y > 0.f ? dl.y : 0.f)};
}

// A chunk's weights added up: of the row, without token `gone`, or (q given) what q leaves.
template <typename R>
__device__ __forceinline__ Two chunk_sum(const R& r, const Weigher& weigh, int n, int lane,
                                         float (&x)[R::kSteps][R::kPer], int gone, const float* q, Two z) {
  Pair sum{0, 0};
#pragma unroll
  for (int s = 0; s < R::kSteps; ++s) {
    const int v = r.first(n, s, lane);
    float qs[R::kPer];
    if (q != nullptr) {
      if (r.whole(v) && (reinterpret_cast<uintptr_t>(q + v) & 15u) == 0) {
#pragma unroll
        for (int e = 0; e < R::kPer; e += 4)
          *reinterpret_cast<float4*>(qs + e) = __ldg(reinterpret_cast<const float4*>(q + v + e));
      } else {
#pragma unroll
        for (int e = 0; e < R::kPer; ++e) qs[e] = v + e >= 0 && v + e < r.V ? __ldg(q + v + e) : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < R::kPer; e += 2) {
      if (v + e == gone) x[s][e] = -INFINITY;
      if (v + e + 1 == gone) x[s][e + 1] = -INFINITY;
      Pair w = weigh(x[s][e], x[s][e + 1]);
      if (q != nullptr) w = rest_of(w, qs[e], qs[e + 1], z);
      f32x2 err;
      sum.hi = two_sum(sum.hi, w.hi, err);
      sum.lo = add2(sum.lo, add2(err, w.lo));
    }
  }
  const float2 h = unpair2(sum.hi), l = unpair2(sum.lo);
  return warp_sum(add_two(Two{h.x, l.x}, Two{h.y, l.y}));
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
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// A list of sums by one warp, a lane a stretch of it in order.
struct Listed {
  int from, to;
  Two upto;  // all up to the end of this lane's
  __device__ __forceinline__ Listed(const float2* list, int n, int lane) {
    const int per = (n + 31) / 32;
    from = min(lane * per, n);
    to = min(from + per, n);
    Two mine{0.f, 0.f};
    for (int i = from; i < to; ++i) {
      const float2 x = __ldcg(list + i);
      mine = add_two(mine, Two{x.x, x.y});
    }
    upto = warp_scan(mine, lane);
  }
  __device__ __forceinline__ Two total() const { return shfl_at(upto, 31); }
};

template <typename T>
__global__ void __launch_bounds__(kDrawThreads) verify_draw_kernel(const DraftArgs a) {
  using R = Row<T, kDrawChunk>;
  constexpr int W = kDrawThreads / 32;
  static_assert(kDrawChunk == 2 * kDrawThreads, "a pair of elements for each thread");
  __shared__ float s_max[kMaxDrafts + 1];
  __shared__ int s_best[kMaxDrafts + 1];
  __shared__ bool s_ok[kMaxDrafts + 1];
  __shared__ Two s_total, s_before, s_want, s_part[W];
  __shared__ int s_chunk, s_token, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = cluster_size(), rank = cluster_rank(), b = blockIdx.x / size;
  griddep_wait();
  const float t = __ldg(a.temperature + b);
  const int n = a.n_drafts != nullptr ? min(max(__ldg(a.n_drafts + b), 0), a.S - 1) : a.S - 1;
  const Warmth c(t);
  float x[R::kSteps][R::kPer];
  if (a.S == 1) {  // no launch in front has looked at the row
    const R r(a, b);
    for (int k = rank * W + warp; k < a.draws; k += size * W) {
      const float m = r.chunk(k, lane, x);
      const int best = c.greedy ? place_of(r, k, lane, x, m) : 0;
      if (lane == 0) a.stats[(long long)b * a.draws + k] = make_float2(m, __int_as_float(best));
    }
    cluster_meet();
  }
  // every row's statistics, and its draft's test
  const int listed = a.S == 1 ? a.draws : a.chunks;
  for (int i = warp; i <= n; i += W) {
    const long long row = (long long)b * a.S + i;
    const float2* const st = a.stats + row * listed;
    const int d = i < n ? __ldg(a.drafts + (long long)b * (a.S - 1) + i) : -1;
    const bool real = d >= 0 && d < a.V;
    float m = -INFINITY;
    for (int k = lane; k < listed; k += 32) m = fmaxf(m, __ldcg(&st[k].x));
    const float xd = real ? logit(static_cast<const T*>(a.logits) + row * a.stride + d) : -INFINITY;
    float q = a.probs != nullptr && real ? __ldg(a.probs + ((long long)b * (a.S - 1) + i) * a.V + d) : 1.f;
    q = q > 0.f ? q : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float z = 0.f, p = 0.f;
    int best = INT_MAX;
    if (c.greedy) {
      for (int k = lane; k < listed; k += 32) {
        const float2 s = __ldcg(st + k);
        if (s.x == m) best = min(best, __float_as_int(s.y));
      }
      best = __reduce_min_sync(0xffffffffu, best);
      z = 1.f;
      p = real && d == best ? 1.f : 0.f;
    } else if (i < n && m != -INFINITY) {
      for (int k = lane; k < listed; k += 32) {
        const float2 s = __ldcg(st + k);
        z += s.y * exp2f((s.x - m) * c.hi);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
      p = exp2f((xd - m) * c.hi);
    }
    if (lane == 0) {
      s_ok[i] = i < n && real && __ldg(a.uniforms + (long long)b * a.S + i) * q * z < p;
      s_max[i] = m;
      s_best[i] = best;
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
  const int gone = missed && a.probs == nullptr ? __ldg(a.drafts + (long long)b * (a.S - 1) + j) : INT_MIN;
  const float* const q = rest ? a.probs + ((long long)b * (a.S - 1) + j) * a.V : nullptr;
  float2* const sums = a.sums + (long long)b * a.draws;
  float2* const rests = a.rests + (long long)b * a.draws;
  for (int k = rank * W + warp; k < a.draws; k += size * W) {
    r.chunk(k, lane, x);
    const Two s = chunk_sum(r, weigh, k, lane, x, gone, nullptr, Two{0.f, 0.f});
    if (lane == 0) sums[k] = make_float2(s.hi, s.lo);
  }
  cluster_meet();
  const float2* list = sums;
  Two z{0.f, 0.f};
  bool left = false;  // whether the drafter's probabilities leave anything
  if (rest) {
    if (warp == 0) {
      const Two all = Listed(sums, a.draws, lane).total();
      if (lane == 0) s_total = all;
    }
    __syncthreads();
    z = s_total;
    for (int k = rank * W + warp; k < a.draws; k += size * W) {
      r.chunk(k, lane, x);
      const Two s = chunk_sum(r, weigh, k, lane, x, INT_MIN, q, z);
      if (lane == 0) rests[k] = make_float2(s.hi, s.lo);
    }
    cluster_meet();
  }
  if (rank != 0) return;
  // the chunk that the draw falls into
  if (warp == 0) {
    Listed l(rest ? rests : sums, a.draws, lane);
    list = rest ? rests : sums;
    left = rest;
    if (rest && !(l.total().hi > 0.f)) {  // nothing: from the row itself
      l = Listed(sums, a.draws, lane);
      list = sums;
      left = false;
    }
    const Two all = l.total();
    const float u = __ldg(a.uniforms + (long long)b * a.S + a.S - 1), p = __fmul_rn(u, all.hi);
    const Two want{p, fmaf(u, all.lo, fmaf(u, all.hi, -p))};
    const unsigned hit = __ballot_sync(0xffffffffu, exceeds(l.upto, want));
    // its lane, and the running sum in front; a random number of 1 and above, or none: the last one's
    const int at = hit ? __ffs(hit) - 1 : 31;
    const Two front = at > 0 ? shfl_at(l.upto, at - 1) : Two{0.f, 0.f};
    if (lane == at) {
      int chunk = -1, i = hit ? l.from : 0;
      Two run = hit ? front : Two{0.f, 0.f}, before = run, bound = want;
      for (; i < a.draws; ++i) {
        const float2 s = __ldcg(list + i);
        const Two next = add_two(run, Two{s.x, s.y});
        if (s.x > 0.f) {
          chunk = i;
          before = run;
          if (exceeds(next, want)) break;
        }
        run = next;
      }
      if (chunk < 0) {  // only roundings of the running sum were behind: the last weight there is
        for (i = l.from - 1; i >= 0 && chunk < 0; --i)
          if (__ldcg(list + i).x > 0.f) chunk = i;
        bound = Two{INFINITY, 0.f};
      }
      s_chunk = all.hi > 0.f ? chunk : -1;
      s_before = before;
      s_want = bound;
      s_total = Two{left ? 1.f : 0.f, 0.f};
      s_token = INT_MAX;
      s_last = -1;
    }
  }
  __syncthreads();
  if (s_chunk < 0) {  // all weight was the draft's that was not kept
    if (tid == 0) a.next[b] = gone;
    return;
  }
  // and the token in it: two elements a thread, in order
  const int v0 = r.first(s_chunk, 0, 0) + 2 * tid;
  Pair w = weigh(v0 == gone ? -INFINITY : r.at(v0), v0 + 1 == gone ? -INFINITY : r.at(v0 + 1));
  if (s_total.hi > 0.f)
    w = rest_of(w, v0 >= 0 && v0 < a.V ? __ldg(q + v0) : 0.f, v0 + 1 >= 0 && v0 + 1 < a.V ? __ldg(q + v0 + 1) : 0.f, z);
  const float2 h = unpair2(w.hi), l = unpair2(w.lo);
  const Two w0{h.x, l.x}, w1{h.y, l.y}, mine = add_two(w0, w1), incl = warp_scan(mine, lane);
  if (lane == 31) s_part[warp] = incl;
  __syncthreads();
  Two run = s_before;
  for (int k = 0; k < warp; ++k) run = add_two(run, s_part[k]);
  const Two up = shfl_up(incl, 1);
  if (lane > 0) run = add_two(run, up);
  const Two want = s_want;
  run = add_two(run, w0);
  if (w0.hi > 0.f) {
    if (exceeds(run, want)) atomicMin(&s_token, v0);
    atomicMax(&s_last, v0);
  }
  run = add_two(run, w1);
  if (w1.hi > 0.f) {
    if (exceeds(run, want)) atomicMin(&s_token, v0 + 1);
    atomicMax(&s_last, v0 + 1);
  }
  __syncthreads();
  if (tid == 0) a.next[b] = s_token != INT_MAX ? s_token : s_last;
}

int chunks_of(int V, int chunk) { return (int)(((long long)V + 7 + chunk - 1) / chunk); }

size_t drafts_stats(int B, int S, int V) {
  return round_256((size_t)B * (S == 1 ? chunks_of(V, kDrawChunk) : (size_t)S * chunks_of(V, kStatChunk)) * 8);
}

size_t drafts_need(int B, int S, int V) {
  if (B < 1 || S < 1 || S > kMaxDrafts + 1 || V < 1 || V > (1 << 24) || B > (1 << 24)) return 0;
  if ((unsigned long long)B * S * ((chunks_of(V, kStatChunk) + 3) / 4) > INT_MAX) return 0;
  return kHeaderBytes + drafts_stats(B, S, V) + 2 * round_256((size_t)B * chunks_of(V, kDrawChunk) * 8);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T>
cudaError_t drafts_launch(const DraftArgs& a, cudaStream_t st) {
  constexpr int W = kStatThreads / 32;
  if (a.S > 1) {
    const unsigned grid = (unsigned)((long long)a.B * a.S * ((a.chunks + W - 1) / W));
    const cudaError_t e = launch_pdl(verify_stats_kernel<T>, dim3(grid), dim3(kStatThreads), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  int cluster = 1;  // CTAs of a sequence: a chunk for every warp, eight at most
  while (cluster < kMaxCluster && cluster * (kDrawThreads / 32) < a.draws) cluster *= 2;
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
  char* const at = static_cast<char*>(ws) + sdv::kHeaderBytes;
  a.stats = reinterpret_cast<float2*>(at);
  a.sums = reinterpret_cast<float2*>(at + sdv::drafts_stats(B, S, V));
  a.rests = a.sums + sdv::round_256((size_t)B * a.draws * 8) / 8;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return sdv::status_of(dtype == SDV_F32   ? sdv::drafts_launch<float>(a, st)
                        : dtype == SDV_F16 ? sdv::drafts_launch<__half>(a, st)
                                           : sdv::drafts_launch<__nv_bfloat16>(a, st));
}

}  // extern "C"

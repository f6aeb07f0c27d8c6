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
// draws from the one row left.
//
// A draw compares running sums of up to 10^5 weights with a random number, so an error of e of
// the total gives another token with a chance of 10^5 e: 32-bit weights, whose errors of 2^-24
// add up to 10^-9 of the total or more, would miss one draw in some thousands.  The row's weights
// are therefore computed to 2^-36 of each as pairs of floats (2^x by a table of 2^(k/32) and a
// short polynomial: Tang, "Table-driven implementation of the exponential function", ACM TOMS
// 1989) and their sums carry the rounding of every addition along (Knuth's two-sum).
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

constexpr int kChunk = 2048;       // logits of a warp's unit of work
constexpr int kStatThreads = 128;
constexpr int kDrawThreads = 256;
constexpr int kMaxDrafts = 31;

struct DraftArgs {
  const void* logits;
  long long stride;           // elements between rows
  const float* temperature;   // [B]
  const int32_t *drafts, *n_drafts;
  const float *probs, *uniforms;
  int32_t *accepted, *next;
  int B, S, V, chunks;
  float2* stats;              // [B * S][chunks]: maximum, sum (greedy: the bits of its place)
  double *sums, *rests;       // [B][chunks]: the drawn row's weights, and what the drafter's leave of them
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
// which lie before the row; a chunk is kChunk elements of groups, 32 groups (one a lane) a step.
template <typename T>
struct Row {
  static constexpr int kPer = 16 / sizeof(T);            // elements of a group
  static constexpr int kSteps = kChunk / kPer / 32;      // groups of a lane in a chunk
  const T* p;
  int V, shift;
  __device__ __forceinline__ Row(const DraftArgs& a, long long row)
      : p(static_cast<const T*>(a.logits) + row * a.stride), V(a.V) {
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  }
  __device__ __forceinline__ int first(int chunk, int step, int lane) const {  // element of a group's start
    return (chunk * (kChunk / kPer) + step * 32 + lane) * kPer - shift;
  }
  __device__ __forceinline__ bool whole(int v) const { return v >= 0 && v + kPer <= V; }
  __device__ __forceinline__ uint4 load(int v) const { return __ldg(reinterpret_cast<const uint4*>(p + v)); }
  // Element v + e as it counts; outside the row -inf.
  __device__ __forceinline__ float at(int v) const {
    return v >= 0 && v < V ? counted_logit((float)__ldg(p + v)) : -INFINITY;
  }
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

// 1 / T in the log2 domain as a pair; greedy where T is 0, below, NaN, or so small that it overflows.
struct Warmth {
  float hi, lo;
  bool greedy;
  __device__ __forceinline__ explicit Warmth(float t) {
    const double c = 1.4426950408889634 / (double)t;
    hi = fmaxf((float)c, 1e-44f);  // an infinite T: all equal, and 0 times -inf nowhere
    lo = (float)(c - (double)hi);
    greedy = !(t > 0.f) || !(hi < INFINITY);
  }
};

template <typename T>
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(const DraftArgs a) {
  using R = Row<T>;
  constexpr int W = kStatThreads / 32;
  const int lane = threadIdx.x & 31, blocks = (a.chunks + W - 1) / W;
  const long long row = blockIdx.x / blocks;
  const int chunk = (int)(blockIdx.x - row * blocks) * W + (threadIdx.x >> 5);
  const int b = (int)(row / a.S), i = (int)(row - (long long)b * a.S);
  griddep_wait();
  griddep_launch_dependents();
  const int n = a.n_drafts != nullptr ? min(max(__ldg(a.n_drafts + b), 0), a.S - 1) : a.S - 1;
  if (chunk >= a.chunks || i > n) return;
  const R r(a, row);
  const Warmth c(__ldg(a.temperature + b));
  uint4 raw[R::kSteps];
#pragma unroll
  for (int s = 0; s < R::kSteps; ++s) {
    const int v = r.first(chunk, s, lane);
    if (r.whole(v)) raw[s] = r.load(v);
  }
  float m = -INFINITY;
  float x[R::kSteps][R::kPer];
#pragma unroll
  for (int s = 0; s < R::kSteps; ++s) {
    const int v = r.first(chunk, s, lane);
    if (r.whole(v)) {
      group_floats(raw[s], x[s], T());
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) x[s][e] = counted_logit(x[s][e]);
    } else {
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) x[s][e] = r.at(v + e);
    }
#pragma unroll
    for (int e = 0; e < R::kPer; ++e) m = fmaxf(m, x[s][e]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float2 out = make_float2(m, 0.f);
  if (c.greedy) {
    int best = INT_MAX;
#pragma unroll
    for (int s = 0; s < R::kSteps; ++s)
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) {
        const int v = r.first(chunk, s, lane) + e;
        if (x[s][e] == m && v >= 0 && v < a.V) best = min(best, v);
      }
    out.y = __int_as_float(__reduce_min_sync(0xffffffffu, best));
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
  if (lane == 0) a.stats[row * a.chunks + chunk] = out;
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

// 2^((x - M) c) for the two x of a pair, to some 2^-36 of each; 0 where it is below 2^-125 and
// where x is -inf.  For all lanes of a warp: lane k holds 2^(k/32).
struct Weigher {
  float M, c_hi, c_lo, pow_hi, pow_lo, least;
  __device__ __forceinline__ Weigher(float m, const Warmth& c, int lane)
      : M(m), c_hi(c.hi), c_lo(c.lo), pow_hi(kPowHi[lane]), pow_lo(kPowLo[lane]), least(m - 125.f / c.hi) {}
  __device__ __forceinline__ Pair operator()(float x0, float x1) const {
    const bool in0 = x0 >= least && x0 > -INFINITY, in1 = x1 >= least && x1 > -INFINITY;
    const f32x2 x = pair2(in0 ? x0 : M, in1 ? x1 : M);
    f32x2 d_lo;
    const f32x2 d = two_sum(x, both(-M), d_lo), ch = both(c_hi);
    const f32x2 t = mul2(d, ch);
    const f32x2 t_lo = fma2(d, ch, neg2(t));
    const f32x2 tl = add2(t_lo, fma2(d, both(c_lo), mul2(d_lo, ch)));
    // t = k / 32 + r, |r| <= 1 / 64: k in the low bits of a number of 1.5 2^23
    const f32x2 magic = both(12582912.f);
    const f32x2 kk = fma2(t, both(32.f), magic);
    const f32x2 r = fma2(sub2(kk, magic), both(-0.03125f), t);
    const float2 kf = unpair2(kk);
    const int k0 = __float_as_int(kf.x) - 0x4b400000, k1 = __float_as_int(kf.y) - 0x4b400000;
    const f32x2 th = pair2(__shfl_sync(0xffffffffu, pow_hi, k0 & 31), __shfl_sync(0xffffffffu, pow_hi, k1 & 31));
    const f32x2 tlo = pair2(__shfl_sync(0xffffffffu, pow_lo, k0 & 31), __shfl_sync(0xffffffffu, pow_lo, k1 & 31));
    // 2^r = 1 + s + g: s = fl(r ln 2), g the rest
    const f32x2 ln_hi = both(0x1.62e430p-1f), ln_lo = both(-0x1.05c610p-29f);
    const f32x2 quad = fma2(r, fma2(r, both(0.009618129f), both(0.05550411f)), both(0.24022651f));
    const f32x2 s = mul2(r, ln_hi);
    f32x2 g = fma2(r, ln_hi, neg2(s));
    g = fma2(r, ln_lo, g);
    g = fma2(tl, ln_hi, g);
    g = fma2(mul2(r, r), quad, g);
    const f32x2 p = mul2(th, s);
    Pair w;
    w.hi = add2(th, p);
    f32x2 l = add2(sub2(th, w.hi), p);  // exact: th is the larger
    l = add2(l, fma2(th, s, neg2(p)));
    l = fma2(th, g, l);
    w.lo = add2(l, fma2(tlo, s, tlo));
    const int n0 = k0 >> 5, n1 = k1 >> 5;
    const f32x2 scale = pair2(in0 ? __int_as_float((n0 + 127) << 23) : 0.f, in1 ? __int_as_float((n1 + 127) << 23) : 0.f);
    w.hi = mul2(w.hi, scale);
    w.lo = mul2(w.lo, scale);
    return w;
  }
};

// What max(w - q Z, 0) leaves, Z = z_hi + z_lo.
__device__ __forceinline__ Pair rest_of(const Pair& w, float q0, float q1, float z_hi, float z_lo) {
  const f32x2 q = pair2(q0 > 0.f ? q0 : 0.f, q1 > 0.f ? q1 : 0.f);
  const f32x2 a = mul2(q, both(z_hi));
  const f32x2 al = fma2(q, both(z_lo), fma2(q, both(z_hi), neg2(a)));
  f32x2 err;
  const f32x2 d = two_sum(w.hi, neg2(a), err);
  const f32x2 l = add2(err, sub2(w.lo, al));
  const float2 sum = unpair2(add2(d, l)), dh = unpair2(d), dl = unpair2(l);
  Pair r;
  r.hi = pair2(sum.x > 0.f ? dh.x : 0.f, sum.y > 0.f ? dh.y : 0.f);
  r.lo = pair2(sum.x > 0.f ? dl.x : 0.f, sum.y > 0.f ? dl.y : 0.f);
  return r;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// A chunk's weights added up: of the row, without token `gone`, or (q given) what q leaves.
template <typename T>
__device__ __forceinline__ double chunk_sum(const Row<T>& r, const Weigher& weigh, int chunk, int lane, int gone,
                                            const float* q, float z_hi, float z_lo) {
  using R = Row<T>;
  Pair sum{both(0.f), both(0.f)};
  constexpr int kAhead = 4;
#pragma unroll 1
  for (int s0 = 0; s0 < R::kSteps; s0 += kAhead) {
    float x[kAhead][R::kPer], qs[kAhead][R::kPer];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int v = r.first(chunk, s0 + s, lane);
      if (r.whole(v)) {
        group_floats(r.load(v), x[s], T());
#pragma unroll
        for (int e = 0; e < R::kPer; ++e) x[s][e] = counted_logit(x[s][e]);
      } else {
#pragma unroll
        for (int e = 0; e < R::kPer; ++e) x[s][e] = r.at(v + e);
      }
#pragma unroll
      for (int e = 0; e < R::kPer; ++e) {
        if (v + e == gone) x[s][e] = -INFINITY;
        qs[s][e] = q != nullptr && v + e >= 0 && v + e < r.V ? __ldg(q + v + e) : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int e = 0; e < R::kPer; e += 2) {
        Pair w = weigh(x[s][e], x[s][e + 1]);
        if (q != nullptr) w = rest_of(w, qs[s][e], qs[s][e + 1], z_hi, z_lo);
        f32x2 err;
        sum.hi = two_sum(sum.hi, w.hi, err);
        sum.lo = add2(sum.lo, add2(err, w.lo));
      }
  }
  const float2 h = unpair2(sum.hi), l = unpair2(sum.lo);
  return warp_sum(((double)h.x + (double)h.y) + ((double)l.x + (double)l.y));
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

// The total of a list of sums, and (u >= 0) the first one at which the running total exceeds
// u of it, with the running total in front: by one warp, in a fixed order.
__device__ __forceinline__ double list_total(const double* sums, int n, int lane) {
  double t = 0.0;
  for (int i = lane; i < n; i += 32) t += __ldcg(sums + i);
  return warp_sum(t);
}

template <typename T>
__global__ void __launch_bounds__(kDrawThreads) verify_draw_kernel(const DraftArgs a) {
  constexpr int W = kDrawThreads / 32;
  __shared__ float s_max[kMaxDrafts + 1];
  __shared__ int s_best[kMaxDrafts + 1];
  __shared__ bool s_ok[kMaxDrafts + 1];
  __shared__ double s_total, s_before, s_part[W];
  __shared__ int s_chunk, s_token, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int size = cluster_size(), rank = cluster_rank(), b = blockIdx.x / size;
  griddep_wait();
  const int n = a.n_drafts != nullptr ? min(max(__ldg(a.n_drafts + b), 0), a.S - 1) : a.S - 1;
  const Warmth c(__ldg(a.temperature + b));
  // every row's statistics, and its draft's test
  for (int i = warp; i <= n; i += W) {
    const long long row = (long long)b * a.S + i;
    const float2* const st = a.stats + row * a.chunks;
    float m = -INFINITY;
    int best = INT_MAX;
    for (int k = lane; k < a.chunks; k += 32) m = fmaxf(m, __ldcg(&st[k].x));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    double z = 0.0;
    if (m != -INFINITY) {
      for (int k = lane; k < a.chunks; k += 32) {
        const float2 s = __ldcg(st + k);
        if (c.greedy) best = s.x == m ? min(best, __float_as_int(s.y)) : best;
        else z += (double)(s.y * exp2f((s.x - m) * c.hi));
      }
    }
    best = __reduce_min_sync(0xffffffffu, best);
    z = warp_sum(z);
    const int d = i < n ? __ldg(a.drafts + (long long)b * (a.S - 1) + i) : -1;
    const bool real = d >= 0 && d < a.V;
    const float x = real ? logit(static_cast<const T*>(a.logits) + row * a.stride + d) : -INFINITY;
    double p = 0.0;  // of the draft, times z
    if (c.greedy) {
      z = 1.0;
      p = real && d == best ? 1.0 : 0.0;
    } else if (m != -INFINITY) {
      const float2 h = unpair2(Weigher(m, c, lane)(x, x).hi);
      p = (double)h.x;
    }
    if (lane == 0) {
      float q = 1.f;
      if (a.probs != nullptr && real) q = __ldg(a.probs + ((long long)b * (a.S - 1) + i) * a.V + d);
      q = q > 0.f ? q : 0.f;
      s_ok[i] = i < n && real && (double)__ldg(a.uniforms + (long long)b * a.S + i) * (double)q * z < p;
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
  const Row<T> r(a, (long long)b * a.S + j);
  const Weigher weigh(m, c, lane);
  const bool rest = missed && a.probs != nullptr;
  const int gone = missed && a.probs == nullptr ? __ldg(a.drafts + (long long)b * (a.S - 1) + j) : INT_MIN;
  const float* const q = rest ? a.probs + ((long long)b * (a.S - 1) + j) * a.V : nullptr;
  double* const sums = a.sums + (long long)b * a.chunks;
  double* const rests = a.rests + (long long)b * a.chunks;
  for (int k = rank * W + warp; k < a.chunks; k += size * W) {
    const double s = chunk_sum(r, weigh, k, lane, gone, nullptr, 0.f, 0.f);
    if (lane == 0) sums[k] = s;
  }
  cluster_meet();
  if (warp == 0) {
    const double t = list_total(sums, a.chunks, lane);
    if (lane == 0) s_total = t;
  }
  __syncthreads();
  double total = s_total;
  const double* list = sums;
  const float* q_list = nullptr;
  const float z_hi = (float)total, z_lo = (float)(total - (double)z_hi);
  if (rest) {
    for (int k = rank * W + warp; k < a.chunks; k += size * W) {
      const double s = chunk_sum(r, weigh, k, lane, INT_MIN, q, z_hi, z_lo);
      if (lane == 0) rests[k] = s;
    }
    cluster_meet();
    if (rank != 0) return;
    __syncthreads();  // s_total has been read
    if (warp == 0) {
      const double t = list_total(rests, a.chunks, lane);
      if (lane == 0) s_total = t;
    }
    __syncthreads();
    if (s_total > 0.0) {
      total = s_total;
      list = rests;
      q_list = q;
    }
  }
  if (rank != 0) return;
  const int without = total > 0.0 ? gone : INT_MIN;
  if (!(total > 0.0)) {
    // nothing is left without the draft: from the row itself, of which only the draft's weight counts
    if (tid == 0) a.next[b] = gone;
    return;
  }
  // the chunk that the draw falls into
  const double want = (double)__ldg(a.uniforms + (long long)b * a.S + a.S - 1) * total;
  if (warp == 0) {
    double before = 0.0, in_front = 0.0;
    int at = -1, last = -1;
    double last_front = 0.0;
    for (int k0 = 0; k0 < a.chunks && at < 0; k0 += 32) {
      const double s = k0 + lane < a.chunks ? __ldcg(list + k0 + lane) : 0.0;
      double incl = s;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, s > 0.0 && before + incl > want);
      const unsigned some = __ballot_sync(0xffffffffu, s > 0.0);
      if (hit) {
        const int l = __ffs(hit) - 1;
        at = k0 + l;
        in_front = before + __shfl_sync(0xffffffffu, incl - s, l);
      } else if (some) {
        const int l = 31 - __clz(some);
        last = k0 + l;
        last_front = before + __shfl_sync(0xffffffffu, incl - s, l);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      s_chunk = at >= 0 ? at : last;
      s_before = at >= 0 ? in_front : last_front;
      s_token = INT_MAX;
      s_last = -1;
    }
  }
  __syncthreads();
  // and the token in it: a thread has eight elements, in order
  constexpr int E = kChunk / kDrawThreads;
  const int v0 = r.first(s_chunk, 0, 0) + tid * E;
  double w[E], mine = 0.0;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    float x[2], qs[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int v = v0 + e + z;
      x[z] = v == without ? -INFINITY : r.at(v);
      qs[z] = q_list != nullptr && v >= 0 && v < a.V ? __ldg(q_list + v) : 0.f;
    }
    Pair p = weigh(x[0], x[1]);
    if (q_list != nullptr) p = rest_of(p, qs[0], qs[1], z_hi, z_lo);
    const float2 h = unpair2(p.hi), l = unpair2(p.lo);
    w[e] = (double)h.x + (double)l.x;
    w[e + 1] = (double)h.y + (double)l.y;
    mine += w[e];
    mine += w[e + 1];
  }
  double incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_part[warp] = incl;
  __syncthreads();
  double run = s_before + (incl - mine);
  for (int k = 0; k < warp; ++k) run += s_part[k];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    run += w[e];
    if (w[e] > 0.0) {
      if (run > want) atomicMin(&s_token, v0 + e);
      atomicMax(&s_last, v0 + e);
    }
  }
  __syncthreads();
  if (tid == 0) a.next[b] = s_token != INT_MAX ? s_token : s_last;
}

int draft_chunks(int V) { return (int)(((long long)V + 7 + kChunk - 1) / kChunk); }

size_t drafts_need(int B, int S, int V) {
  if (B < 1 || S < 1 || S > kMaxDrafts + 1 || V < 1 || V > (1 << 24) || B > (1 << 24)) return 0;
  const size_t chunks = draft_chunks(V);
  if ((unsigned long long)B * S * ((chunks + 3) / 4) > INT_MAX) return 0;
  return kHeaderBytes + round_256((size_t)B * S * chunks * 8) + 2 * round_256((size_t)B * chunks * 8);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T>
cudaError_t drafts_launch(const DraftArgs& a, cudaStream_t st) {
  constexpr int W = kStatThreads / 32;
  const unsigned grid = (unsigned)((long long)a.B * a.S * ((a.chunks + W - 1) / W));
  cudaError_t e = launch_pdl(verify_stats_kernel<T>, dim3(grid), dim3(kStatThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  const int cluster = 8;
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
  a.chunks = sdv::draft_chunks(V);
  char* const at = static_cast<char*>(ws) + sdv::kHeaderBytes;
  a.stats = reinterpret_cast<float2*>(at);
  a.sums = reinterpret_cast<double*>(at + sdv::round_256((size_t)B * S * a.chunks * 8));
  a.rests = a.sums + sdv::round_256((size_t)B * a.chunks * 8) / 8;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return sdv::status_of(dtype == SDV_F32   ? sdv::drafts_launch<float>(a, st)
                        : dtype == SDV_F16 ? sdv::drafts_launch<__half>(a, st)
                                           : sdv::drafts_launch<__nv_bfloat16>(a, st));
}

}  // extern "C"

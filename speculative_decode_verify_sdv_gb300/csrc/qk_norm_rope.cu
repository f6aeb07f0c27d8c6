// Norms of query and key heads, the rotation by their positions, and the rows' way out: queries
// to a tensor, keys and values into a paged cache (sdv_qk_norm_rope); the angles per position
// (sdv_rope_steps).
//
// Per head of `dim` elements: y = x / sqrt(mean x^2 + eps) w; then its first rot_dim elements in
// pairs (a, b) at angle phi: (A (a cos phi - b sin phi), A (b cos phi + a sin phi)).  phi of
// position p and pair i is 2 pi frac(p step_i / 2^64): the 64-bit product p step_i wraps around
// whole turns, so the angle of any position is exact to 2^-26 turns (the fraction's rounding to a
// float) where p * frequency in 32 bits would have lost 2^-24 of hundreds of turns.
//
// A warp per token and part of its heads; a head takes dim / 8 lanes of eight elements each.
// The token's angles are computed once, one or more a lane, and go round through shared memory;
// cos and sin times the norm's weights then serve all query heads, and once more all key heads.
// Reading the rows and writing them bounds it: six prompts, 24,857 rows of 32 heads over 8 of 128
// in fp16, 611 MB, in 119 us, 5.1 TB/s; 58 M warp instructions take half the issue slots there, and
// blocks for one wave (five an SM, four for fp32 rows) loop over the tokens.  One row is the call itself,
// 2.9 us on the GPU, 257 rows of a round 4.3: the loads' latencies one after another, position, row and steps.
//
// What it is built for is heads that fill their lanes, rotated whole, in pairs or by a multiple of 16.
// 24,857 rows of some 6000 elements, times of the floor (bytes at the copy's rate), 16-bit and fp32 rows: heads of
// 64, 128 and 256 in halves 1.29 1.12, 1.23 1.10, 1.35 1.18, in pairs 1.23 1.06, 1.16 1.04, 1.27 1.10.  Heads
// of 80 leave six of their 16 lanes idle: 1.79 1.55 and 1.65 1.40; of 96 four, 1.54 1.34 and 1.43 1.23.
// A part of another length in halves (a quarter of the head, 12 to 60 elements) goes element by element
// through shared memory: 2.2 to 2.5 times the floor for heads of 64, 128 and 256, 3.6 and 3.1 for 80 and 96.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "host_util.h"
#include "mixing.h"
#include "sdv.h"
#include "sdv_device.cuh"
#include "tc_util.cuh"

namespace sdv {

namespace {

struct RopeArgs {
  const void *q, *k, *v;                     // rows of a token at strides in elements; q or k and v may be null
  long long q_stride, k_stride, v_stride;
  const float *q_weight, *k_weight;          // or null: no norm
  float eps;
  const unsigned long long* steps;           // [rot / 2]
  float amplitude;
  int rot;
  const int32_t *positions, *slots;          // [tokens]
  void *q_out, *ck, *cv;
  long long tokens;
  int q_heads, kv_heads, dim, page;
  long long slots_most;                      // n_pages * page
  int lanes;                                 // lanes of a head, a power of two
  int parts, per_part;                       // parts of a token, heads of one (a multiple of a warp's)
  int* status;
};

// 1 / sqrt(x), to 2^-22.
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

enum RopeForm { kRopeNone, kRopePairs, kRopeHalf, kRopeHalfOdd };

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;  // heads loaded before the first is used

template <typename T>
struct Chunk {  // eight elements as they lie
  uint4 x;
  __device__ __forceinline__ void load(const T* p) { x = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void pairs(f32x2 (&f)[4]) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = unpack16<T>(w[i]);
      f[i] = pair2(y.x, y.y);
    }
  }
  __device__ __forceinline__ void clear() { x = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void from_lane(int lane) {
    x.x = __shfl_sync(0xffffffffu, x.x, lane);
    x.y = __shfl_sync(0xffffffffu, x.y, lane);
    x.z = __shfl_sync(0xffffffffu, x.z, lane);
    x.w = __shfl_sync(0xffffffffu, x.w, lane);
  }
  template <typename TO>
  __device__ __forceinline__ uint4 packed() const {
    static_assert(std::is_same<T, TO>::value, "rows of the cache's type");
    return x;
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void pairs(f32x2 (&f)[4]) const {
    f[0] = pair2(a.x, a.y), f[1] = pair2(a.z, a.w), f[2] = pair2(b.x, b.y), f[3] = pair2(b.z, b.w);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void from_lane(int lane) {
    float* const f[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) *f[e] = __shfl_sync(0xffffffffu, *f[e], lane);
  }
  template <typename TO>
  __device__ __forceinline__ uint4 packed() const {
    return make_uint4(pack16<TO>(a.x, a.y), pack16<TO>(a.z, a.w), pack16<TO>(b.x, b.y), pack16<TO>(b.z, b.w));
  }
};

// Signed turns of position p at a step of 2^-64 turns, doubled: half turns in [-1, 1).
__device__ __forceinline__ float half_turns(int p, unsigned long long step) {
  return (float)(int)((step * (unsigned long long)p) >> 32) * 0x1p-31f;
}

// A head's eight elements of this lane, those of the partners in the same order.
template <typename TI, typename T, int FORM>
struct RopeLane {
  int lane, c, e0, half, rot;
  bool mine, turned;
  float* mem;  // the head's elements, for partners that are not a lane's chunk

  __device__ __forceinline__ void partners(const Chunk<TI>& raw, const f32x2 (&x)[4], f32x2 (&other)[4]) const {
    if constexpr (FORM == kRopePairs) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = unpair2(x[e]);
        other[e] = e0 + 2 * e < rot ? pair2(v.y, v.x) : 0;
      }
    } else if constexpr (FORM == kRopeHalf) {
      const int from = (lane - c + (e0 < half ? c + half / 8 : c - half / 8)) & 31;
      Chunk<TI> o = raw;
      o.from_lane(from);
      if (!turned) o.clear();
      o.pairs(other);
    } else if constexpr (FORM == kRopeHalfOdd) {
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<f32x2*>(mem + e0 + 2 * e) = x[e];
      __syncwarp();
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int el = e0 + e;
        y[e] = el < half ? mem[el + half] : el < rot ? mem[el - half] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) other[e] = pair2(y[2 * e], y[2 * e + 1]);
    }
  }
};

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// LANES: of a head (0: any number, read from the arguments).
template <typename TI, typename T, int FORM, int LANES>
__global__ void __launch_bounds__(kRopeThreads, sizeof(TI) == 2 ? 5 : 4) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int W = kRopeThreads / 32;
  __shared__ alignas(16) float exchange[FORM == kRopeHalfOdd ? kRopeThreads * 8 : 1];
  __shared__ alignas(16) float2 turns[FORM == kRopeNone ? 1 : W][FORM == kRopeNone ? 1 : 128 + 4];  // A cos, A sin of a pair
  const int lane = threadIdx.x & 31;
  const int L = LANES != 0 ? LANES : a.lanes, sub = lane / L, at_once = 32 / L;
  RopeLane<TI, T, FORM> me;
  me.lane = lane;
  me.c = lane & (L - 1);
  me.e0 = me.c * 8;
  me.rot = a.rot;
  me.half = a.rot / 2;
  me.mine = me.e0 < a.dim;
  me.turned = me.mine && me.e0 < a.rot;
  me.mem = exchange + (FORM == kRopeHalfOdd ? (threadIdx.x - me.c) * 8 : 0);
  const int e0 = me.e0;
  const bool mine = me.mine;
  float2* const angle = turns[FORM == kRopeNone ? 0 : threadIdx.x >> 5];
  const long long warp = (long long)blockIdx.x * W + (threadIdx.x >> 5);
  const long long warps = (long long)gridDim.x * W;
  const float inv_dim = 1.f / (float)a.dim;
  griddep_wait();
  griddep_launch_dependents();
  const int q_heads = a.q_heads, kv = a.kv_heads, all = q_heads + 2 * kv;
  for (long long item = warp; item < a.tokens * a.parts; item += warps) {
    const long long t = a.parts == 1 ? item : item / a.parts;
    const int h0 = (int)(item - t * a.parts) * a.per_part, h1 = min(h0 + a.per_part, all);
    const int pos = __ldg(a.positions + t);
    if (pos < 0) continue;  // uniform in the warp: not a row
    int slot = -1;
    if (h1 > q_heads) {
      slot = __ldg(a.slots + t);
      if (slot >= a.slots_most) {
        if (lane == 0 && a.status != nullptr) atomicOr(a.status, kDevErrIndex);
        slot = -1;
      }
    }
    const int id = slot < 0 ? 0 : slot / a.page;
    const long long row = ((long long)id * kv * a.page + (slot - id * a.page)) * a.dim;  // head 0 of the slot
    // the first query heads' loads go out before the angles are computed
    Chunk<TI> raw[kRopeAhead];
    const bool early = h0 < q_heads && h0 + at_once * kRopeAhead <= min(h1, q_heads);
    if (early) {
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        if (mine) raw[u].load(static_cast<const TI*>(a.q) + t * a.q_stride + (h0 + u * at_once + sub) * a.dim + e0);
        else raw[u].clear();
      }
    }
    if constexpr (FORM != kRopeNone) {
      if (h0 < q_heads + kv) {
        __syncwarp();  // the last token's have been read
        for (int i = lane; i < me.half; i += 32) {
          float s, co;
          sincospif(half_turns(pos, __ldg(a.steps + i)), &s, &co);
          angle[i] = make_float2(co * a.amplitude, s * a.amplitude);
        }
        __syncwarp();
      }
    }
    // query heads, then key heads
#pragma unroll 1
    for (int keys = 0; keys < 2; ++keys) {
      const int first = keys ? q_heads : 0, end = keys ? q_heads + kv : q_heads;
      const int from = max(h0, first), to = min(h1, end);
      if (from >= to || (keys && slot < 0)) continue;
      const float* const w = keys ? a.k_weight : a.q_weight;
      // the factors of this lane's elements and of their partners: y = x cos + partner sin, where the
      // first of a pair takes - sin and the second + sin
      float fo[8], ff[8], wo[8], wf[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wo[e] = wf[e] = 1.f;
      if (w != nullptr && mine) {
        load8(w + e0, wo);
        if (FORM == kRopeHalf && me.turned) load8(w + (e0 < me.half ? e0 + me.half : e0 - me.half), wf);
      }
      if constexpr (FORM == kRopeHalf) {
        float cs[16];
        const float2* const at = angle + (me.turned ? (e0 < me.half ? e0 : e0 - me.half) : 0);
        load8(reinterpret_cast<const float*>(at), cs);
        load8(reinterpret_cast<const float*>(at) + 8, cs + 8);
        const float sign = e0 < me.half ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          fo[e] = me.turned ? cs[2 * e] * wo[e] : wo[e];
          ff[e] = me.turned ? sign * cs[2 * e + 1] * wf[e] : 0.f;
        }
      } else if constexpr (FORM == kRopePairs) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const bool in = e0 + e < a.rot;
          const float2 cs = in ? angle[(e0 + e) / 2] : make_float2(1.f, 0.f);
          fo[e] = cs.x * wo[e];
          fo[e + 1] = cs.x * wo[e + 1];
          ff[e] = -cs.y * wo[e + 1];
          ff[e + 1] = cs.y * wo[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int el = e0 + e;
          fo[e] = wo[e];
          ff[e] = 0.f;
          if (FORM == kRopeNone || el >= a.rot) continue;
          const bool second = el >= me.half;
          const float2 cs = angle[second ? el - me.half : el];
          fo[e] *= cs.x;
          ff[e] = (second ? cs.y : -cs.y) * (w != nullptr && mine ? __ldg(w + (second ? el - me.half : el + me.half)) : 1.f);
        }
      }
      f32x2 own[4], far[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        own[e] = pair2(fo[2 * e], fo[2 * e + 1]);
        far[e] = pair2(ff[2 * e], ff[2 * e + 1]);
      }
      const TI* src = (keys ? static_cast<const TI*>(a.k) + t * a.k_stride : static_cast<const TI*>(a.q) + t * a.q_stride) + e0;
      T* dst = (keys ? static_cast<T*>(a.ck) + row : static_cast<T*>(a.q_out) + t * q_heads * a.dim) + e0;
      const int in_step = at_once * a.dim;                                           // elements between a lane's heads
      const long long out_step = (long long)at_once * (keys ? (long long)a.page * a.dim : a.dim);
      src += (from - first + sub) * a.dim;
      dst += (from - first + sub) * (keys ? (long long)a.page * a.dim : a.dim);
      auto work = [&](const Chunk<TI>& raw, bool live) {
        f32x2 x[4], y[4];
        raw.pairs(x);
        float r = 1.f;
        if (w != nullptr) {
          const f32x2 s2 = fma2(x[3], x[3], fma2(x[2], x[2], fma2(x[1], x[1], mul2(x[0], x[0]))));
          float sum = unpair2(s2).x + unpair2(s2).y;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1)
            if (off < L) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          r = rsqrt_approx(fmaf(sum, inv_dim, a.eps));
        }
        const f32x2 r2 = pair2(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(x[e], own[e]);
        if constexpr (FORM != kRopeNone) {
          f32x2 other[4];
          me.partners(raw, x, other);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = fma2(other[e], far[e], y[e]);
        }
        if (live)
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack16<T>(mul2(y[0], r2)), pack16<T>(mul2(y[1], r2)),
                                                      pack16<T>(mul2(y[2], r2)), pack16<T>(mul2(y[3], r2)));
        dst += out_step;
      };
      int hb = from;
      for (; hb + at_once * kRopeAhead <= to; hb += at_once * kRopeAhead) {
        if (keys || hb > from) {
#pragma unroll
          for (int u = 0; u < kRopeAhead; ++u) {
            if (mine) raw[u].load(src + u * in_step);
            else raw[u].clear();
          }
        }
        src += kRopeAhead * in_step;
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) work(raw[u], mine);
      }
#pragma unroll 1
      for (; hb < to; hb += at_once) {
        Chunk<TI> one;
        const bool live = mine && hb + sub < to;
        if (live) one.load(src);
        else one.clear();
        src += in_step;
        work(one, live);
      }
    }
    // values as they are
    const int from = max(h0, q_heads + kv);
    if (from >= h1 || slot < 0 || !mine) continue;
    const TI* const src = static_cast<const TI*>(a.v) + t * a.v_stride + e0;
    T* const dst = static_cast<T*>(a.cv) + row + e0;
#pragma unroll 4
    for (int h = from + sub; h < h1; h += at_once) {
      Chunk<TI> raw;
      raw.load(src + (h - q_heads - kv) * a.dim);
      *reinterpret_cast<uint4*>(dst + (long long)(h - q_heads - kv) * a.page * a.dim) = raw.template packed<T>();
    }
  }
}

template <typename TI, typename T, int FORM>
cudaError_t rope_form(const RopeArgs& a, int blocks, cudaStream_t st) {
  auto kernel = a.lanes == 16 ? qk_norm_rope_kernel<TI, T, FORM, 16> : qk_norm_rope_kernel<TI, T, FORM, 0>;
  return launch_pdl(kernel, dim3(blocks), dim3(kRopeThreads), 0, st, a);
}

template <typename TI, typename T>
cudaError_t rope_launch(int form, const RopeArgs& a, int blocks, cudaStream_t st) {
  switch (form) {
    case kRopeNone: return rope_form<TI, T, kRopeNone>(a, blocks, st);
    case kRopePairs: return rope_form<TI, T, kRopePairs>(a, blocks, st);
    case kRopeHalf: return rope_form<TI, T, kRopeHalf>(a, blocks, st);
    default: return rope_form<TI, T, kRopeHalfOdd>(a, blocks, st);
  }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool rope_rows(const void* p, long long stride, int heads, int dim) {
  return p != nullptr && is_aligned16(p) && stride % 8 == 0 && stride >= (long long)heads * dim;
}

}  // namespace

}  // namespace sdv

extern "C" {

sdv_status sdv_rope_steps(int32_t rot_dim, double theta, const sdv_rope_scaling* s, uint64_t* steps,
                          float* amplitude_or_null) {
  const int kind = s == nullptr ? SDV_ROPE_PLAIN : s->kind;
  if (steps == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || !(theta > 1.0) || !std::isfinite(theta))
    return SDV_ERR_INVALID_ARG;
  if (kind < SDV_ROPE_PLAIN || kind > SDV_ROPE_BANDS) return SDV_ERR_INVALID_ARG;
  const bool ramp = kind == SDV_ROPE_RAMP || kind == SDV_ROPE_BANDS;
  if (kind != SDV_ROPE_PLAIN && (!(s->factor >= 1.0) || !std::isfinite(s->factor))) return SDV_ERR_INVALID_ARG;
  if (kind == SDV_ROPE_BASE && rot_dim < 4) return SDV_ERR_INVALID_ARG;
  if (ramp && (s->trained < 1 || !(s->low > 0.0) || !(s->high > s->low) || !std::isfinite(s->high)))
    return SDV_ERR_INVALID_ARG;
  const double turn = 6.283185307179586476925;
  if (kind == SDV_ROPE_BASE) theta *= std::pow(s->factor, (double)rot_dim / (rot_dim - 2));
  double from = 0.0, to = 0.0;
  if (kind == SDV_ROPE_RAMP) {
    // the pair's index at which a wave has made `turns` turns in the trained positions
    auto index = [&](double turns) { return rot_dim * std::log(s->trained / (turn * turns)) / (2.0 * std::log(theta)); };
    from = std::fmax(std::floor(index(s->high)), 0.0);
    to = std::fmin(std::ceil(index(s->low)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    double share = 0.0;  // of the interpolated frequency
    if (kind == SDV_ROPE_LINEAR) share = 1.0;
    if (kind == SDV_ROPE_RAMP) share = (i - from) / std::fmax(to - from, 0.001);
    if (kind == SDV_ROPE_BANDS) share = 1.0 - (s->trained * f / turn - s->low) / (s->high - s->low);
    share = std::fmin(1.0, std::fmax(0.0, share));
    if (share > 0.0) f = f / s->factor * share + f * (1.0 - share);
    // turns per position, at most 1 / (2 pi): far below the 2^64 that would wrap
    steps[i] = (uint64_t)std::nearbyint(f / turn * 18446744073709551616.0);
  }
  if (amplitude_or_null != nullptr)
    *amplitude_or_null = kind == SDV_ROPE_RAMP ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.f;
  return SDV_OK;
}

sdv_status sdv_qk_norm_rope(const sdv_kvcache* cache, int32_t in_dtype, const void* q_or_null, const void* k_or_null,
                            const void* v_or_null, int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t B,
                            int32_t T, int32_t Hq, const float* q_weight_or_null, const float* k_weight_or_null,
                            float eps, const sdv_rope* rope_or_null, const int32_t* positions,
                            const int32_t* slots_or_null, void* q_out_or_null, void* ws_or_null,
                            sdv_stream_t stream) {
  using sdv::is_aligned16;
  if (cache == nullptr || (cache->dtype != SDV_F16 && cache->dtype != SDV_BF16) || cache->dim < 8 || cache->dim % 8 != 0)
    return SDV_ERR_INVALID_ARG;
  if (in_dtype != SDV_F32 && in_dtype != cache->dtype) return SDV_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || positions == nullptr || !sdv::aligned4(positions) || !sdv::aligned4(slots_or_null) ||
      !(eps >= 0.f) || !std::isfinite(eps) || !is_aligned16(q_weight_or_null) || !is_aligned16(k_weight_or_null))
    return SDV_ERR_INVALID_ARG;
  const bool q = q_or_null != nullptr, kv = k_or_null != nullptr;
  if ((!q && !kv) || kv != (v_or_null != nullptr) || q != (q_out_or_null != nullptr)) return SDV_ERR_INVALID_ARG;
  if (q && (Hq < 1 || !sdv::rope_rows(q_or_null, q_stride, Hq, cache->dim) || !is_aligned16(q_out_or_null)))
    return SDV_ERR_INVALID_ARG;
  if (kv) {
    if (cache->n_pages < 1 || cache->heads < 1 || cache->page_size < 1 || cache->k == nullptr || cache->v == nullptr ||
        !is_aligned16(cache->k) || !is_aligned16(cache->v) || slots_or_null == nullptr)
      return SDV_ERR_INVALID_ARG;
    if (!sdv::rope_rows(k_or_null, k_stride, cache->heads, cache->dim) ||
        !sdv::rope_rows(v_or_null, v_stride, cache->heads, cache->dim))
      return SDV_ERR_INVALID_ARG;
  }
  int form = sdv::kRopeNone;
  if (rope_or_null != nullptr) {
    const sdv_rope& r = *rope_or_null;
    if (r.rot_dim < 2 || r.rot_dim % 2 != 0 || r.rot_dim > cache->dim || r.steps == nullptr ||
        (reinterpret_cast<uintptr_t>(r.steps) & 7u) != 0 || !std::isfinite(r.amplitude))
      return SDV_ERR_INVALID_ARG;
    if (r.layout == SDV_ROPE_PAIRS) form = sdv::kRopePairs;
    else if (r.layout == SDV_ROPE_HALF) form = r.rot_dim % 16 == 0 ? sdv::kRopeHalf : sdv::kRopeHalfOdd;
    else return SDV_ERR_INVALID_ARG;
  }
  if (!is_aligned16(ws_or_null)) return SDV_ERR_WORKSPACE;
  if (cache->dim > 256 || (q && Hq > 4096) || (kv && cache->heads > 4096)) return SDV_ERR_UNSUPPORTED;
  sdv::RopeArgs a{};
  a.q = q_or_null;
  a.k = k_or_null;
  a.v = v_or_null;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = q_weight_or_null;
  a.k_weight = k_weight_or_null;
  a.eps = eps;
  if (rope_or_null != nullptr) {
    a.steps = reinterpret_cast<const unsigned long long*>(rope_or_null->steps);
    a.amplitude = rope_or_null->amplitude;
    a.rot = rope_or_null->rot_dim;
  }
  a.positions = positions;
  a.slots = slots_or_null;
  a.q_out = q_out_or_null;
  a.ck = cache->k;
  a.cv = cache->v;
  a.tokens = (long long)B * T;
  a.q_heads = q ? Hq : 0;
  a.kv_heads = kv ? cache->heads : 0;
  a.dim = cache->dim;
  a.page = kv ? cache->page_size : 1;
  a.slots_most = kv ? (long long)cache->n_pages * cache->page_size : 0;
  a.status = static_cast<int*>(ws_or_null);
  a.lanes = 1;
  while (a.lanes * 8 < a.dim) a.lanes *= 2;
  const int sms = sdv::sm_count();
  if (sms <= 0) return SDV_ERR_CUDA;
  // a token's heads to as many warps as fill the GPU, a warp's load of heads each at least
  const int heads = a.q_heads + 2 * a.kv_heads, least = 32 / a.lanes;
  const long long room = 16ll * sms;
  int parts = (heads + least - 1) / least;
  if (parts * a.tokens > room) parts = (int)((room + a.tokens - 1) / a.tokens);
  a.per_part = (heads + parts - 1) / parts;
  a.per_part = (a.per_part + least - 1) / least * least;
  a.parts = (heads + a.per_part - 1) / a.per_part;
  const long long per_block = sdv::kRopeThreads / 32, want = (a.tokens * a.parts + per_block - 1) / per_block;
  const long long room_blocks = (in_dtype == SDV_F32 ? 4ll : 5ll) * sms;
  const int blocks = (int)(want < room_blocks ? want : room_blocks);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SDV_BF16;
  cudaError_t e;
  if (in_dtype == SDV_F32)
    e = bf ? sdv::rope_launch<float, __nv_bfloat16>(form, a, blocks, st) : sdv::rope_launch<float, __half>(form, a, blocks, st);
  else
    e = bf ? sdv::rope_launch<__nv_bfloat16, __nv_bfloat16>(form, a, blocks, st)
           : sdv::rope_launch<__half, __half>(form, a, blocks, st);
  return sdv::status_of(e);
}

}  // extern "C"

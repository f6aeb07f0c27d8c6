// Norms of query and key heads, the rotation by their positions, and the rows' way out: queries
// to a tensor, keys and values into a paged cache (sdv_qk_norm_rope); the angles per position
// (sdv_rope_steps).
//
// Per head of `dim` elements: y = x / sqrt(mean x^2 + eps) w; then its first rot_dim elements in
// pairs (a, b) at angle phi: (A (a cos phi - b sin phi), A (b cos phi + a sin phi)).  phi of
// position p and pair i is 2 pi frac(p step_i / 2^64): the 64-bit product p step_i wraps around
// whole turns, so the angle of any position is exact to 2^-32 turns where p * frequency in 32 bits
// would have lost 2^-24 of hundreds of turns.
//
// A warp per token and part of its heads; a head takes dim / 8 lanes of eight elements each.
// cos and sin of a lane's eight elements are computed once a token and serve all heads.
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

enum RopeForm { kRopeNone, kRopePairs, kRopeHalf, kRopeHalfOdd };

constexpr int kRopeThreads = 128;
constexpr int kRopeAhead = 4;  // heads loaded before the first is used

template <typename T>
struct Chunk {  // eight elements as they lie
  uint4 x;
  __device__ __forceinline__ void load(const T* p) { x = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void floats(float* f) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = unpack16<T>(w[i]);
      f[2 * i] = y.x;
      f[2 * i + 1] = y.y;
    }
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void floats(float* f) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

// Signed turns of position p at a step of 2^-64 turns, doubled: half turns in [-1, 1).
__device__ __forceinline__ float half_turns(int p, unsigned long long step) {
  return (float)(int)((step * (unsigned long long)p) >> 32) * 0x1p-31f;
}

template <typename TI, typename T, int FORM>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a) {
  __shared__ float exchange[FORM == kRopeHalfOdd ? kRopeThreads * 8 : 1];
  const int lane = threadIdx.x & 31;
  const int L = a.lanes, c = lane & (L - 1), sub = lane / L, heads_at_once = 32 / L;
  const int e0 = c * 8, half = a.rot / 2;
  const bool mine = e0 < a.dim;
  const long long warp = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const long long warps = (long long)gridDim.x * (kRopeThreads / 32);
  griddep_wait();
  griddep_launch_dependents();
  const int q_heads = a.q_heads, kv = a.kv_heads, all = q_heads + 2 * kv;
  for (long long item = warp; item < a.tokens * a.parts; item += warps) {
    const long long t = item / a.parts;
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
    // the rotation of this lane's elements
    float cs[8], sn[8];
    bool turned = false;
    if constexpr (FORM != kRopeNone) {
      turned = mine && e0 < a.rot;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int el = e0 + e;
        const bool in = el < a.rot;
        const int i = FORM == kRopePairs ? el / 2 : el < half ? el : el - half;
        if (FORM == kRopePairs && (e & 1)) {
          cs[e] = cs[e - 1];
          sn[e] = -sn[e - 1];
          continue;
        }
        float s = 0.f, co = 1.f;
        if (in) {
          sincospif(half_turns(pos, __ldg(a.steps + i)), &s, &co);
          s *= a.amplitude;
          co *= a.amplitude;
        }
        // y = x cos + partner sn: the first of a pair takes - sin, the second + sin
        cs[e] = co;
        sn[e] = FORM == kRopePairs || el < half ? -s : s;
      }
    }
    for (int hb = h0; hb < h1; hb += heads_at_once * kRopeAhead) {
      Chunk<TI> raw[kRopeAhead];
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        const int h = hb + u * heads_at_once + sub;
        if (!mine || h >= h1) continue;
        const TI* const src = h < q_heads ? static_cast<const TI*>(a.q) + t * a.q_stride + (long long)h * a.dim
                              : h < q_heads + kv
                                  ? static_cast<const TI*>(a.k) + t * a.k_stride + (long long)(h - q_heads) * a.dim
                                  : static_cast<const TI*>(a.v) + t * a.v_stride + (long long)(h - q_heads - kv) * a.dim;
        raw[u].load(src + e0);
      }
#pragma unroll
      for (int u = 0; u < kRopeAhead; ++u) {
        const int h = hb + u * heads_at_once + sub;
        if (hb + u * heads_at_once >= h1) break;  // of every lane
        const bool live = mine && h < h1, value = h >= q_heads + kv;
        float x[8];
        if (live) {
          raw[u].floats(x);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
        }
        const float* const w = h < q_heads ? a.q_weight : a.k_weight;
        // (the sum's shuffles are for all lanes)
        if (a.q_weight != nullptr || a.k_weight != nullptr) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
          for (int off = L / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          if (w != nullptr && live && !value) {
            const float r = 1.f / sqrtf(sum / (float)a.dim + a.eps);
            const float4 wa = __ldg(reinterpret_cast<const float4*>(w + e0)), wb = __ldg(reinterpret_cast<const float4*>(w + e0) + 1);
            const float ws[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * r * ws[e];
          }
        }
        if constexpr (FORM != kRopeNone) {
          float other[8];
          if constexpr (FORM == kRopePairs) {
#pragma unroll
            for (int e = 0; e < 8; ++e) other[e] = x[e ^ 1];
          } else if constexpr (FORM == kRopeHalf) {
            const int from = lane - c + (e0 < half ? c + half / 8 : c - half / 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) other[e] = __shfl_sync(0xffffffffu, x[e], from & 31);
          } else {
            float* const mem = exchange + (threadIdx.x - c) * 8;  // the head's elements
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) mem[e0 + e] = x[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int el = e0 + e;
              other[e] = el < half ? mem[el + half] : el < a.rot ? mem[el - half] : 0.f;
            }
          }
          if (turned && !value) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e0 + e < a.rot) x[e] = fmaf(other[e], sn[e], x[e] * cs[e]);
          }
        }
        if (!live) continue;
        T* dst;
        if (h < q_heads) dst = static_cast<T*>(a.q_out) + (t * q_heads + h) * a.dim;
        else if (slot < 0) continue;
        else if (!value) dst = static_cast<T*>(a.ck) + row + (long long)(h - q_heads) * a.page * a.dim;
        else dst = static_cast<T*>(a.cv) + row + (long long)(h - q_heads - kv) * a.page * a.dim;
        *reinterpret_cast<uint4*>(dst + e0) = make_uint4(pack16<T>(x[0], x[1]), pack16<T>(x[2], x[3]),
                                                         pack16<T>(x[4], x[5]), pack16<T>(x[6], x[7]));
      }
    }
  }
}

template <typename TI, typename T>
cudaError_t rope_launch(int form, const RopeArgs& a, int blocks, cudaStream_t st) {
  auto kernel = form == kRopeNone    ? qk_norm_rope_kernel<TI, T, kRopeNone>
                : form == kRopePairs ? qk_norm_rope_kernel<TI, T, kRopePairs>
                : form == kRopeHalf  ? qk_norm_rope_kernel<TI, T, kRopeHalf>
                                     : qk_norm_rope_kernel<TI, T, kRopeHalfOdd>;
  return launch_pdl(kernel, dim3(blocks), dim3(kRopeThreads), 0, st, a);
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
  const int blocks = (int)(want < 12ll * sms ? want : 12ll * sms);
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

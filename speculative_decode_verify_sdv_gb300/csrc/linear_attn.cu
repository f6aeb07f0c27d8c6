// Linear attention with a decay for each head (sdv_linear_attn): the recurrent
// kernel and the entry points.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "linear_args.h"
#include "mixing.h"
#include "sdv.h"
#include "sdv_device.cuh"

namespace sdv {

namespace {

__device__ __forceinline__ void lin_round(float x, __half& y) { y = __float2half_rn(x); }
__device__ __forceinline__ void lin_round(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// Recurrent form: the state's definition, token by token.  A CTA holds 128 value
// columns of one head's state in registers: lane l the columns 4l .. 4l+3, warp w
// the key rows w * R .. w * R + R - 1, so a state row of the CTA is one 512-byte
// access per warp and a thread has R 16-byte loads in flight.  Reading and writing
// the state bounds it for one token (4096 heads of 128 x 128: 540 MB in 95.9 us,
// 5.6 TB/s; 32 heads: 9.9 us, the call itself); the outputs' sum over the key rows
// crosses the warps through shared memory.  At 64 value columns half of each warp has no
// column: 4096 heads of 128 x 64 take 69 us, 3.9 TB/s, where 64 x 128 takes 50, 5.4 TB/s;
// with 256 key rows 4.7 TB/s.
constexpr int kRecWarps = 8;
constexpr int kRecTokens = 8;  // tokens staged at once

// With `repair` it recomputes the heads noted there.
template <typename T, int R>
__global__ void __launch_bounds__(32 * kRecWarps) linear_recurrent_kernel(const LinArgs a) {
  __shared__ float qs[kRecTokens][kRecWarps * R], ks[kRecTokens][kRecWarps * R];
  __shared__ float4 vs[kRecTokens][32];
  __shared__ float ds[kRecTokens];
  __shared__ float4 red[kRecWarps][32];
  griddep_wait();
  if (a.repair != nullptr) {  // (one block a head: Dv is at most 128 here)
    if (a.repair[(long long)blockIdx.z * a.H + blockIdx.y] == 0) return;
  }
  const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hqk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 128 + lane * 4;  // value columns
  const bool col = c < a.Dv;
  const int r0 = warp * R;
  const int n = lin_tokens(a, b);
  const long long sbase = ((long long)b * a.H + h) * a.Dk * a.Dv + c;
  float4 m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.s_in != nullptr && col && r0 + r < a.Dk)
      m[r] = *reinterpret_cast<const float4*>(a.s_in + sbase + (long long)(r0 + r) * a.Dv);
  }
  const T* const q = static_cast<const T*>(a.q);
  const T* const k = static_cast<const T*>(a.k);
  const T* const v = static_cast<const T*>(a.v);
  T* const o = static_cast<T*>(a.o);
  for (int t0 = 0; t0 < n; t0 += kRecTokens) {
    const int nt = min(kRecTokens, n - t0);
    __syncthreads();
    for (int e = threadIdx.x; e < nt * kRecWarps * R; e += blockDim.x) {
      const int t = e / (kRecWarps * R), d = e % (kRecWarps * R);
      const long long row = (long long)b * a.T + t0 + t;
      ks[t][d] = d < a.Dk ? lin_float(k[row * a.k_stride + hk * a.Dk + d]) : 0.f;
      qs[t][d] = d < a.Dk && o != nullptr ? lin_float(q[row * a.q_stride + hk * a.Dk + d]) : 0.f;
    }
    for (int e = threadIdx.x; e < nt * 128; e += blockDim.x) {
      const int t = e >> 7, d = e & 127;
      const long long row = (long long)b * a.T + t0 + t;
      reinterpret_cast<float*>(vs[t])[d] =
          blockIdx.x * 128 + d < a.Dv ? lin_float(v[row * a.v_stride + h * a.Dv + blockIdx.x * 128 + d]) : 0.f;
    }
    if (threadIdx.x < nt) ds[threadIdx.x] = expf(lin_decay(a, b, t0 + threadIdx.x, h));
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float f = ds[t];
      const float4 x = vs[t][lane];
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      // a decay of exactly 0 drops the state whatever it holds
      if (f == 0.f) {
#pragma unroll
        for (int r = 0; r < R; ++r) m[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float kk = ks[t][r0 + r], qq = qs[t][r0 + r];
        m[r].x = fmaf(kk, x.x, m[r].x * f);
        m[r].y = fmaf(kk, x.y, m[r].y * f);
        m[r].z = fmaf(kk, x.z, m[r].z * f);
        m[r].w = fmaf(kk, x.w, m[r].w * f);
        y.x = fmaf(qq, m[r].x, y.x);
        y.y = fmaf(qq, m[r].y, y.y);
        y.z = fmaf(qq, m[r].z, y.z);
        y.w = fmaf(qq, m[r].w, y.w);
      }
      if (o == nullptr) continue;
      red[warp][lane] = y;
      __syncthreads();
      if (threadIdx.x < 128 && blockIdx.x * 128 + threadIdx.x < a.Dv) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kRecWarps; ++w) s += reinterpret_cast<const float*>(red[w])[threadIdx.x];
        T r;
        lin_round(s * a.scale, r);
        o[(((long long)b * a.T + t0 + t) * a.H + h) * a.Dv + blockIdx.x * 128 + threadIdx.x] = r;
      }
      __syncthreads();
    }
  }
  if (o != nullptr && col) {
    T z;
    lin_round(0.f, z);
    for (int t = n + warp; t < a.T; t += kRecWarps)
      for (int i = 0; i < 4; ++i) o[(((long long)b * a.T + t) * a.H + h) * a.Dv + c + i] = z;
  }
  if (a.s_out != nullptr && col) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r0 + r < a.Dk) *reinterpret_cast<float4*>(a.s_out + sbase + (long long)(r0 + r) * a.Dv) = m[r];
  }
}

template <typename T>
cudaError_t launch_recurrent(const LinArgs& a, cudaStream_t st) {
  const dim3 grid((a.Dv + 127) / 128, a.H, a.B), block(32 * kRecWarps);
  if (a.Dk <= 64) return launch_pdl(linear_recurrent_kernel<T, 8>, grid, block, 0, st, a);
  if (a.Dk <= 128) return launch_pdl(linear_recurrent_kernel<T, 16>, grid, block, 0, st, a);
  return launch_pdl(linear_recurrent_kernel<T, 32>, grid, block, 0, st, a);
}

bool lin_shape(int B, int T, int H, int Dk, int Dv) {
  return B >= 1 && T >= 1 && H >= 1 && Dk >= 8 && Dk % 8 == 0 && Dv >= 8 && Dv % 8 == 0;
}

// The chunked form's workspace: notes of heads to repair, the CTAs' local states.
size_t lin_notes(int B, int H) { return round_256((size_t)B * H * 4); }
size_t lin_parts(int ctas, int Dk, int Dv) { return (size_t)ctas * (sizeof(LinPart) + 2 * (size_t)Dk * Dv * 4); }

// Which form (head sizes of 64 and 128; others are the recurrent form's, as one token is).
// The recurrent form's time grows with the tokens, the window form's with the state: the
// tokens from which the latter is the faster one depend on what a call computes and on the
// state's proportions.  GPU us, recurrent against window form, 512 heads and 4096 of them,
// fp16 (bf16 is within 5 %):
//   128 x 128  both     6: 25.6 to 29.1, 169 to 190   8: 29.9 to 29.9, 197 to 194
//              outputs  3: 14.5 to 15.2,  94 to 87    4: 15.8 to 15.3, 103 to 88
//              state    2: 15.7 to 15.8, 100 to 94    4: 18.9 to 16.5, 122 to 98
//   128 x 64   both     4: 16.6 to 18.1, 108 to 100   5: 19.8 to 18.3, 129 to 101
//              outputs  2:  9.8 to 9.5,   61 to 47
//              state    2: 11.0 to 10.1,  69 to 50
//   64 x 64    both     6: 11.1 to 12.1,  66 to 61    8: 12.8 to 12.5,  78 to 62
//              outputs  3:  6.8 to 7.1,   38 to 32    4:  7.5 to 7.1,   43 to 32
//              state    2:  6.2 to 6.1,   34 to 28
//   64 x 128   both    10: 17.9 to 21.5, 106 to 132  13: 21.3 to 22.3, 126 to 136
//              outputs  6: 10.9 to 12.3,  65 to 67    8: 12.7 to 12.2,  76 to 67
//              state    2:  8.8 to 9.8,   50 to 51    4:  9.9 to 10.0,  58 to 53
// Window against chunked form at 32 tokens, the window form's most (128 x 128, 512 heads and
// 32): 48.8 to 59.0 and 18.1 to 23.2.
int lin_window_from(int Dk, int Dv, bool outputs, bool state) {
  if (outputs && state) return Dv < Dk ? 5 : Dv == Dk ? 7 : 12;
  if (outputs) return Dv < Dk ? 2 : Dv == Dk ? 4 : 7;
  return Dv <= Dk ? 2 : 3;
}
bool lin_window(int T, int Dk, int Dv, bool outputs, bool state) {
  return linear_tc_takes(Dk, Dv) && T >= lin_window_from(Dk, Dv, outputs, state) && T <= kLinWindow;
}
bool lin_chunked(int B, int T, int H, int Dk, int Dv) {
  // the tensor maps' coordinates and the split's arithmetic are 32-bit
  const long long chunks = (long long)B * H * ((T + kLinChunk - 1) / kLinChunk);
  return linear_tc_takes(Dk, Dv) && T > kLinWindow && (long long)B * T <= INT32_MAX - 2 * kLinChunk &&
         chunks <= INT32_MAX / 512;
}

bool lin_limits(int B, int H, int Dk, int Dv) { return B <= 65535 && H <= 4096 && Dk <= 256 && Dv <= 256; }

bool lin_rows(const void* p, long long stride, int heads, int dim) {
  return p != nullptr && is_aligned16(p) && stride % 8 == 0 && stride >= (long long)heads * dim;
}

}  // namespace

}  // namespace sdv

extern "C" {

size_t sdv_linear_attn_workspace_bytes(int32_t B, int32_t T, int32_t H, int32_t Dk, int32_t Dv) {
  if (!sdv::lin_shape(B, T, H, Dk, Dv) || !sdv::lin_limits(B, H, Dk, Dv)) return 0;
  // (also where a prompt is too long for the chunked form: shorter ones fit its workspace)
  if (!sdv::linear_tc_takes(Dk, Dv) || T <= sdv::kLinWindow) return sdv::kHeaderBytes;
  const int sms = sdv::sm_count();
  return sdv::kHeaderBytes + sdv::lin_notes(B, H) + sdv::lin_parts(sms > 0 ? sms : 256, Dk, Dv);
}

sdv_status sdv_linear_attn(int32_t dtype, const void* q_or_null, const void* k, const void* v, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const float* log_decay, int32_t decay_per_token,
                           float scale, int32_t B, int32_t T, int32_t H, int32_t Hqk, int32_t Dk, int32_t Dv,
                           const int32_t* n_tokens_or_null, const float* state_in_or_null, float* state_out_or_null,
                           void* o_or_null, void* ws, size_t ws_bytes, sdv_stream_t stream) {
  using namespace sdv;
  if (dtype != SDV_F16 && dtype != SDV_BF16) return SDV_ERR_INVALID_ARG;
  if (!lin_shape(B, T, H, Dk, Dv) || Hqk < 1 || H % Hqk != 0) return SDV_ERR_INVALID_ARG;
  if (!lin_rows(k, k_stride, Hqk, Dk) || !lin_rows(v, v_stride, H, Dv)) return SDV_ERR_INVALID_ARG;
  if (o_or_null != nullptr && !lin_rows(q_or_null, q_stride, Hqk, Dk)) return SDV_ERR_INVALID_ARG;
  if (o_or_null == nullptr && state_out_or_null == nullptr) return SDV_ERR_INVALID_ARG;
  if (log_decay == nullptr || (reinterpret_cast<uintptr_t>(log_decay) & 3u) ||
      (reinterpret_cast<uintptr_t>(n_tokens_or_null) & 3u) || (decay_per_token != 0 && decay_per_token != 1))
    return SDV_ERR_INVALID_ARG;
  if (!is_aligned16(o_or_null) || !is_aligned16(state_in_or_null) || !is_aligned16(state_out_or_null) ||
      !std::isfinite(scale))
    return SDV_ERR_INVALID_ARG;
  if (!lin_limits(B, H, Dk, Dv)) return SDV_ERR_UNSUPPORTED;
  const bool chunked = lin_chunked(B, T, H, Dk, Dv);
  const size_t need = chunked ? sdv_linear_attn_workspace_bytes(B, T, H, Dk, Dv) : kHeaderBytes;
  if (ws == nullptr || !is_aligned16(ws) || ws_bytes < need) return SDV_ERR_WORKSPACE;
  LinArgs a{};
  a.q = q_or_null;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.g = log_decay;
  a.g_token = decay_per_token;
  a.scale = scale;
  a.B = B;
  a.T = T;
  a.H = H;
  a.Hqk = Hqk;
  a.Dk = Dk;
  a.Dv = Dv;
  a.n_tokens = n_tokens_or_null;
  a.s_in = state_in_or_null;
  a.s_out = state_out_or_null;
  a.o = o_or_null;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (lin_window(T, Dk, Dv, a.o != nullptr, a.s_out != nullptr)) return status_of(launch_linear_window(dtype, a, st));
  if (chunked) {
    a.ctas = sm_count();
    if (a.ctas <= 0) return SDV_ERR_CUDA;
    char* const w8 = static_cast<char*>(ws);
    a.status = reinterpret_cast<int*>(w8);
    a.fault = debug_fault();
    a.repair = reinterpret_cast<int*>(w8 + kHeaderBytes);
    a.part = reinterpret_cast<float*>(w8 + kHeaderBytes + lin_notes(B, H));
    a.part_in = a.part + (size_t)a.ctas * Dk * Dv;
    a.parts = reinterpret_cast<LinPart*>(a.part_in + (size_t)a.ctas * Dk * Dv);
    const cudaError_t e = launch_linear_tc(dtype, a, st);
    if (e != cudaSuccess) return status_of(e);
  }
  return status_of(dtype == SDV_F16 ? launch_recurrent<__half>(a, st) : launch_recurrent<__nv_bfloat16>(a, st));
}

}  // extern "C"

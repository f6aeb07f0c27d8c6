// Arguments of the linear-attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mixing.h"

namespace sdv {

// A sum of log2 decays as a pair of floats (48 bits).
struct DecaySum {
  float hi = 0.f, lo = 0.f;
#ifdef __CUDACC__
  // log2 of e^x, x at most 0; -1e4 (a decay of 0 in fp32) for anything below; NaN stays.
  static __device__ __forceinline__ DecaySum log2_of(float x) {
    constexpr float c = 1.4426950216293335f, cl = 1.925963033500583e-08f;  // log2 e = c + cl
    x = x < -1e4f ? -1e4f : x;
    const float h = __fmul_rn(x, c);
    return DecaySum{h, fmaf(x, cl, fmaf(x, c, -h))};
  }
  // The exact sum of the high parts (two-sum), the low parts beside it.
  __device__ __forceinline__ void add(const DecaySum& o) {
    const float s = __fadd_rn(hi, o.hi), b = __fadd_rn(s, -hi);
    const float e = __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(o.hi, -b));
    const float l = __fadd_rn(__fadd_rn(lo, o.lo), e);
    hi = __fadd_rn(s, l);
    lo = __fadd_rn(l, -__fadd_rn(hi, -s));
  }
  __device__ __forceinline__ float minus(const DecaySum& o) const { return (hi - o.hi) + (lo - o.lo); }
#endif
};

struct LinPart {
  DecaySum decay;  // its log2 decay
  int bad;         // a key or value is not finite
  int pad;
};

struct LinArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const float* g;
  int g_token;             // 1: [B][T][H], 0: [H]
  float scale;
  int B, T, H, Hqk, Dk, Dv;
  const int32_t* n_tokens;
  const float* s_in;
  float* s_out;
  void* o;
  // chunked form: what the first launch leaves of each CTA, heads with keys or values that
  // are not finite (recomputed by the recurrent kernel), status
  float* part;             // [CTAs][Dv / 4][Dk][4] local states
  float* part_in;          // [CTAs][Dk][Dv] the given state of a head that starts in the CTA and goes on
  LinPart* parts;          // [CTAs]
  int* repair;             // [B][H]
  int* status;
  int ctas;
  int pass;                // 0: local states, 1: outputs and final states
  DebugFault fault;        // the timeout path's test hook: a chunk whose keys are never asked for
};

struct LinMaps {
  CUtensorMap q, k, v;
};

constexpr int kLinChunk = 128;   // tokens of a chunk
constexpr int kLinRuns = 16;     // CTAs are 16 times the heads of all sequences at most (a long
                                 // sequence among short ones may have more of them than that)

constexpr int kLinWindow = 32;   // tokens of the window form at most

// Whether the chunked and the window form have an instance for the head sizes.
inline bool linear_tc_takes(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }
cudaError_t launch_linear_window(int dtype, const LinArgs& a, cudaStream_t st);
cudaError_t launch_linear_tc(int dtype, const LinArgs& a, cudaStream_t st);
cudaError_t linear_tc_f16(const LinMaps& m, const LinArgs& a, cudaStream_t st);
cudaError_t linear_tc_bf16(const LinMaps& m, const LinArgs& a, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ int lin_tokens(const LinArgs& a, int b) {
  return a.n_tokens != nullptr ? min(max(__ldg(a.n_tokens + b), 0), a.T) : a.T;
}

__device__ __forceinline__ float lin_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float lin_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// The log decay of token t, head h: at most 0 (NaN stays NaN).
__device__ __forceinline__ float lin_clamp_decay(float g) { return g > 0.f ? 0.f : g; }
__device__ __forceinline__ float lin_decay(const LinArgs& a, int b, int t, int h) {
  return lin_clamp_decay(__ldg(a.g + (a.g_token ? ((long long)b * a.T + t) * a.H + h : h)));
}
#endif

}  // namespace sdv

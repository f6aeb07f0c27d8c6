// Arguments of the linear-attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace sdv {

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
  // chunked form: a CTA's local state and its log2 decay, heads whose values are not
  // finite (recomputed by the recurrent kernel), status
  float* part;             // [CTAs][Dk][Dv]
  double* part_decay;      // [CTAs]
  int* repair;             // [B][H]
  int* status;
  int ctas;
  int pass;                // 0: local states, 1: outputs and final states
};

struct LinMaps {
  CUtensorMap q, k, v;
};

constexpr int kLinChunk = 128;   // tokens of a chunk
constexpr int kLinRuns = 16;     // CTAs that share one head at most

// Whether the chunked form has an instance for the head sizes.
inline bool linear_tc_takes(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }
cudaError_t launch_linear_tc(int dtype, const LinArgs& a, cudaStream_t st);
cudaError_t linear_tc_f16(const LinMaps& m, const LinArgs& a, cudaStream_t st);
cudaError_t linear_tc_bf16(const LinMaps& m, const LinArgs& a, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ int lin_tokens(const LinArgs& a, int b) {
  return a.n_tokens != nullptr ? min(max(__ldg(a.n_tokens + b), 0), a.T) : a.T;
}

// The log decay of token t, head h: at most 0 (NaN stays NaN).
__device__ __forceinline__ float lin_decay(const LinArgs& a, int b, int t, int h) {
  const float g = __ldg(a.g + (a.g_token ? ((long long)b * a.T + t) * a.H + h : h));
  return g > 0.f ? 0.f : g;
}
#endif

}  // namespace sdv

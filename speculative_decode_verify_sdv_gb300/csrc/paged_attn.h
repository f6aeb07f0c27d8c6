// The paged attention behind its checks, for the entry points that build on it.
#pragma once

#include <cuda_runtime.h>

#include "attn_sched.cuh"
#include "sdv.h"

namespace sdv {

// The checks of sdv_paged_attn, those of its workspace excepted (SDV_OK where they pass).
sdv_status attn_check(const sdv_kvcache* cache, const void* q, int64_t q_stride, int32_t B, int32_t S, int32_t Hq,
                      const int32_t* ctx, const int32_t* n_rows, const uint32_t* mask, float scale, const void* out,
                      const float* lse);

// Workspace bytes of calls of up to S rows on a GPU of `sms` SMs (0: not known); 0 for invalid arguments.
size_t attn_bytes(int B, int S, int Hq, int heads, int dim, int sms);

// A checked call's arguments, without outputs and workspace.
AttnArgs attn_args(const sdv_kvcache* cache, const void* q, int64_t q_stride, int32_t B, int32_t S, int32_t Hq,
                   const int32_t* ctx, const int32_t* n_rows, const uint32_t* mask, float scale);

// Its launches.
sdv_status attn_run(const sdv_kvcache* cache, AttnArgs a, void* ws, cudaStream_t st);

}  // namespace sdv

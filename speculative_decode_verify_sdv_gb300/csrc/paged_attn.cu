// A paged key/value cache and the attention of a verify window over it: the
// append, the CUDA-core attention for shapes the tensor-core kernel does not take,
// the join of split units, and the entry points (sdv_kv_append, sdv_paged_attn).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "attn_sched.cuh"
#include "attn_tc.h"
#include "host_util.h"
#include "mixing.h"
#include "paged_attn.h"
#include "sdv.h"
#include "sdv_device.cuh"

namespace sdv {

namespace {

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float x, __half& y) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// ---- append ---------------------------------------------------------------------------

struct AppendArgs {
  const uint4 *k, *v;         // 16-byte units throughout
  long long k_stride, v_stride;
  uint4 *ck, *cv;
  const int32_t *table, *ctx, *n_rows;
  int T, heads, vec, n_pages, page, max_pages;  // vec: units per head row
  int* status;
};

// Row (b, t) of one tensor per warp: a copy of heads * vec 16-byte units, units
// of one head contiguous on both sides.  The copy bounds it: 148 MB read and written for
// eight prompts of up to 4096 rows in 26.1 us, 5.7 TB/s; one row is the call itself, 8.6 us.
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  griddep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int n = a.n_rows != nullptr ? min(max(__ldg(a.n_rows + b), 0), a.T) : a.T;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= n) return;
  const long long pos = (long long)__ldg(a.ctx + b) + t;
  const long long slot = pos / a.page;
  int id = -1;
  if (pos >= 0 && slot < a.max_pages) id = __ldg(a.table + (size_t)b * a.max_pages + slot);
  if (id < 0 || id >= a.n_pages) {
    if (lane == 0 && a.status != nullptr) atomicOr(a.status, kDevErrIndex);
    return;
  }
  const bool values = blockIdx.z != 0;
  const uint4* const src = (values ? a.v : a.k) + ((long long)b * a.T + t) * (values ? a.v_stride : a.k_stride);
  uint4* const dst = (values ? a.cv : a.ck) + ((long long)id * a.heads * a.page + pos % a.page) * a.vec;
  for (int u = lane; u < a.heads * a.vec; u += 32) {
    const int h = u / a.vec, c = u % a.vec;
    dst[(long long)h * a.page * a.vec + c] = __ldg(src + u);
  }
}

// ---- CUDA-core attention --------------------------------------------------------------

// The sum of what is not finite in column d of the values that a row sees among positions
// from .. to - 1 (`word`: its window positions).
template <typename T>
__device__ __noinline__ float attn_odd_sum(const AttnArgs& a, int b, int h, int ctx, int from, int to, uint32_t word,
                                           int d) {
  float sum = 0.f;
  for (int p = from; p < to; ++p) {
    if (p >= ctx && !(word >> (p - ctx) & 1u)) continue;
    const int id = __ldg(a.table + (size_t)b * a.max_pages + p / a.page);
    if (id < 0 || id >= a.n_pages) continue;
    const float x = to_float(static_cast<const T*>(a.v)[(((long long)id * a.Hkv + h) * a.page + p % a.page) * a.D + d]);
    if (!(fabsf(x) < INFINITY)) sum += x;
  }
  return sum;
}

// One CTA walks its range of tiles (attn_sched.cuh) with 8 query rows per tile.
// Positions come 32 at a time through shared memory; a warp holds the running
// maximum and sum of two rows, each thread the outputs of up to two columns of
// all rows.  It is the form for head sizes and page sizes outside the tensor-core
// kernel's; a position a row does not see has weight -0 and is skipped, so nothing its
// values hold reaches the row.  A weight of +0 times an infinity makes the sum NaN, and
// an output that is not finite is then told from the values themselves.  Its arithmetic
// bounds it: 8 sequences of 4000 positions, 32 heads over 8 of 96: 374 us for one row each
// (0.3 TB/s of cache), 2.7 ms for 17; the tensor-core kernel at heads of 128 takes 30 and 43.
template <typename T>
__global__ void __launch_bounds__(128) attn_simple_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int R = kAttnSimpleRows, P = kAttnSimpleTile;
  extern __shared__ float sm[];
  const int D = a.D, ld = D + 1;
  float* const qs = sm;                    // [R][D]
  float* const ks = qs + R * D;            // [P][D + 1]
  float* const vs = ks + P * ld;           // [P][D]
  float* const ps = vs + P * D;            // [R][P] scores, then weights
  float* const al = ps + R * P;            // [R] factor of the old sum and output
  __shared__ uint32_t words[R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  AttnWalk w;
  if (!w.start(a, blockIdx.x, lane)) return;
  while (w.more()) {
    const int count = w.segment();
    const int h = w.unit / a.row_tiles, r0 = (w.unit % a.row_tiles) * a.row_tile;
    const int nr = min(a.row_tile, a.rows - r0);
    const int total = w.seq.ctx + w.seq.n;
    if (w.seq.bad && tid == 0) atomicOr(a.status, kDevErrIndex);
    __syncthreads();
    for (int e = tid; e < R * D; e += 128) {
      const int r = e / D, row = r0 + r;
      float x = 0.f;
      if (r < nr && row / a.G < w.seq.n) {
        const long long at = ((long long)w.b * a.S + row / a.G) * a.q_stride + (h * a.G + row % a.G) * D + e % D;
        x = to_float(static_cast<const T*>(a.q)[at]);
      }
      qs[e] = x;
    }
    if (tid < R) words[tid] = tid < nr ? attn_word(a, w.b, (r0 + tid) / a.G, w.seq.n) : 0u;
    float o[2][R], m[2], l[2];
#pragma unroll
    for (int r = 0; r < R; ++r) o[0][r] = o[1][r] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    for (int t = w.tile; t < w.tile + count; ++t) {
      const int p0 = t * P;
      __syncthreads();
      for (int j = warp; j < P; j += 4) {  // a position per warp
        const int p = p0 + j;
        int id = -1;
        if (p < total) {
          id = __ldg(a.table + (size_t)w.b * a.max_pages + p / a.page);
          if (id < 0 || id >= a.n_pages) {
            if (lane == 0) atomicOr(a.status, kDevErrIndex);
            id = -1;
          }
        }
        const long long at = (((long long)id * a.Hkv + h) * a.page + p % a.page) * D;
        for (int d = lane; d < D; d += 32) {
          ks[j * ld + d] = id < 0 ? __int_as_float(0x7fc00000) : to_float(static_cast<const T*>(a.k)[at + d]);
          vs[j * D + d] = id < 0 ? 0.f : to_float(static_cast<const T*>(a.v)[at + d]);
        }
        if (lane == 0) ps[j] = id < 0 ? 1.f : 0.f;  // absent
      }
      __syncthreads();
      const bool absent = ps[lane] != 0.f;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // warp's rows 2 warp + i, lane = position
        const int r = 2 * warp + i, p = p0 + lane;
        const int row = r0 + r;
        bool see = !absent && p < total && r < nr && row / a.G < w.seq.n;
        if (see && p >= w.seq.ctx) see = (words[r] >> (p - w.seq.ctx)) & 1u;
        float s = -INFINITY;
        if (see) {
          s = 0.f;
#pragma unroll 4
          for (int d = 0; d < D; ++d) s = fmaf(qs[r * D + d], ks[lane * ld + d], s);
          s *= a.scale_log2;
        }
        float mx = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float e = see ? exp2f(s - ref) : -0.f;
        const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - ref);
        float sum = e;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[i] = l[i] * f + sum;
        m[i] = mn;
        ps[r * P + lane] = e;
        if (lane == 0) al[r] = f;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = tid + 128 * c;
        if (d >= D) continue;
#pragma unroll
        for (int r = 0; r < R; ++r) o[c][r] *= al[r];
#pragma unroll 2
        for (int j = 0; j < P; ++j) {
          const float x = vs[j * D + d];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float e = ps[r * P + j];
            if (__float_as_uint(e) != 0x80000000u) o[c][r] = fmaf(e, x, o[c][r]);
          }
        }
      }
    }
    __syncthreads();
    if (lane < 2) {  // the rows' statistics for the columns' threads
      ps[2 * warp + lane] = lane == 0 ? m[0] : m[1];
      al[2 * warp + lane] = lane == 0 ? l[0] : l[1];
    }
    __syncthreads();
    const bool starts = w.tile == 0, ends = w.tile + count == w.seq.tiles;
    const size_t slot = 2 * (size_t)blockIdx.x + (starts ? 1 : 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= nr) break;
      const int row = r0 + r;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = tid + 128 * c;
        if (d < D && !(fabsf(o[c][r]) < INFINITY) && al[r] > 0.f) {
          const float odd = attn_odd_sum<T>(a, w.b, h, w.seq.ctx, w.tile * P, min((w.tile + count) * P, total), words[r], d);
          if (!(fabsf(odd) < INFINITY)) o[c][r] = odd;
        }
      }
      if (starts && ends) {
        const long long orow = ((long long)w.b * a.S + row / a.G) * a.Hq + h * a.G + row % a.G;
        const float inv = al[r] > 0.f ? 1.f / al[r] : (al[r] == 0.f ? 0.f : al[r]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int d = tid + 128 * c;
          if (d >= D) continue;
          const float y = al[r] == 0.f ? 0.f : o[c][r] * inv;
          if (a.out32 != nullptr) a.out32[orow * D + d] = y;
          else from_float(y, static_cast<T*>(a.out)[orow * D + d]);
        }
        if (tid == 0 && a.lse != nullptr)
          a.lse[orow] = al[r] == 0.f ? -INFINITY : (ps[r] + log2f(al[r])) * 0.6931471805599453f;
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int d = tid + 128 * c;
          if (d < D) a.part_o[((slot * (D / 4) + d / 4) * a.row_tile + r) * 4 + d % 4] = o[c][r];
        }
        if (tid == 0) {
          a.part_ml[(slot * a.row_tile + r) * 2] = ps[r];
          a.part_ml[(slot * a.row_tile + r) * 2 + 1] = al[r];
        }
      }
    }
    w.advance(a, count);
  }
}

// ---- join -----------------------------------------------------------------------------

// Adds the partials of the units that several CTAs shared:
//   M = max m_j, out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j.
// A thread per row and four columns (a unit's rows side by side, as the partials
// lie) and quarter of the partials, eight loads in flight each: the partials sit in
// L2, so latency is what there is to hide.  The order of the sums is fixed by the
// split.  48 units of 96 rows x 128 columns, four partials each: 15 us with the partials
// in memory; fewer blocks that loop over their items took as long.
constexpr int kJoinItems = 64, kJoinParts = 4;

template <typename T>
__global__ void __launch_bounds__(kJoinItems* kJoinParts) attn_join_kernel(const AttnArgs a, bool by_cta) {
  __shared__ float4 so[kJoinParts][kJoinItems];
  __shared__ float2 sml[kJoinParts][kJoinItems];
  const int lane = threadIdx.x & 31;
  griddep_wait();
  int unit, c0, c1;
  AttnWalk w;
  if (by_cta) {
    // the unit that the first tile of a CTA's range lies inside, by its second sharer
    const int c = blockIdx.x + 1;
    const bool some = w.start(a, c, lane);
    if (!some || w.tile == 0) return;
    w.sharers(c0, c1);
    if (c0 != c - 1) return;
    unit = w.unit;
  } else {
    const int units = a.Hkv * a.row_tiles;
    w.b = blockIdx.x / units;
    unit = blockIdx.x % units;
    long long before = 0, all = 0;
    for (int s = lane; s < a.B; s += 32) {
      const int t = attn_seq(a, s).tiles + a.lead;
      all += t;
      if (s < w.b) before += t;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, off);
      before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    const AttnSeq seq = attn_seq(a, w.b);
    const long long total = all * units, first = before * units + (long long)unit * (seq.tiles + a.lead) + a.lead;
    const int live = attn_live_ctas(a.ctas, total);
    c0 = attn_owner(total, live, first);
    c1 = attn_owner(total, live, first + seq.tiles - 1);
    if (c0 == c1) return;
  }
  const int b = w.b;
  const int h = unit / a.row_tiles, r0 = (unit % a.row_tiles) * a.row_tile;
  const int item = threadIdx.x % kJoinItems, part = threadIdx.x / kJoinItems;
  const int e = blockIdx.y * kJoinItems + item, r = e % a.row_tile, d4 = e / a.row_tile;
  const bool mine = d4 < a.D / 4 && r < a.rows - r0;
  AttnSum sum;
  if (mine) {
    const float2* const ml = reinterpret_cast<const float2*>(a.part_ml) + r;
    const float4* const po = reinterpret_cast<const float4*>(a.part_o) + (size_t)d4 * a.row_tile + r;
    const size_t step = (size_t)(a.D / 4) * a.row_tile;
    const int per = (c1 - c0 + kJoinParts) / kJoinParts, from = c0 + part * per, to = min(from + per - 1, c1);
    sum = attn_sum_parts<false>(ml, po, a.row_tile, step, c0, from, to);
    if (!sum.finite()) sum = attn_sum_odd_parts(ml, po, a.row_tile, step, c0, from, to);
  }
  so[part][item] = sum.o;
  sml[part][item] = make_float2(sum.m, sum.l);
  __syncthreads();
  if (part != 0 || !mine) return;
#pragma unroll
  for (int j = 1; j < kJoinParts; ++j) sum.add<true>(sml[j][item].x, sml[j][item].y, so[j][item]);
  const int row = r0 + r;
  const long long orow = ((long long)b * a.S + row / a.G) * a.Hq + h * a.G + row % a.G;
  const bool none = sum.l == 0.f;
  const float inv = none ? 0.f : 1.f / sum.l;
  attn_store4<T>(a, orow * a.D + d4 * 4, none ? 0.f : sum.o.x * inv, none ? 0.f : sum.o.y * inv,
                 none ? 0.f : sum.o.z * inv, none ? 0.f : sum.o.w * inv);
  if (d4 == 0 && a.lse != nullptr) a.lse[orow] = sum.lse();
}

int simple_smem(int D) {
  constexpr int R = kAttnSimpleRows, P = kAttnSimpleTile;
  return (R * D + P * (D + 1) + P * D + R * P + R) * 4;
}

}  // namespace

cudaError_t launch_attn_simple(int dtype, const AttnArgs& a, cudaStream_t st) {
  auto kernel = dtype == SDV_F16 ? attn_simple_kernel<__half> : attn_simple_kernel<__nv_bfloat16>;
  const int smem = simple_smem(a.D);
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.ctas), dim3(128), smem, st, a);
}

cudaError_t launch_attn_join(int dtype, const AttnArgs& a, cudaStream_t st) {
  auto kernel = dtype == SDV_F16 ? attn_join_kernel<__half> : attn_join_kernel<__nv_bfloat16>;
  // blocks for the units, or for the CTAs' ranges, in each of which one shared unit at most begins
  // to be another CTA's: whichever are fewer (2048 units of 20 rows: 92 us by unit, mostly blocks
  // with nothing to do)
  const int units = a.B * a.Hkv * a.row_tiles;
  const bool by_cta = a.ctas <= units;
  return launch_pdl(kernel, dim3(by_cta ? a.ctas - 1 : units, (a.row_tile * (a.D / 4) + kJoinItems - 1) / kJoinItems),
                    dim3(kJoinItems * kJoinParts), 0, st, a, by_cta);
}

}  // namespace sdv

namespace {

using sdv::AttnArgs;

constexpr int kMaxWindow = 32;
constexpr int kMaxDim = 256;
constexpr int kMaxSeqs = 65535;      // a grid dimension of the append
constexpr int kMaxHeads = 4096;
constexpr long long kMaxUnits = 1ll << 30;

bool valid_cache(const sdv_kvcache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->table == nullptr) return false;
  if (c->dtype != SDV_F16 && c->dtype != SDV_BF16) return false;
  if (c->n_pages < 1 || c->heads < 1 || c->page_size < 1 || c->max_pages < 1) return false;
  if (c->dim < 8 || c->dim % 8 != 0) return false;
  return sdv::is_aligned16(c->k) && sdv::is_aligned16(c->v) &&
         (reinterpret_cast<uintptr_t>(c->table) & 3u) == 0;
}

bool valid_rows(const void* p, long long stride, int heads, int dim) {
  return p != nullptr && sdv::is_aligned16(p) && stride % 8 == 0 && stride >= (long long)heads * dim;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Row tiles: the fewest that hold the rows, of equal size.
void set_rows(AttnArgs& a, int most) {
  a.row_tiles = (a.rows + most - 1) / most;
  a.row_tile = (a.rows + a.row_tiles - 1) / a.row_tiles;
}

// The tensor-core kernel's: whole window rows, at most 128 query rows.
void set_window_rows(AttnArgs& a) {
  const int most = a.G < sdv::kAttnTcRows ? sdv::kAttnTcRows / a.G : 1;
  a.row_tiles = (a.S + most - 1) / most;
  a.tile_wrows = (a.S + a.row_tiles - 1) / a.row_tiles;
  a.row_tile = a.tile_wrows * a.G;
}

// Behind the header: (max, sum) partials, output partials.
size_t part_bytes(int ctas, int row_tile, int D) {
  return sdv::round_256((size_t)2 * ctas * row_tile * 8) + sdv::round_256((size_t)2 * ctas * row_tile * D * 4);
}

constexpr int kSimplePerSm = 2;

// What a call of S rows needs on a GPU of `sms` SMs; 0 for invalid arguments.
size_t attn_need(int B, int S, int Hq, int heads, int dim, int sms) {
  if (B < 1 || S < 1 || S > kMaxWindow || heads < 1 || Hq < 1 || Hq % heads != 0 || dim < 8 || dim % 8 != 0 ||
      dim > kMaxDim || heads > kMaxHeads || Hq > kMaxHeads)
    return 0;
  AttnArgs a{};
  a.S = S;
  a.G = Hq / heads;
  a.rows = S * a.G;
  // the larger of the two kernels' needs: which one runs depends on the page size too
  set_rows(a, sdv::kAttnSimpleRows);
  const size_t simple = part_bytes(kSimplePerSm * (sms > 0 ? sms : 256), a.row_tile, dim);
  set_window_rows(a);
  const size_t tc = part_bytes(sms > 0 ? sms : 256, a.row_tile, dim);
  return sdv::kHeaderBytes + (simple > tc ? simple : tc);
}

}  // namespace

namespace sdv {

size_t attn_bytes(int B, int S, int Hq, int heads, int dim, int sms) {
  size_t most = attn_need(B, S, Hq, heads, dim, sms);
  // shorter windows too: a row tile has fewer rows where a second one begins
  for (int s = 1; most != 0 && s < S; ++s) {
    const size_t need = attn_need(B, s, Hq, heads, dim, sms);
    if (need > most) most = need;
  }
  return most;
}

sdv_status attn_check(const sdv_kvcache* cache, const void* q, int64_t q_stride, int32_t B, int32_t S, int32_t Hq,
                      const int32_t* ctx, const int32_t* n_rows, const uint32_t* mask, float scale, const void* out,
                      const float* lse) {
  if (!valid_cache(cache) || ctx == nullptr || out == nullptr || B < 1 || S < 1 || Hq < 1)
    return SDV_ERR_INVALID_ARG;
  if (Hq % cache->heads != 0 || !valid_rows(q, q_stride, Hq, cache->dim)) return SDV_ERR_INVALID_ARG;
  if (!aligned4(ctx) || !aligned4(n_rows) || !aligned4(mask) || !aligned4(lse) || !is_aligned16(out) ||
      !std::isfinite(scale))
    return SDV_ERR_INVALID_ARG;
  if (S > kMaxWindow || cache->dim > kMaxDim || Hq > kMaxHeads || (long long)B * Hq * S > kMaxUnits)
    return SDV_ERR_UNSUPPORTED;
  return SDV_OK;
}

AttnArgs attn_args(const sdv_kvcache* cache, const void* q, int64_t q_stride, int32_t B, int32_t S, int32_t Hq,
                   const int32_t* ctx, const int32_t* n_rows, const uint32_t* mask, float scale) {
  AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k = cache->k;
  a.v = cache->v;
  a.table = cache->table;
  a.ctx = ctx;
  a.n_rows = n_rows;
  a.mask = mask;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.B = B;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = cache->heads;
  a.G = Hq / cache->heads;
  a.D = cache->dim;
  a.n_pages = cache->n_pages;
  a.page = cache->page_size;
  a.max_pages = cache->max_pages;
  a.rows = S * a.G;
  return a;
}

sdv_status attn_run(const sdv_kvcache* cache, AttnArgs a, void* ws, cudaStream_t st) {
  a.status = static_cast<int*>(ws);
  a.fault = debug_fault();
  const int sms = sm_count();
  if (sms <= 0) return SDV_ERR_CUDA;
  const bool tc = attn_tc_takes(a.D, a.G, a.page, (long long)a.n_pages * a.Hkv * a.page);
  if (tc) set_window_rows(a);
  else set_rows(a, kAttnSimpleRows);
  a.tile = tc ? attn_tc_tile(a.D) : kAttnSimpleTile;
  // (0, 1 and 2: six tree windows 43.0, 35.5 and 33.4 us, 48 ragged contexts 120.8, 104.4
  // and 104.4)
  a.lead = tc ? 2 : 1;
  a.ctas = tc ? sms : kSimplePerSm * sms;
  // Shared units are joined by their last CTA where a partial is at most 2 KB (single
  // tokens), larger ones by a launch of many CTAs.  GPU us a call, launch against last CTA,
  // fp16, 8 cache heads: one sequence of 613, 5000 and 30,000 positions, then 48 of 40 to
  // 15,550.  4 rows x 128 (512 elements): 10.9 to 10.7, 15.2 to 16.5, 29.5 to 31.3, 236 to
  // 233, and the host issues one launch less (8.1 against 6.6 us).  8 x 128 (1024): 11.6 to
  // 12.9, 15.9 to 22.1, 30.0 to 36.9, 240 to 235; 4 x 256: 12.6 to 14.8, 19.3 to 23.3, 47.0
  // to 52.0, 454 to 448.  16 x 128 (2048): 12.5 to 16.0, 17.0 to 28.9, 30.9 to 44.2, 247 to 239.
  if (tc && a.row_tile * a.D <= 512 && a.ctas <= kAttnSharedBytes)
    a.shared = reinterpret_cast<unsigned*>(static_cast<char*>(ws) + kAttnSharedAt);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes);
  a.part_o = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part_ml) +
                                      round_256((size_t)2 * a.ctas * a.row_tile * 8));
  cudaError_t e = tc ? launch_attn_tc(cache->dtype, a, st) : launch_attn_simple(cache->dtype, a, st);
  // the join, unless the kernel joins or no unit can have more than one tile
  if (e == cudaSuccess && a.shared == nullptr && (long long)a.max_pages * a.page > a.tile) e = launch_attn_join(cache->dtype, a, st);
  return status_of(e);
}

}  // namespace sdv

extern "C" {

sdv_status sdv_kv_append(const sdv_kvcache* cache, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                         int32_t B, int32_t T, const int32_t* ctx, const int32_t* n_rows_or_null, void* ws_or_null,
                         sdv_stream_t stream) {
  if (!valid_cache(cache) || ctx == nullptr || !aligned4(ctx) || !aligned4(n_rows_or_null) || B < 1 || T < 1)
    return SDV_ERR_INVALID_ARG;
  if (!valid_rows(k, k_stride, cache->heads, cache->dim) || !valid_rows(v, v_stride, cache->heads, cache->dim))
    return SDV_ERR_INVALID_ARG;
  if (!sdv::is_aligned16(ws_or_null)) return SDV_ERR_WORKSPACE;
  if (B > kMaxSeqs || cache->dim > kMaxDim || cache->heads > kMaxHeads) return SDV_ERR_UNSUPPORTED;
  sdv::AppendArgs a{};
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.k_stride = k_stride / 8;
  a.v_stride = v_stride / 8;
  a.ck = static_cast<uint4*>(cache->k);
  a.cv = static_cast<uint4*>(cache->v);
  a.table = cache->table;
  a.ctx = ctx;
  a.n_rows = n_rows_or_null;
  a.T = T;
  a.heads = cache->heads;
  a.vec = cache->dim / 8;
  a.n_pages = cache->n_pages;
  a.page = cache->page_size;
  a.max_pages = cache->max_pages;
  a.status = static_cast<int*>(ws_or_null);
  const int warps = T < 8 ? T : 8;
  return sdv::status_of(sdv::launch_pdl(sdv::kv_append_kernel, dim3((T + warps - 1) / warps, B, 2), dim3(32 * warps),
                                        0, reinterpret_cast<cudaStream_t>(stream), a));
}

size_t sdv_paged_attn_workspace_bytes(int32_t B, int32_t S, int32_t Hq, int32_t heads, int32_t dim) {
  return sdv::attn_bytes(B, S, Hq, heads, dim, sdv::sm_count());
}

sdv_status sdv_paged_attn(const sdv_kvcache* cache, const void* q, int64_t q_stride, int32_t B, int32_t S, int32_t Hq,
                          const int32_t* ctx, const int32_t* n_rows_or_null, const uint32_t* mask_or_null,
                          float scale, void* out, float* lse_or_null, void* ws, size_t ws_bytes,
                          sdv_stream_t stream) {
  const sdv_status ok = sdv::attn_check(cache, q, q_stride, B, S, Hq, ctx, n_rows_or_null, mask_or_null, scale, out,
                                        lse_or_null);
  if (ok != SDV_OK) return ok;
  const size_t need = attn_need(B, S, Hq, cache->heads, cache->dim, sdv::sm_count());
  if (ws == nullptr || !sdv::is_aligned16(ws) || need == 0 || ws_bytes < need) return SDV_ERR_WORKSPACE;
  AttnArgs a = sdv::attn_args(cache, q, q_stride, B, S, Hq, ctx, n_rows_or_null, mask_or_null, scale);
  a.out = out;
  a.lse = lse_or_null;
  return sdv::attn_run(cache, a, ws, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

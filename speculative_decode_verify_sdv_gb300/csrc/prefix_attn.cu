// Attention of a batch over a prefix that its sequences share, computed once for all, and each
// sequence's own cache (sdv_prefix_attn): the prefix for head and page sizes that the tcgen05
// kernel does not take, the join, and the entry point.
//
// Per query row, with the prefix's positions in parts j and the row's own positions:
//   M = max m_j;  out = sum_j 2^(m_j - M) O_j / sum_j 2^(m_j - M) l_j;  lse = M + log sum.
// The query rows of all sequences stand side by side as the rows of one product with the
// prefix, which is so read once, not once a sequence; the own caches go through a kernel of their
// own (prefix_own.cu), or, where they may be long, through the paged attention, which deals any
// lengths evenly and leaves fp32 outputs here; the join adds them all, or the own positions' kernel does.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "attn_tc.h"
#include "host_util.h"
#include "mixing.h"
#include "paged_attn.h"
#include "prefix_attn.cuh"
#include "prefix_own.cuh"
#include "prefix_tc.h"
#include "sdv.h"
#include "sdv_device.cuh"

namespace sdv {

namespace {

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// ---- the prefix for any head and page size ----------------------------------------------

// What is not finite in column d of the values from position `from` to `to` - 1.
template <typename T>
__device__ __noinline__ uint32_t prefix_odd(const PrefixArgs& a, int h, int from, int to, int d) {
  uint32_t odd = 0;
  for (int p = from; p < to; ++p) {
    const int id = __ldg(a.table + p / a.page);
    if (id < 0 || id >= a.n_pages) continue;
    const float x = to_float(static_cast<const T*>(a.v)[(((long long)id * a.Hkv + h) * a.page + p % a.page) * a.D + d]);
    if (!(fabsf(x) < INFINITY)) odd |= x != x ? kOddNan : x > 0.f ? kOddPlus : kOddMinus;
  }
  return odd;
}

// Outputs of a row, two columns of every eight from `first` on, once more where they are not finite.
template <typename T>
__device__ __noinline__ void prefix_mend(const PrefixArgs& a, int h, int from, int to, float* row, int first) {
  for (int d = first; d < a.D; d += d & 1 ? 7 : 1) {
    if (fabsf(row[d]) < INFINITY) continue;
    const uint32_t odd = prefix_odd<T>(a, h, from, to, d);
    if (odd) row[d] = odd_value(odd);
  }
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

// Any head size and any page size.  One CTA walks its range of tiles with 64 query rows, 16 a warp:
// 32 positions at a time, the next ones on their way, by m16n8k16 MMAs out of rows that are padded so
// that eight of them meet no bank twice.  NB: blocks of eight columns, at least as many as a head has.
// 64 rows of 32 heads over 8 of 96, 8192 positions and 100 of their own 240 us a call (by the CUDA cores
// 3218), eight rows 72 (315); copies a position a warp and two barriers for 32 positions bound it.
template <typename T, int NB>
__global__ void __launch_bounds__(128, 2) prefix_simple_kernel(const __grid_constant__ PrefixArgs a) {
  constexpr int R = kPrefixSimpleRows, P = kPrefixSimpleTile, NT = P / 8;
  constexpr float kLift = std::is_same<T, __nv_bfloat16>::value ? -kPrefixDrop : 6.f;  // P's power of two
  extern __shared__ uint4 smem_wide[];
  const int D = a.D, chunks = D / 8, steps = (D + 15) / 16, ld = steps * 16 + 8;  // elements between rows
  T* const qs = reinterpret_cast<T*>(smem_wide);  // [R][ld]
  T* const ks = qs + R * ld;                     // [2][P][ld]
  T* const vs = ks + 2 * P * ld;                 // [2][P][ld]
  __shared__ bool gone[2][P];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  bool bad;
  const int length = prefix_length(a, bad);
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.status, kDevErrIndex);
  PrefixWalk w;
  if (!w.start(a, length, blockIdx.x)) return;
  for (int e = tid; e < (R + 4 * P) * ld / 8; e += 128) smem_wide[e] = make_uint4(0, 0, 0, 0);
  // The copies of a tile: a position a warp, 16 bytes a lane.
  auto copy = [&](int h, int t, int buf) {
#pragma unroll
    for (int i = 0; i < P / 4; ++i) {
      const int j = warp + 4 * i, p = t * P + j;
      int id = -1;
      if (p < length) {
        id = __ldg(a.table + p / a.page);
        if (id < 0 || id >= a.n_pages) {
          if (lane == 0) atomicOr(a.status, kDevErrIndex);
          id = -1;
        }
      }
      if (lane == 0) gone[buf][j] = id < 0;
      if (lane < chunks) {
        const long long at = id < 0 ? 0 : (((long long)id * a.Hkv + h) * a.page + p % a.page) * D + lane * 8;
        const int to = (buf * P + j) * ld + lane * 8;
        cp_async16(smem_addr(ks + to), static_cast<const T*>(a.k) + at, id >= 0);
        cp_async16(smem_addr(vs + to), static_cast<const T*>(a.v) + at, id >= 0);
      }
    }
    cp_async_commit();
  };
  while (w.more()) {
    const int count = w.segment();
    const int h = w.unit / a.row_tiles, r0 = (w.unit % a.row_tiles) * a.row_tile;
    const int nr = min(a.row_tile, a.tokens * a.G - r0);
    __syncthreads();
    for (int e = tid; e < R * chunks; e += 128) {
      const int r = e / chunks, ch = e - r * chunks, row = r0 + r;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < nr)
        x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (long long)(row / a.G) * a.q_stride +
                                                 (h * a.G + row % a.G) * D) + ch);
      *reinterpret_cast<uint4*>(qs + r * ld + ch * 8) = x;
    }
    float out[NB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[n][e] = 0.f;
    const bool busy = warp * 16 < nr;
    copy(h, w.tile, 0);
    for (int i = 0; i < count; ++i) {
      const int buf = i & 1;
      if (i + 1 < count) copy(h, w.tile + i + 1, buf ^ 1);
      else cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      if (busy) {
        const T* const k0 = ks + (buf * P + g) * ld + 2 * c;
        const T* const q0 = qs + (warp * 16 + g) * ld + 2 * c;
        auto word = [](const T* p) { return *reinterpret_cast<const uint32_t*>(p); };
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll 2
        for (int k = 0; k < steps; ++k) {
          const T* const q = q0 + k * 16;
          const uint32_t a0 = word(q), a1 = word(q + 8 * ld), a2 = word(q + 8), a3 = word(q + 8 * ld + 8);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const T* const x = k0 + n * 8 * ld + k * 16;
            mma16816<T>(s[n], a0, a1, a2, a3, word(x), word(x + 8));
          }
        }
        const uint32_t there = ~__ballot_sync(0xffffffffu, gone[buf][lane]);
        uint32_t p16[2][NT];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[2 * NT];
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e) {
            const bool see = there >> ((e >> 1) * 8 + c * 2 + (e & 1)) & 1u;
            x[e] = see ? s[e >> 1][half * 2 + (e & 1)] * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, x[e]);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const bool grow = mx > m[half] + 8.f;  // also from -inf to any number
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow && m[half] != -INFINITY ? exp2f(m[half] - mx) : 1.f;
            if (grow) m[half] = mx;
            l[half] *= f;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              out[n][half * 2] *= f;
              out[n][half * 2 + 1] *= f;
            }
          }
          const float ref = m[half] == -INFINITY ? -kLift : m[half] - kLift;
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * NT; e += 2) {
            const float y0 = exp2f(x[e] - ref), y1 = exp2f(x[e + 1] - ref);
            sum += y0 + y1;
            p16[half][e >> 1] = pack16<T>(y0, y1);
          }
          l[half] += sum;
        }
        // lane's row of the four 8 x 8 blocks: 16 positions by 16 columns
        const uint32_t v0 = smem_addr(vs + (buf * P + (lane & 15)) * ld + (lane >> 4) * 8);
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          if (n >= chunks) break;
#pragma unroll
          for (int k = 0; k < NT / 2; ++k) {
            uint32_t b[4];
            ldmatrix4_trans(b, v0 + (k * 16 * ld + n * 8) * 2);
            mma16816<T>(out[n], p16[0][2 * k], p16[1][2 * k], p16[0][2 * k + 1], p16[1][2 * k + 1], b[0], b[1]);
            mma16816<T>(out[n + 1], p16[0][2 * k], p16[1][2 * k], p16[0][2 * k + 1], p16[1][2 * k + 1], b[2], b[3]);
          }
        }
      }
      __syncthreads();  // everyone has read the tile
    }
    const size_t place = (size_t)w.unit * a.sharers + w.place(blockIdx.x);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float sum = l[half];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = warp * 16 + half * 8 + g;
      if (r >= nr) continue;
      float* const row = a.part_o + (place * a.row_tile + r) * D;
      bool finite = true;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (n >= chunks) break;
        const float2 y = sum == 0.f ? make_float2(0.f, 0.f) : make_float2(out[n][half * 2], out[n][half * 2 + 1]);
        finite &= fabsf(y.x) + fabsf(y.y) < INFINITY;
        *reinterpret_cast<float2*>(row + n * 8 + 2 * c) = y;
      }
      // (a weight of 0 times an infinity, or a value's own; NaN scores leave NaN)
      if (!finite && sum > 0.f) prefix_mend<T>(a, h, w.tile * P, min((w.tile + count) * P, length), row, 2 * c);
      if (c == 0)
        *reinterpret_cast<float2*>(a.part_ml + (place * a.row_tile + r) * 2) =
            make_float2(m[half] == -INFINITY ? -INFINITY : m[half] - kLift, sum);
    }
    w.advance(count);
  }
}

template <typename T, int NB>
cudaError_t simple_launch(const PrefixArgs& a, cudaStream_t st) {
  auto kernel = prefix_simple_kernel<T, NB>;
  const int smem = (kPrefixSimpleRows + 4 * kPrefixSimpleTile) * ((a.D + 15) / 16 * 16 + 8) * 2;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.ctas), dim3(128), smem, st, a);
}
template <typename T>
cudaError_t simple_dispatch(const PrefixArgs& a, cudaStream_t st) {
  return a.D <= 64    ? simple_launch<T, 8>(a, st)
         : a.D <= 128 ? simple_launch<T, 16>(a, st)
                      : simple_launch<T, 32>(a, st);
}
cudaError_t launch_prefix_simple(int dtype, const PrefixArgs& a, cudaStream_t st) {
  return dtype == SDV_F16 ? simple_dispatch<__half>(a, st) : simple_dispatch<__nv_bfloat16>(a, st);
}

// ---- join -------------------------------------------------------------------------------

// A row's softmax sums over some columns, partial by partial.
template <int N>
struct RowSum {
  float m = -INFINITY, l = 0.f;
  float4 o[N];
  template <bool ODD>
  __device__ __forceinline__ void add(float2 ml, const float4 (&x)[N]) {
    if (ml.x == -INFINITY && ml.y == 0.f) return;
    const float mn = fmaxf(m, ml.x), f = exp2f(m - mn), f2 = exp2f(ml.x - mn);
    m = mn;
    l = l * f + ml.y * f2;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      o[k].x = weighted<ODD>(o[k].x, f) + weighted<ODD>(x[k].x, f2);
      o[k].y = weighted<ODD>(o[k].y, f) + weighted<ODD>(x[k].y, f2);
      o[k].z = weighted<ODD>(o[k].z, f) + weighted<ODD>(x[k].z, f2);
      o[k].w = weighted<ODD>(o[k].w, f) + weighted<ODD>(x[k].w, f2);
    }
  }
};

constexpr int kJoinThreads = 128;
// CTAs per SM up to which a row has more threads with more partials in flight each: six partials of
// 3456 rows of 256 columns 12.4 us by 8 threads a row, 10.7 by 32; three to four partials of 40,960 rows
// of 128 columns 21 us by 8 threads, 35 by 16.
constexpr int kJoinFewCtas = 8;

// kRowThreads threads a row, each with every kRowThreads-th four columns (N of them) of all its
// partials, `AHEAD` partials in flight.
template <typename T, int kRowThreads, int N, int AHEAD>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ JoinArgs j) {
  const PrefixArgs& a = j.prefix;
  const AttnArgs& own = j.own.attn;
  const int D = a.D, j4 = threadIdx.x % kRowThreads;
  const long long orow = (long long)blockIdx.x * (kJoinThreads / kRowThreads) + threadIdx.x / kRowThreads;
  // The split first, while the launches in front end: its lengths are read behind the word that passes
  // the first one's wait on.
  const bool beside = a.passed != nullptr && passed_on(a.passed);
  if (!beside) griddep_wait();
  const bool is = orow < (long long)a.tokens * a.Hq;
  const int token = is ? (int)(orow / a.Hq) : 0, head = is ? (int)(orow - (long long)token * a.Hq) : 0;
  const int h = head / a.G, row = token * a.G + head - h * a.G, rt = row / a.row_tile, r = row - rt * a.row_tile;
  const int per_head = (a.row_tiles + a.unit_tiles - 1) / a.unit_tiles;
  const int unit = h * per_head + rt / a.unit_tiles, sub = rt % a.unit_tiles;
  const int b = token / own.S, s = token - b * own.S;
  const AttnSeq seq = attn_seq(own, b);
  bool bad;
  const int length = prefix_length(a, bad), tiles = prefix_tiles(a, length);
  const long long total = (long long)tiles * a.units, first = (long long)unit * tiles;
  const int live = attn_live_ctas(a.ctas, total);
  const bool row_is = s < seq.n;
  const bool in_parts = j.own.prefix_parts > 0;
  int parts = 0;
  if (row_is && tiles > 0)
    parts = in_parts ? own_live_parts((length + kOwnTile - 1) / kOwnTile, j.own.prefix_parts)
                     : attn_owner(total, live, first + tiles - 1) - attn_owner(total, live, first) + 1;
  const int own_parts = row_is && j.own.parts > 0 ? own_live_parts(seq.tiles, j.own.parts) : 0;
  griddep_wait();
  griddep_launch_dependents();
  if (a.passed != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.passed = 0;  // (who starts now finds them ended)
  if (!is) return;
  RowSum<N> sum;
  auto gather = [&](auto odd, const float2* ml, const float4* po, long long ml_step, long long po_step, int count) {
    for (int k0 = 0; k0 < count; k0 += AHEAD) {
      float2 ms[AHEAD];
      float4 x[AHEAD][N];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (k0 + k >= count) break;
        ms[k] = __ldcg(ml + (k0 + k) * ml_step);
#pragma unroll
        for (int n = 0; n < N; ++n)
          x[k][n] = j4 + n * kRowThreads < D / 4 ? __ldcg(po + (k0 + k) * po_step + j4 + n * kRowThreads)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (k0 + k >= count) break;
        sum.template add<decltype(odd)::value>(ms[k], x[k]);
      }
    }
  };
  auto all = [&](auto odd) {
    sum.m = -INFINITY;
    sum.l = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) sum.o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
    const long long step2 = (long long)a.tokens * a.Hq, step = in_parts ? step2 : (long long)a.unit_tiles * a.row_tile;
    const long long at = in_parts ? orow : ((long long)unit * a.sharers * a.unit_tiles + sub) * a.row_tile + r;
    gather(odd, reinterpret_cast<const float2*>(a.part_ml) + at, reinterpret_cast<const float4*>(a.part_o) + at * (D / 4),
           step, step * (D / 4), parts);
    if (j.own.parts > 0) {
      gather(odd, j.own.part_ml + orow, reinterpret_cast<const float4*>(j.own.part_o) + orow * (D / 4), step2,
             step2 * (D / 4), own_parts);
    } else if (row_is) {
      // the own positions' output is that of a sum of 1 at a maximum of their lse
      const float lse = __ldcg(own.lse + orow);
      float4 x[N];
#pragma unroll
      for (int n = 0; n < N; ++n)
        x[n] = j4 + n * kRowThreads < D / 4
                   ? __ldcg(reinterpret_cast<const float4*>(own.out32) + orow * (D / 4) + j4 + n * kRowThreads)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      if (lse != -INFINITY) sum.template add<decltype(odd)::value>(make_float2(lse * 1.4426950408889634f, 1.f), x);
    }
  };
  all(std::false_type());
  bool finite = true;
#pragma unroll
  for (int n = 0; n < N; ++n)
    finite &= fabsf(sum.o[n].x) + fabsf(sum.o[n].y) + fabsf(sum.o[n].z) + fabsf(sum.o[n].w) < INFINITY;
  if (!finite) all(std::true_type());
  const bool none = !row_is || sum.l == 0.f;
  const float inv = 1.f / sum.l;
  uint2* const dst = reinterpret_cast<uint2*>(static_cast<T*>(j.out) + orow * D);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (j4 + n * kRowThreads < D / 4)
      dst[j4 + n * kRowThreads] =
          none ? make_uint2(0u, 0u)
               : make_uint2(pack16<T>(sum.o[n].x * inv, sum.o[n].y * inv), pack16<T>(sum.o[n].z * inv, sum.o[n].w * inv));
  if (j4 == 0 && j.lse != nullptr)
    j.lse[orow] = none ? -INFINITY : (sum.m + log2f(sum.l)) * 0.6931471805599453f;
}

template <typename T, int kRowThreads, int N, int AHEAD>
cudaError_t join_launch(const JoinArgs& j, cudaStream_t st) {
  const long long rows = (long long)j.prefix.tokens * j.prefix.Hq, per = kJoinThreads / kRowThreads;
  return launch_pdl(prefix_join_kernel<T, kRowThreads, N, AHEAD>, dim3((unsigned)((rows + per - 1) / per)),
                    dim3(kJoinThreads), 0, st, j);
}

template <typename T>
cudaError_t join_dispatch(const JoinArgs& j, int sms, cudaStream_t st) {
  const int D = j.prefix.D;
  const bool few = (long long)j.prefix.tokens * j.prefix.Hq * (D <= 64 ? 8 : D <= 128 ? 16 : 32) <=
                   (long long)kJoinFewCtas * kJoinThreads * sms;
  if (D <= 64) return few ? join_launch<T, 8, 2, 8>(j, st) : join_launch<T, 8, 2, 4>(j, st);
  if (D <= 128) return few ? join_launch<T, 16, 2, 8>(j, st) : join_launch<T, 8, 4, 4>(j, st);
  return few ? join_launch<T, 32, 2, 8>(j, st) : join_launch<T, 8, 8, 2>(j, st);
}

cudaError_t launch_prefix_join(int dtype, const JoinArgs& j, int sms, cudaStream_t st) {
  return dtype == SDV_F16 ? join_dispatch<__half>(j, sms, st) : join_dispatch<__nv_bfloat16>(j, sms, st);
}

constexpr int kSimplePerSm = 2;
// Partials of a row that the own positions' kernel adds up itself, where it has all of a sequence's
// positions in one part: no launch and no partials of its own for the join.  256 windows of five rows,
// 32 heads over 8 of 128, up to 500 positions 123 us a call against 132, up to 1001 behind 16,384
// 352 against 362; 199 of 20 rows, one position 38 against 43; 450 of one row, up to 60 43 against 42;
// 256 of 16 rows, heads of 64, 52 against 55.  Heads of 256 have no registers for it (72 against 59).
constexpr int kLastSharers = 4;
// CTAs for the own positions, were all tables full (some end at once): per SM 16 of one warp (16, 24, 32,
// 48: 64 sequences of up to 2001 positions 72.1, 71.3, 71.0, 73.1 us a call), 8 of more (8, 12, 16: 256
// windows of five rows, up to 1001 positions, 361.8, 360.6, 361.7).
int own_ctas(int warps, int sms) { return (warps > 1 ? 8 : 16) * sms; }

// Up to 16 rows a kv head, heads of up to 128 and up to 8192 positions: the prefix goes into the
// launch of the own positions, in at most 32 parts a head (the join reads them all: 75 parts of 4800
// positions 21.3 us, 25 of them 18.0).  Against the tensor-core kernel in front of that launch,
// four rows of 32 heads over 8 of 128, 100 positions of their own: 300 positions 11.9 against
// 13.3 us, 2400 16.0 against 21.8, 8000 23.1 against 25.0; one row 11.2 against 13.0, 14.4 against
// 21.4, 21.1 against 24.3.  32 rows a head (two row tiles a warp) lose, 18.3 against 14.8 at 1201
// positions, and so do heads of 256, 25.6 against 22.1 at 4800.  Its partials are at most
// 2 sms * 16 rows, a quarter of what the workspace has room for.
constexpr int kPrefixFewRows = 16;
constexpr int kPrefixFewParts = 32;
constexpr int kPrefixFewTiles = 4;  // of kOwnTile positions in a part of it

// Row tiles and units of a call; `tc`: of the tensor-core kernel.
void set_units(PrefixArgs& a, bool tc, int sms) {
  if (tc) {
    // whole tokens, at most 128 rows, tiles of equal size
    const int most = a.G < kPrefixTcRows ? kPrefixTcRows / a.G : 1;
    a.tiles_most = (a.tokens + most - 1) / most;
    a.tile_tokens = (a.tokens + a.tiles_most - 1) / a.tiles_most;
    a.row_tiles = (a.tokens + a.tile_tokens - 1) / a.tile_tokens;
    a.row_tile = a.tile_tokens * a.G;
    a.unit_tiles = prefix_tc_streams(a.D, a.tiles_most);
    a.tile = kPrefixTcTile;
    a.ctas = sms;
  } else {
    a.row_tile = kPrefixSimpleRows;
    a.row_tiles = (a.tokens * a.G + a.row_tile - 1) / a.row_tile;
    a.unit_tiles = 1;
    a.tile = kPrefixSimpleTile;
    a.ctas = kSimplePerSm * sms;
  }
  a.units = a.Hkv * ((a.row_tiles + a.unit_tiles - 1) / a.unit_tiles);
  // a unit's tiles take at most ceil(ctas / units) CTAs' ranges, and begin and end inside one
  a.sharers = (a.ctas + a.units - 1) / a.units + 1;
}

// Parts of a sequence's own positions: enough CTAs for two rounds of them, and no more than tiles.
// The prefix too where there are few rows and a part of it is short.
void set_parts(OwnArgs& o, int sms) {
  const AttnArgs& a = o.attn;
  const long long tiles = ((long long)a.max_pages * a.page + kOwnTile - 1) / kOwnTile;
  const long long prefix_tiles = ((long long)o.prefix_pages * a.page + kOwnTile - 1) / kOwnTile;
  const int room = 2 * sms / a.Hkv, most = room < kPrefixFewParts ? room : kPrefixFewParts;
  const long long prefix_parts = prefix_tiles < most ? prefix_tiles : most;
  const bool few = a.D <= 128 && (long long)a.B * a.rows <= kPrefixFewRows && prefix_tiles <= kPrefixFewTiles * prefix_parts;
  o.prefix_parts = few ? (int)prefix_parts : 0;
  o.warps = a.rows <= 16 || a.D > 128 ? 1 : a.rows <= 32 ? 2 : 4;
  o.row_groups = (a.rows + 16 * o.warps - 1) / (16 * o.warps);
  const long long units = (long long)a.B * a.Hkv * o.row_groups;
  long long parts = ((long long)own_ctas(o.warps, sms) + units - 1) / units;
  if (parts > kOwnMaxParts) parts = kOwnMaxParts;
  o.parts = parts < tiles ? (int)parts : (int)tiles;
}

struct PrefixBytes {
  size_t part_ml, part_o, own_ml, own_o, total;  // offsets; own_ml, own_o: or the outputs' lse and fp32 values
};

PrefixBytes prefix_layout(const PrefixArgs& a, size_t own, int B, int S, int sms) {
  // units * sharers partials of unit_tiles * row_tile rows each, in terms that grow with the call
  const int most = a.tile_tokens == 0 ? a.row_tile : kPrefixTcRows;
  const size_t tiles_most = a.tile_tokens == 0 ? a.row_tiles : a.tiles_most;
  const size_t units_most = a.Hkv * ((tiles_most + a.unit_tiles - 1) / a.unit_tiles);
  const size_t rows = (a.ctas + 2 * units_most) * a.unit_tiles * most, outs = (size_t)B * S * a.Hq;
  // parts * units * 16 warps rows, parts at most own_ctas / units + 1, in terms that grow with the call
  const int wide = a.D > 128 ? 1 : 4;
  const size_t groups = ((size_t)S * a.G + 16 * wide - 1) / (16 * wide) * a.Hkv * B;
  const size_t parts = (own_ctas(wide, sms) + groups) * 16 * wide;
  const size_t own_rows = parts > outs ? parts : outs;
  PrefixBytes p;
  p.part_ml = round_256(own);
  p.part_o = p.part_ml + round_256(rows * 8);
  p.own_ml = p.part_o + round_256(rows * a.D * 4);
  p.own_o = p.own_ml + round_256(own_rows * 8);
  p.total = p.own_o + round_256(own_rows * a.D * 4);
  return p;
}

PrefixArgs prefix_shape(int B, int S, int Hq, int heads, int dim, bool tc, int sms) {
  PrefixArgs a{};
  a.tokens = B * S;
  a.Hq = Hq;
  a.Hkv = heads;
  a.G = Hq / heads;
  a.D = dim;
  set_units(a, tc, sms);
  return a;
}

// `own`: attn_bytes of the call.
size_t prefix_need(size_t own, int B, int S, int Hq, int heads, int dim, int sms) {
  if (own == 0 || (long long)B * S * Hq > (1ll << 30)) return 0;
  if (sms <= 0) sms = 256;
  size_t most = 0;
  for (int tc = 0; tc < 2; ++tc) {
    const size_t n = prefix_layout(prefix_shape(B, S, Hq, heads, dim, tc, sms), own, B, S, sms).total;
    if (n > most) most = n;
  }
  return most;
}

}  // namespace

}  // namespace sdv

extern "C" {

size_t sdv_prefix_attn_workspace_bytes(int32_t B, int32_t S, int32_t Hq, int32_t heads, int32_t dim) {
  const int sms = sdv::sm_count();
  return sdv::prefix_need(sdv::attn_bytes(B, S, Hq, heads, dim, sms), B, S, Hq, heads, dim, sms);
}

sdv_status sdv_prefix_attn(const sdv_kvcache* cache, const int32_t* prefix_table, int32_t prefix_pages,
                           const int32_t* prefix_len, const void* q, int64_t q_stride, int32_t B, int32_t S,
                           int32_t Hq, const int32_t* ctx, const int32_t* n_rows_or_null,
                           const uint32_t* mask_or_null, float scale, void* out, float* lse_or_null, void* ws,
                           size_t ws_bytes, sdv_stream_t stream) {
  const sdv_status ok = sdv::attn_check(cache, q, q_stride, B, S, Hq, ctx, n_rows_or_null, mask_or_null, scale, out,
                                        lse_or_null);
  if (ok != SDV_OK) return ok;
  if (prefix_table == nullptr || prefix_len == nullptr || prefix_pages < 1 ||
      ((reinterpret_cast<uintptr_t>(prefix_table) | reinterpret_cast<uintptr_t>(prefix_len)) & 3u) != 0)
    return SDV_ERR_INVALID_ARG;
  const int sms = sdv::sm_count();
  const size_t own_bytes = sdv::attn_bytes(B, S, Hq, cache->heads, cache->dim, sms);
  const size_t need = sdv::prefix_need(own_bytes, B, S, Hq, cache->heads, cache->dim, sms);
  if (ws == nullptr || !sdv::is_aligned16(ws) || need == 0 || ws_bytes < need) return SDV_ERR_WORKSPACE;
  if (sms <= 0) return SDV_ERR_CUDA;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool tc = sdv::attn_tc_takes(cache->dim, Hq / cache->heads, cache->page_size,
                                     (long long)cache->n_pages * cache->heads * cache->page_size);
  sdv::PrefixArgs a = sdv::prefix_shape(B, S, Hq, cache->heads, cache->dim, tc, sms);
  a.q = q;
  a.q_stride = q_stride;
  a.k = cache->k;
  a.v = cache->v;
  a.table = prefix_table;
  a.length = prefix_len;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_pages = cache->n_pages;
  a.page = cache->page_size;
  a.max_pages = prefix_pages;
  a.status = static_cast<int*>(ws);
  a.fault = sdv::debug_fault();
  const sdv::PrefixBytes at = sdv::prefix_layout(a, own_bytes, B, S, sms);
  char* const base = static_cast<char*>(ws);
  a.part_ml = reinterpret_cast<float*>(base + at.part_ml);
  a.part_o = reinterpret_cast<float*>(base + at.part_o);
  sdv::JoinArgs j{};
  j.out = out;
  j.lse = lse_or_null;
  sdv::OwnArgs& own = j.own;
  own.attn = sdv::attn_args(cache, q, q_stride, B, S, Hq, ctx, n_rows_or_null, mask_or_null, scale);
  own.status = a.status;
  own.prefix_table = prefix_table;
  own.prefix_length = prefix_len;
  own.prefix_pages = prefix_pages;
  sdv::set_parts(own, sms);
  own.attn.fault = sdv::debug_fault();
  const bool parts = tc && sdv::own_takes(own, sms);
  if (!parts) own.prefix_parts = 0;
  if (parts) a.passed = reinterpret_cast<unsigned*>(static_cast<char*>(ws) + sdv::kPassedAt);
  if (own.prefix_parts > 0) {
    own.prefix_o = a.part_o;
    own.prefix_ml = reinterpret_cast<float2*>(a.part_ml);
  } else {
    const cudaError_t e =
        tc ? sdv::launch_prefix_tc(cache->dtype, a, st) : sdv::launch_prefix_simple(cache->dtype, a, st);
    if (e != cudaSuccess) return sdv::status_of(e);
  }
  j.prefix = a;
  if (parts) {
    own.attn.tile = sdv::kOwnTile;
    own.part_ml = reinterpret_cast<float2*>(base + at.own_ml);
    own.part_o = reinterpret_cast<float*>(base + at.own_o);
    const bool last = own.prefix_parts == 0 && own.parts == 1 && a.D <= 128 && a.sharers <= sdv::kLastSharers;
    const cudaError_t e2 = sdv::launch_prefix_own(cache->dtype, j, last, st);
    if (e2 != cudaSuccess || last) return sdv::status_of(e2);
  } else {
    own.parts = 0;
    own.attn.out32 = reinterpret_cast<float*>(base + at.own_o);
    own.attn.lse = reinterpret_cast<float*>(base + at.own_ml);
    const sdv_status run = sdv::attn_run(cache, own.attn, ws, st);
    if (run != SDV_OK) return run;
    own.attn.tile = 1;  // (of no meaning to the join)
  }
  return sdv::status_of(sdv::launch_prefix_join(cache->dtype, j, sms, st));
}

}  // extern "C"

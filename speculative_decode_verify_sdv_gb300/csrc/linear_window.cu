// Linear attention of a short window (2 to 32 tokens): the outputs from the state as it
// stands, and the state behind it.
//
// Per head, with G the cumulative log decay of the window and M the state before it:
//   O_t = scale (e^{G_t} q_t M + sum_{s <= t} (q_t . k_s) e^{G_t - G_s} v_s)
//   M'  = e^{G_n} M + sum_{s < n} e^{G_n - G_s} k_s v_s^T
// Reading the state (and writing it) bounds both: 64 KB a head at 128 x 128 against 17
// rows of a few hundred bytes.  The outputs' products are too many for fp32 units (a
// window of 17: 0.6 MFLOP for 64 KB) and too small to fill a 128-row tcgen05 tile, whose
// chain of copies took 40 us for 512 heads; they run on mma.sync (m16n8k16) with the
// state going from global memory into operand registers as it comes, a CTA per head,
// several per SM so that one's loads hide the other's arithmetic.  The state's update is
// fp32 multiply-adds in registers.
//
// 17 tokens, 512 heads of 128 x 128, fp16, calls in a row on states that are not in L2:
// outputs 18.9 us (1.8 TB/s: two CTAs an SM do not hide the products and the sum over the key
// rows behind the read), the state 23.9 us at 17 tokens and 18.1 at 9 (3.7 TB/s read and
// written: 1024 CTAs, three on an SM, are 2.2 waves of load, update and store; a token more
// is 0.3 to 0.7 us), a round of both 33 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "linear_args.h"
#include "mixing.h"
#include "sdv.h"
#include "tc_util.cuh"

namespace sdv {

namespace {

constexpr int kWin = kLinWindow;      // 32: two row tiles of the MMA
constexpr int kWinThreads = 256;      // of the commit

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma_16816(d, a[0], a[1], a[2], a[3], b0, b1, d);
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D += A B, m16n8k8, tf32 operands (10-bit mantissas, fp32's range), fp32 sums.
__device__ __forceinline__ void mma8_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Decays of a window, one token a lane: G_t in pairs of floats.
__device__ __forceinline__ DecaySum window_decay(const LinArgs& a, int b, int h, int n, int lane) {
  const float x = lane < n ? lin_decay(a, b, lane, h) : 0.f;
  DecaySum g = DecaySum::log2_of(x);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const DecaySum o{__shfl_up_sync(0xffffffffu, g.hi, off), __shfl_up_sync(0xffffffffu, g.lo, off)};
    if (lane >= off) g.add(o);
  }
  return g;
}

// ---- outputs --------------------------------------------------------------------------

// DV / 16 warps: 32 value columns (DV / 32 groups) x half of the key rows.  Element
// (row, column) of the state goes to operand registers by 16-byte loads: lane l's
// columns 4 (l / 4) .. + 3 of the group are column l / 4 of four n-tiles, its rows
// 2 (l % 4) + {0, 1, 8, 9} a k-tile's.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(DV * 2, 512 / (DV * 2)) linear_window_kernel(const LinArgs a) {
  constexpr int kThreads = DV * 2, kWarps = DV / 16;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kGroups = DV / 32, kParts = 2, kRows = DK / kParts, kSteps = kRows / 16;
  constexpr int ld = DK + 8, ldv = DV + 8;  // padded rows: ldmatrix without conflicts
  __shared__ alignas(16) T sq[kWin][ld], sk[kWin][ld], sv[kWin][ldv];
  __shared__ float sp[kWin][kWin + 1];        // decayed scores
  __shared__ DecaySum sg[kWin];
  __shared__ float smax[kWarps];
  __shared__ alignas(16) float ssum[(kParts - 1) * kWin * DV];  // the other parts' sums
  griddep_wait();
  const int h = blockIdx.x, b = blockIdx.y, hk = h / (a.H / a.Hqk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lin_tokens(a, b);
  const int grp = warp % kGroups, part = warp / kGroups;
  const int kr = 2 * (lane & 3), nc = lane >> 2;
  // the state's loads first: everything else hides behind them
  float4 m[kSteps][4];
  const float* const s_in = a.s_in + ((long long)b * a.H + h) * DK * DV;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = part * kRows + 16 * s + kr + (e & 1) + 8 * (e >> 1);
      m[s][e] = a.s_in != nullptr ? *reinterpret_cast<const float4*>(s_in + (long long)row * DV + 32 * grp + 4 * nc)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  // the window's rows, zeros behind its end (all of q, k, v is then finite or counts)
  const T* const q = static_cast<const T*>(a.q) + (long long)b * a.T * a.q_stride + hk * DK;
  const T* const k = static_cast<const T*>(a.k) + (long long)b * a.T * a.k_stride + hk * DK;
  const T* const v = static_cast<const T*>(a.v) + (long long)b * a.T * a.v_stride + h * DV;
  for (int e = threadIdx.x; e < kWin * (DK / 8); e += kThreads) {
    const int t = e / (DK / 8), c = e % (DK / 8) * 8;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (t < n) {
      x = __ldg(reinterpret_cast<const uint4*>(q + t * a.q_stride + c));
      y = __ldg(reinterpret_cast<const uint4*>(k + t * a.k_stride + c));
    }
    *reinterpret_cast<uint4*>(&sq[t][c]) = x;
    *reinterpret_cast<uint4*>(&sk[t][c]) = y;
  }
  uint32_t vmax = 0;
  for (int e = threadIdx.x; e < kWin * (DV / 8); e += kThreads) {
    const int t = e / (DV / 8), c = e % (DV / 8) * 8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (t < n) x = __ldg(reinterpret_cast<const uint4*>(v + t * a.v_stride + c));
    *reinterpret_cast<uint4*>(&sv[t][c]) = x;
    vmax = __vmaxu2(vmax, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
  }
  const bool odd = max(vmax & 0xffffu, vmax >> 16) >= (kBf16 ? 0x7f80u : 0x7c00u);
  if (warp == 0) sg[lane] = window_decay(a, b, h, n, lane);
  // the largest finite entry of the state sets the copy's power of two (fp16)
  if (!kBf16) {
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x[4] = {fabsf(m[s][e].x), fabsf(m[s][e].y), fabsf(m[s][e].z), fabsf(m[s][e].w)};
#pragma unroll
        for (int z = 0; z < 4; ++z) big = fmaxf(big, x[z] < INFINITY ? x[z] : 0.f);
      }
    const uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
    if (lane == 0) smax[warp] = __uint_as_float(mx);
  }
  const bool infinite = __syncthreads_or(odd);  // a value that is not finite
  float up = 1.f, down = 1.f;
  if (!kBf16) {
    float big = smax[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) big = fmaxf(big, smax[w]);
    const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 120);
    up = exp2f((float)(14 - ex));
    down = exp2f((float)(ex - 14));
  }
  // scores: warp = 8 tokens s of a 16-row tile of t; s_ts e^{G_t - G_s}, 0 behind t
#pragma unroll
  for (int tile = warp; tile < 8; tile += kWarps) {
    const int mt = tile & 1, nt = tile >> 1;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    if (8 * nt <= 16 * mt + 15) {
      const uint32_t qa = smem_addr(&sq[16 * mt + (lane & 15)][8 * (lane >> 4)]);
#pragma unroll
      for (int s = 0; s < DK / 16; ++s) {
        uint32_t fa[4];
        ldsm4(qa + 32 * s, fa);
        const T* const kp = &sk[8 * nt + nc][16 * s + kr];
        mma16<T>(d, fa, *reinterpret_cast<const uint32_t*>(kp), *reinterpret_cast<const uint32_t*>(kp + 8));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * mt + nc + 8 * (e >> 1), s = 8 * nt + kr + (e & 1);
      const float w = s <= t ? exp2_approx(sg[t].minus(sg[s])) : 0.f;
      sp[t][s] = w == 0.f ? 0.f : d[e] * w;
    }
  }
  // e^{G_t} q_t M for this warp's columns and key rows
  float o[2][4][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
  const bool two = n > 16;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    uint32_t fa[2][4];
    const uint32_t qa = smem_addr(&sq[lane & 15][part * kRows + 16 * s + 8 * (lane >> 4)]);
    ldsm4(qa, fa[0]);
    if (two) ldsm4(qa + 16 * ld * 2, fa[1]);
    const float* const x[4] = {&m[s][0].x, &m[s][1].x, &m[s][2].x, &m[s][3].x};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b0 = pack16<T>(x[0][j] * up, x[1][j] * up), b1 = pack16<T>(x[2][j] * up, x[3][j] * up);
      mma16<T>(o[0][j], fa[0], b0, b1);
      if (two) mma16<T>(o[1][j], fa[1], b0, b1);
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const DecaySum g = sg[16 * mt + nc + 8 * (e >> 1)];
      const float eg = exp2_approx(g.hi + g.lo), f = eg * down;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[mt][j][e] = eg == 0.f ? 0.f : o[mt][j][e] * f;  // drops whatever the state holds
    }
  // the window's own tokens: P V in steps of 8 tokens dealt to the parts.  P as tf32 keeps
  // fp32's range (scores need no scale) and 11 bits; a value of the type is one of tf32's.
  __syncthreads();
  if (!infinite) {
#pragma unroll 1
    for (int s0 = 8 * part; s0 < n; s0 += 8 * kParts) {
      const int s = s0 + (lane & 3);
      const uint2 x0 = *reinterpret_cast<const uint2*>(&sv[s][32 * grp + 4 * nc]);
      const uint2 x1 = *reinterpret_cast<const uint2*>(&sv[s + 4][32 * grp + 4 * nc]);
      const float2 u0 = unpack16<T>(x0.x), u1 = unpack16<T>(x0.y), w0 = unpack16<T>(x1.x), w1 = unpack16<T>(x1.y);
      const float b0[4] = {u0.x, u0.y, u1.x, u1.y}, b1[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        if (mt == 1 && !two) break;
        const uint32_t fa[4] = {to_tf32(sp[16 * mt + nc][s]), to_tf32(sp[16 * mt + nc + 8][s]),
                                to_tf32(sp[16 * mt + nc][s + 4]), to_tf32(sp[16 * mt + nc + 8][s + 4])};
#pragma unroll
        for (int j = 0; j < 4; ++j) mma8_tf32(o[mt][j], fa, __float_as_uint(b0[j]), __float_as_uint(b1[j]));
      }
    }
  }
  // the parts' sums to part 0
  if (part > 0) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ssum[((part - 1) * kWin + 16 * mt + nc + 8 * (e >> 1)) * DV + 32 * grp + 4 * (kr + (e & 1)) + j] = o[mt][j][e];
  }
  __syncthreads();
  if (part > 0) return;
#pragma unroll
  for (int p = 0; p < kParts - 1; ++p)
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 y = *reinterpret_cast<const float4*>(
            &ssum[(p * kWin + 16 * mt + nc + 8 * (e >> 1)) * DV + 32 * grp + 4 * (kr + (e & 1))]);
        o[mt][0][e] += y.x;
        o[mt][1][e] += y.y;
        o[mt][2][e] += y.z;
        o[mt][3][e] += y.w;
      }
  T* const out = static_cast<T*>(a.o) + ((long long)b * a.T * a.H + h) * DV;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int t = 16 * mt + nc + 8 * hf;
      if (t >= a.T) continue;
      if (infinite) {
        // One by one: a weight of zero must not meet them, and what is not finite goes
        // through the state, as the sum over the key rows of q (k v), not as (q k) v.
        for (int s = 0; s <= t && s < n; ++s) {
          if (exp2_approx(sg[t].minus(sg[s])) == 0.f) continue;
          const float p = sp[t][s];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint2 x = *reinterpret_cast<const uint2*>(&sv[s][32 * grp + 4 * (kr + e)]);
            const float2 y0 = unpack16<T>(x.x), y1 = unpack16<T>(x.y);
            const float y[4] = {y0.x, y0.y, y1.x, y1.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float add = p * y[j];
              if (!(fabsf(y[j]) < INFINITY)) {
                add = 0.f;
#pragma unroll 1
                for (int r = 0; r < DK; ++r) add = fmaf(lin_float(sq[t][r]), lin_float(sk[s][r]) * y[j], add);
              }
              o[mt][j][2 * hf + e] += add;
            }
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = a.scale;
        const uint2 y = t < n ? make_uint2(pack16<T>(o[mt][0][2 * hf + e] * f, o[mt][1][2 * hf + e] * f),
                                           pack16<T>(o[mt][2][2 * hf + e] * f, o[mt][3][2 * hf + e] * f))
                              : make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(out + (long long)t * a.H * DV + 32 * grp + 4 * (kr + e)) = y;
      }
    }
}

// ---- the state behind the window --------------------------------------------------------

// A CTA per head and 64 value columns; thread = 4 columns x DK / 16 rows of the state: 77
// registers at 128 key rows, three CTAs per SM (one CTA of twice the rows per head was 1.7
// waves of two: 21.8 us for 512 heads).  Keys and values come from shared memory in fp32.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kWinThreads) linear_commit_kernel(const LinArgs a) {
  constexpr int kCols = 16, kRowSets = kWinThreads / kCols, kRows = DK / kRowSets;
  __shared__ float4 sk[kWin][DK / 4], sv[kWin][kCols];
  __shared__ float sw[kWin], sdec;
  griddep_wait();
  const int h = blockIdx.x / (DV / 64), c0 = blockIdx.x % (DV / 64) * 64, b = blockIdx.y, hk = h / (a.H / a.Hqk);
  const int n = lin_tokens(a, b);
  const int c = threadIdx.x % kCols, r0 = threadIdx.x / kCols * kRows;
  const long long at = ((long long)b * a.H + h) * DK * DV + (long long)r0 * DV + c0 + 4 * c;
  float4 m[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    m[r] = a.s_in != nullptr ? *reinterpret_cast<const float4*>(a.s_in + at + (long long)r * DV)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const DecaySum g = window_decay(a, b, h, n, lane);
    const DecaySum all{__shfl_sync(0xffffffffu, g.hi, 31), __shfl_sync(0xffffffffu, g.lo, 31)};
    sw[lane] = exp2f(all.minus(g));
    if (lane == 0) sdec = exp2f(all.hi + all.lo);
  }
  const T* const k = static_cast<const T*>(a.k) + (long long)b * a.T * a.k_stride + hk * DK;
  const T* const v = static_cast<const T*>(a.v) + (long long)b * a.T * a.v_stride + h * DV + c0;
  for (int e = threadIdx.x; e < n * (DK / 4); e += kWinThreads) {
    const int t = e / (DK / 4), d = e % (DK / 4);
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(k + t * a.k_stride + 4 * d));
    const float2 y = unpack16<T>(x.x), z = unpack16<T>(x.y);
    sk[t][d] = make_float4(y.x, y.y, z.x, z.y);
  }
  for (int e = threadIdx.x; e < n * kCols; e += kWinThreads) {
    const int t = e / kCols, d = e % kCols;
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(v + t * a.v_stride + 4 * d));
    const float2 y = unpack16<T>(x.x), z = unpack16<T>(x.y);
    sv[t][d] = make_float4(y.x, y.y, z.x, z.y);
  }
  __syncthreads();
  const float dec = sdec;
#pragma unroll
  for (int r = 0; r < kRows; ++r)  // a decay of 0 drops the state whatever it holds
    m[r] = dec == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                      : make_float4(m[r].x * dec, m[r].y * dec, m[r].z * dec, m[r].w * dec);
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    const float w = sw[t];
    if (w == 0.f) continue;  // dropped since, whatever its values are
    float4 x = sv[t][c];
    x.x *= w;
    x.y *= w;
    x.z *= w;
    x.w *= w;
#pragma unroll
    for (int r = 0; r < kRows; r += 4) {
      const float4 y = sk[t][(r0 + r) / 4];
      const float kk[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        m[r + z].x = fmaf(kk[z], x.x, m[r + z].x);
        m[r + z].y = fmaf(kk[z], x.y, m[r + z].y);
        m[r + z].z = fmaf(kk[z], x.z, m[r + z].z);
        m[r + z].w = fmaf(kk[z], x.w, m[r + z].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) *reinterpret_cast<float4*>(a.s_out + at + (long long)r * DV) = m[r];
}

template <typename T, int DK, int DV>
cudaError_t window_launch(const LinArgs& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.o != nullptr)
    e = launch_pdl(linear_window_kernel<T, DK, DV>, dim3(a.H, a.B), dim3(DV * 2), 0, st, a);
  // behind the outputs: the two states may be one array
  if (e == cudaSuccess && a.s_out != nullptr)
    e = launch_pdl(linear_commit_kernel<T, DK, DV>, dim3(a.H * (DV / 64), a.B), dim3(kWinThreads), 0, st, a);
  return e;
}

template <typename T>
cudaError_t window_dispatch(const LinArgs& a, cudaStream_t st) {
  if (a.Dk == 128) return a.Dv == 128 ? window_launch<T, 128, 128>(a, st) : window_launch<T, 128, 64>(a, st);
  return a.Dv == 128 ? window_launch<T, 64, 128>(a, st) : window_launch<T, 64, 64>(a, st);
}

}  // namespace

cudaError_t launch_linear_window(int dtype, const LinArgs& a, cudaStream_t st) {
  return dtype == SDV_F16 ? window_dispatch<__half>(a, st) : window_dispatch<__nv_bfloat16>(a, st);
}

}  // namespace sdv

// tcgen05 building blocks of the token-mixing kernels: 128-byte-swizzled operand
// descriptors, single MMAs issued by one thread, 32-column tensor-memory accesses.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mixing.h"
#include "sdv_device.cuh"

namespace sdv {

// Operand tiles in shared memory are blocks of 64 16-bit elements (128 bytes) per
// row under the 128-byte swizzle: 16-byte chunk c of row r sits at chunk
// c ^ (r % 8), 8 rows (1024 bytes) to a swizzle atom.
__device__ __forceinline__ uint32_t swz128(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// Shared-memory matrix descriptor under the 128-byte swizzle.  K-major operand
// (64 reduction elements per row): sbo = 1024 between 8-row groups, lbo unused;
// 16 reduction elements further = 32 bytes further.  MN-major operand (64 rows
// or columns of the matrix per 128 bytes, one reduction index per row): sbo = 1024
// between groups of 8 reduction indices, lbo = bytes between 64-element blocks.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of this tensor-core generation
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// Instruction descriptor of kind::f16: 16-bit A and B of one type, fp32 D.
__host__ __device__ constexpr uint32_t idesc_16_f32(bool bf16, int m, int n, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn_major ? 1u << 15 : 0u) |
         (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Four MMAs (K = 16 each, 64 along the reduction) issued by one elected lane of a
// converged warp; operands are the same in every lane.  _ss: A and B in shared memory,
// DA and DB 16-byte units further each (a K-major operand under the 128-byte swizzle: 2,
// an MN-major one: 128); _ts: A in tensor memory, 8 columns further each, B MN-major.
// The first overwrites D unless `accumulate`.
template <int DA = 2, int DB = 2>
__device__ __forceinline__ void tc_mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 ta, tb;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.u64 ta, %1, %5;\n\tadd.u64 tb, %2, %8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ta, tb, %3, t;\n\t"
      "add.u64 ta, %1, %6;\n\tadd.u64 tb, %2, %9;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ta, tb, %3, t;\n\t"
      "add.u64 ta, %1, %7;\n\tadd.u64 tb, %2, %10;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], ta, tb, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(DA), "n"(2 * DA), "n"(3 * DA), "n"(DB), "n"(2 * DB), "n"(3 * DB)
      : "memory");
}
__device__ __forceinline__ void tc_mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 ta;\n\t.reg .b64 tb;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 ta, %1, 8;\n\tadd.u64 tb, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], tb, %3, t;\n\t"
      "add.u32 ta, %1, 16;\n\tadd.u64 tb, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], tb, %3, t;\n\t"
      "add.u32 ta, %1, 24;\n\tadd.u64 tb, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], tb, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Negates A in the product.
constexpr uint32_t kIdescNegateA = 1u << 13;

#define SDV_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), \
                     "=r"(v[o + 6]), "=r"(v[o + 7])
#define SDV_W8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), \
                     "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of a warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SDV_R8(v, 0), SDV_R8(v, 8), SDV_R8(v, 16), SDV_R8(v, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      SDV_W8(v, 0), SDV_W8(v, 8), SDV_W8(v, 16), SDV_W8(v, 24)
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               SDV_W8(v, 0)
               : "memory");
}
#undef SDV_R8
#undef SDV_W8

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// 3-D tiled TMA load of the box at (x, y, z).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// A bounded wait by a whole warp, in few instructions: the roles of one kernel share
// the SM's instruction cache, so what follows a first look in vain is one function for
// all of them.  On expiry the status word is set.  The limit stands in shared memory,
// where one thread has put it before the block's first barrier, so that the many places of
// a wait carry no argument for it.
constexpr int kWaitLimitBytes = 16;  // of static shared memory
__device__ __forceinline__ volatile uint64_t& wait_limit_ns() {
  __shared__ alignas(kWaitLimitBytes) volatile uint64_t limit;
  return limit;
}
__device__ __forceinline__ void set_wait_limit(const DebugFault& f) {
  wait_limit_ns() = f.wait_ns != 0 ? f.wait_ns : kWaitLimitNs;
}
static __device__ __noinline__ bool mbar_wait_on(uint32_t bar, uint32_t parity, int* status) {
  const uint64_t t0 = global_timer_ns();
  do {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  } while (__all_sync(0xffffffffu, global_timer_ns() - t0 < wait_limit_ns()));
  if ((threadIdx.x & 31) == 0) atomicOr(status, 1 /* kDevErrTimeout */);
  return false;
}
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || mbar_wait_on(bar, parity, status);
}

// Four bytes into shared memory behind the thread's back, zeros where `real` is false.
__device__ __forceinline__ void cp_async4(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// L2 policy of data that other CTAs read too.
__device__ __forceinline__ uint64_t l2_policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction, on register pairs.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair2(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two floats to a packed pair of the 16-bit type (a in the low half).
template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(f32x2 x) {
  const float2 y = unpair2(x);
  return pack16<T>(y.x, y.y);
}

// A packed pair to two floats.
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Whether either half of a packed pair is an infinity or NaN: bits of the halves that are.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite16(uint32_t x);
template <>
__device__ __forceinline__ uint32_t nonfinite16<__half>(uint32_t x) {
  return ((x & 0x7C00u) == 0x7C00u ? 1u : 0u) | ((x & 0x7C000000u) == 0x7C000000u ? 2u : 0u);
}
template <>
__device__ __forceinline__ uint32_t nonfinite16<__nv_bfloat16>(uint32_t x) {
  return ((x & 0x7F80u) == 0x7F80u ? 1u : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 2u : 0u);
}

}  // namespace sdv

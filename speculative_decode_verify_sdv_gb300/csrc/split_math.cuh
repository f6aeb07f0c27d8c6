// Arithmetic of the work splits that live on the device.
#pragma once

namespace sdv {

// x * y / z and x / z with small numbers (the common case) in 32 bits: a 64-bit
// division takes most of a microsecond of a lone warp's time.
static __device__ __noinline__ long long div_long(unsigned long long p, unsigned long long z) { return (long long)(p / z); }

__device__ __forceinline__ long long div_fast(unsigned long long p, unsigned long long z) {
  return (p | z) >> 32 == 0 ? (long long)((unsigned)p / (unsigned)z) : div_long(p, z);
}
__device__ __forceinline__ long long muldiv(long long x, int y, long long z) {
  return div_fast((unsigned long long)x * (unsigned)y, z);
}

}  // namespace sdv

// Masses floor(w 2^40) of weights w in [0, 1], their sums, and the goal of a draw among them; packed float32 pairs.
#pragma once

#include "common.cuh"
#include "verify_common.cuh"

namespace dspark {

__device__ __forceinline__ unsigned long long f32x2_add(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long f32x2_mul(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long f32x2_add_rz(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long f32x2_fma_rz(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Sum of floor(w 2^40) over weights in [0, 1], as two sums of 20-bit halves: adding 8 with rounding
// towards zero leaves floor(w 2^20) in the low mantissa bits, and what it cut off gives the other half.
// Up to 2^11 weights fit.
struct MassPair {  // the two halves of two masses, above the bits of 8
  uint32_t hi[2], lo[2];
  __device__ __forceinline__ MassPair(float w0, float w1) {
    const unsigned long long w = f32x2_pack(w0, w1), eight = f32x2_pack(8.f, 8.f);
    const unsigned long long a = f32x2_add_rz(w, eight);
    const unsigned long long cut = f32x2_add(a, f32x2_pack(-8.f, -8.f));                  // exact
    const unsigned long long rest = f32x2_fma(cut, f32x2_pack(-1.f, -1.f), w);             // exact
    const unsigned long long b = f32x2_fma_rz(rest, f32x2_pack(0x1p20f, 0x1p20f), eight);
    float x, y;
    f32x2_unpack(a, x, y);
    hi[0] = __float_as_uint(x);
    hi[1] = __float_as_uint(y);
    f32x2_unpack(b, x, y);
    lo[0] = __float_as_uint(x);
    lo[1] = __float_as_uint(y);
  }
};
struct MassSum {
  uint32_t hi = 0, lo = 0, n = 0;  // n of the masses were added with the bits of 8
  __device__ __forceinline__ void add(const MassPair& m) {
    hi += m.hi[0] + m.hi[1];
    lo += m.lo[0] + m.lo[1];
    n += 2;
  }
  __device__ __forceinline__ void add_if(const MassPair& m, bool p0, bool p1) {
    const uint32_t k0 = p0 ? 0x7fffffu : 0u, k1 = p1 ? 0x7fffffu : 0u;
    hi += (m.hi[0] & k0) + (m.hi[1] & k1);
    lo += (m.lo[0] & k0) + (m.lo[1] & k1);
  }
  __device__ __forceinline__ unsigned long long total() const {
    const uint32_t eights = n * 0x41000000u;
    return ((unsigned long long)(hi - eights) << 20) + (lo - eights);
  }
};

// floor(x S) for x in [0, 1), x to 53 bits, from the bits of x (FP64 instructions are slow here)
__device__ __forceinline__ unsigned long long scale_mass(double x, unsigned long long S) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(x), one = 1ull << 53;
  const int e = (int)(b >> 52);  // sign and exponent
  const unsigned long long m = (b & ((1ull << 52) - 1)) | (1ull << 52);
  // negative, NaN: 0; 1 and above: the largest below 1
  const unsigned long long k = e >= 0x7ff ? 0ull : e >= 1023 ? one - 1 : e < 1023 - 54 ? 0ull : m >> (1022 - e);
  return scale_u53(k, S);
}

}  // namespace dspark

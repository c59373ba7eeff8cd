// Quotients by a quantisation scale, and the codes of symmetric int8 rows.  Host and device: a CPU test
// compiles the same source and compares it with whole-number arithmetic.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace moe {

// A row's (or group's) quantisation scale, prepared for quotients v / s.  k: a power of two that keeps
// s normal and 1 / s finite.
struct Scale {
  float s, r, k;  // s and 1 / s, both times / over k
  __host__ __device__ __forceinline__ explicit Scale(float sc) {
    k = sc < 0x1p-60f ? 0x1p64f : 1.0f;
    s = sc * k;
    r = 1.0f / s;
  }
  // fp32(v / s): the product by the reciprocal, corrected by its remainder (which is +0 for a zero of
  // either sign, so the sign is put back)
  __host__ __device__ __forceinline__ float div(float v) const {
    v *= k;
    const float q = v * r;
    return copysignf(fmaf(fmaf(-q, s, v), r, q), v);
  }
  // v / s rounded to a whole number in [-127, 127], ties to even: the rounded product is at most one off, and the
  // remainder, exact in fp32 (a multiple of half an ulp of s, at most s), says so.  (Rounding fp32(v / s)
  // would not do: amax / 2 over s is 63.4999999, and comes out as 63.5 and then 64.)  A remainder of
  // exactly half of s is a tie, and an odd n then goes to the even side: with 1 / s rounded (s of few bits
  // but no power of two) the product may lie on either side of it.
  __host__ __device__ __forceinline__ int whole(float v) const {
    v *= k;
    const float n = __builtin_rintf(v * r), e = fmaf(-n, s, v), h = 0.5f * s;
    const int i = (int)n;
    const bool off = fabsf(e) > h || (fabsf(e) == h && (i & 1));
    const int q = i + (off ? (e > 0.0f ? 1 : -1) : 0);
    return q > 127 ? 127 : q < -127 ? -127 : q;
  }
};

// Symmetric int8 rows: s = fp32(amax / 127) (1 when amax is 0 or the quotient underflows to 0; NaN
// when amax is not finite, so that whatever is multiplied by it shows it).  |v| <= amax keeps |v| / s
// below 127 (1 + 2^-23), but for a subnormal s of few bits, where it may reach 190: whole() cuts it at 127.
__host__ __device__ __forceinline__ float i8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __builtin_bit_cast(float, 0x7FC00000u);
  const float s = __builtin_bit_cast(float, amax_bits) / 127.0f;
  return s == 0.0f ? 1.0f : s;
}
// Four codes in a dword.
__host__ __device__ __forceinline__ uint32_t i8_pack4(const float* v, const Scale& sc) {
  uint32_t p = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) p |= (uint32_t(sc.whole(v[i])) & 0xFFu) << (8 * i);
  return p;
}

}  // namespace moe

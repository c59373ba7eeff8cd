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
  // v / s rounded to a whole number, ties to even, |v| / s < 127.5: the rounded product is at most one off,
  // and the remainder, exact in fp32 (a multiple of half an ulp of s, at most s), says so.  (Rounding
  // fp32(v / s) would not do: amax / 2 over s is 63.4999999, and comes out as 63.5 and then 64.)
  // A remainder of exactly half of s is a tie, and an odd n then goes to the even side: with 1 / s rounded
  // (s of few bits but no power of two) the product may lie on either side of it.  BF16 rows have no such
  // ties: fp32(amax / 127) of a bf16 amax has few bits only as a power of two, whose reciprocal is exact,
  // so the product is the tie and rounds to even.
  template <bool BF16>
  __host__ __device__ __forceinline__ int whole(float v) const {
    v *= k;
    const float n = __builtin_rintf(v * r), e = fmaf(-n, s, v), h = 0.5f * s;
    const int i = (int)n;
    if (BF16) return i + (e > h ? 1 : 0) - (e < -h ? 1 : 0);
    // (over half: a positive difference, or none and an odd n)
    const int over = __builtin_bit_cast(int, fmaf(2.0f, fabsf(e), -s)) + (i & 1);
    return i + (over > 0 ? (__builtin_bit_cast(int, e) >> 31 | 1) : 0);
  }
};

// Symmetric int8 rows: s = fp32(amax / 127) (1 when amax is 0 or the quotient underflows to 0; NaN
// when amax is not finite, so that whatever is multiplied by it shows it).  A subnormal s has few bits, and
// amax over it may reach 190: where it would round past 127, s is the next float up.  So |v| <= amax keeps
// |v| / s below 127.5 and the codes in [-127, 127].
__host__ __device__ __forceinline__ float i8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __builtin_bit_cast(float, 0x7FC00000u);
  const float amax = __builtin_bit_cast(float, amax_bits), s = amax / 127.0f;
  if (s >= 0x1p-126f) return s;
  if (s == 0.0f) return 1.0f;
  return fmaf(s * 0x1p64f, 127.5f, -amax * 0x1p64f) > 0.0f
             ? s
             : __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, s) + 1);
}
// 4 N codes, four in a dword.  For fp32 rows a value's nearest whole number is taken from its product with r
// and counts unless v / s, from r and what it is off, lies within 2^-23 of a half step; then all of them are
// found from their remainders.  (That for every value: the norm of 4096 rows of 4096 19.7 us against 17.5, of
// 16 rows of 7168 4.5 against 4.2; h of 8192 x 14336 98.9 against 96.7.)  bf16 rows hold +-amax / 2, which is
// near a half step, every few hundred values, and the remainders' way is the faster (2048 rows of 4096 8.0
// us against 10.5).
template <int N, bool BF16>
__host__ __device__ __forceinline__ void i8_pack(const float* v, const Scale& sc, uint32_t* out) {
  constexpr float kWhole = 0x1.8p23f;  // added, it leaves whole numbers: the sum's low byte is the code
  uint32_t c[4 * N];
  float far = BF16 ? 1.0f : 0.0f;
  if (!BF16) {
    const float lo = fmaf(-sc.s, sc.r, 1.0f) * sc.r;  // 1 / s - r
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      const float a = v[i] * sc.k, t = fmaf(a, sc.r, kWhole);
      c[i] = __builtin_bit_cast(uint32_t, t);
      // (the product less the whole number is exact but for its last bit, 2^-25 at most)
      far = fmaxf(far, fabsf(fmaf(a, lo, fmaf(a, sc.r, kWhole - t))));
    }
  }
  if (far > 0.5f - 0x1p-23f) {
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) c[i] = (uint32_t)sc.whole<BF16>(v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    out[i] = (c[4 * i] & 0xFFu) | (c[4 * i + 1] & 0xFFu) << 8 | (c[4 * i + 2] & 0xFFu) << 16 | c[4 * i + 3] << 24;
}

}  // namespace moe

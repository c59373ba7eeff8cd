// Pieces of the norm kernels (norm.hip, block_norm.hip): a row's reciprocal root in and out of fp32's
// range, and conversions.
#pragma once

#include "rows_dev.h"

namespace moe {

enum NormFormat { kNormBf16 = 0, kNormFp8 = 1, kNormMx = 2, kNormI8 = 3 };

// Four e4m3 codes in a dword, by the conversion instruction: to nearest, ties to even, the sign kept.
// It equals e4m3_encode on values up to 448 in magnitude and does not saturate above 464, so the caller
// limits its values.
__device__ __forceinline__ uint32_t e4m3_pack4(const float* v) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
}

// A vector through an opaque move (computations on it stay where they are written).
__device__ __forceinline__ uint4 opaque(uint4 v) {
  asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
  return v;
}

// Whether fp32 held the squares of a row: its mean square (with eps) is finite and so far above
// the smallest float that what underflowed does not count (2^-149 a term against 2^-100).
__device__ __forceinline__ bool row_in_range(double sum, double inv_d, float eps) {
  const float m = float(sum * inv_d) + eps;
  return m >= 0x1p-100f && m < __uint_as_float(kInfBits);
}
// 1 / sqrt(sum / d + eps) of a row in range.
__device__ __forceinline__ float row_rstd(double sum, double inv_d, float eps) {
  return 1.0f / sqrtf(float(sum * inv_d) + eps);
}
// The same rounded once instead of four times: the instruction's root, and a Newton step in fp64.
__device__ __forceinline__ float row_rstd_once(double sum, double inv_d, float eps) {
  const double m = fma(sum, inv_d, (double)eps), r = (double)__builtin_amdgcn_rsqf((float)m);
  return (float)fma(0.5 * r, fma(-m * r, r, 1.0), r);
}
// The same of any row, from squares summed in fp64 (which bf16's never leave): for a small row the value
// over 2^32, which kSmallRow times the row's values make good; NaN for a row that holds an infinity or
// NaN, so that the whole row shows it (and for a zero row without eps, 0 / 0).
constexpr float kSmallRow = 0x1p32f;
__device__ __forceinline__ float wide_rstd(double sum, double inv_d, float eps, bool& small) {
  const double m = sum * inv_d + (double)eps;
  small = m < 0x1p-100;
  if (small) return 0x1p68f / sqrtf(float(m * 0x1p200));
  if (m <= 0x1p100) return 1.0f / sqrtf(float(m));  // (the gradient's products may leave the range alone)
  return m < __builtin_inf() ? 0x1p-100f / sqrtf(float(m * 0x1p-200)) : __uint_as_float(0x7FC00000u);
}

// The wide sums of a row out of range, two values at a time in a loop, and its values times kSmallRow
// (exact: a small row's are below 2^-42): a path that must not cost the other one registers.
__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }
__device__ __forceinline__ uint4 turned(const uint4& v) { return make_uint4(v.y, v.z, v.w, v.x); }
__device__ __forceinline__ void add_squares(uint4 h, double& sum) {
#pragma unroll 1
  for (int j = 0; j < 4; ++j, h = turned(h)) {
    const double a = bf16_lo(h.x), b = bf16_hi(h.x);
    sum = fma(b, b, fma(a, a, sum));
  }
}
__device__ __forceinline__ void add_products(uint4 h, uint4 g, uint4 w, double& sum) {
#pragma unroll 1
  for (int j = 0; j < 4; ++j, h = turned(h), g = turned(g), w = turned(w)) {
    sum = fma((double)bf16_lo(g.x) * (double)bf16_lo(w.x), (double)bf16_lo(h.x), sum);
    sum = fma((double)bf16_hi(g.x) * (double)bf16_hi(w.x), (double)bf16_hi(h.x), sum);
  }
}
__device__ __forceinline__ uint4 enlarged(uint4 h) {
#pragma unroll 1
  for (int j = 0; j < 4; ++j, h = turned(h))
    h.x = pack_bf16x2(bf16_lo(h.x) * kSmallRow, bf16_hi(h.x) * kSmallRow);
  return h;
}

// Column sums of part [nb][d] by workgroups of 256 threads: 32 columns each (whole 128-byte lines), its 32 groups of
// 8 threads take every 32nd partial, 16 in fp32 at a time and those in fp64 (one time for up to 512 partials).
// red[g][c]: group g's sum of the workgroup's column c, 0 past d (d % 4 == 0), behind a barrier.
__device__ __forceinline__ void sum_parts(const float* __restrict__ part, int nb, int d, float (*red)[33]) {
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, col = blockIdx.x * 32 + c * 4;
  double t[4] = {0.0, 0.0, 0.0, 0.0};
  if (col < d) {
    for (int b0 = r; b0 < nb; b0 += 16 * 32) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int b = b0; b < min(b0 + 16 * 32, nb); b += 32) {
        const uint4 v = ld16(part, ((size_t)b * d + col) / 4);
        s[0] += __uint_as_float(v.x);
        s[1] += __uint_as_float(v.y);
        s[2] += __uint_as_float(v.z);
        s[3] += __uint_as_float(v.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] += (double)s[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[r][c * 4 + j] = (float)t[j];
  __syncthreads();
}

}  // namespace moe

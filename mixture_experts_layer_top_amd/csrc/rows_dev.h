// Pieces of the row kernels (norm, int8 row quantisation, combine gradient): a row of d bf16 or fp32
// values is spread over R threads, 8 consecutive values (one 16-byte bf16 vector) per thread and
// step, V steps, and stays in registers between the passes over it.
#pragma once

#include "common.h"

namespace moe {

// Longest row: 512 threads x 8 steps x 8 values.
constexpr int kMaxRow = 32768;

// Threads (R) and steps (V) for a row of nvec 8-value vectors: one wavefront while 8 steps are
// enough (no barrier), then the fewest wavefronts; V is the row's own step count, so no step is
// empty.  Calls f with both as integral constants.  nvec <= kMaxRow / 8.
template <int R, int V, int VMAX, class F>
inline void with_steps(int v, F&& f) {
  if constexpr (V < VMAX) {
    if (v > V) return with_steps<R, V + 1, VMAX>(v, f);
  }
  f(std::integral_constant<int, R>{}, std::integral_constant<int, V>{});
}
template <class F>
inline void with_row_shape(int nvec, F&& f) {
  if (nvec <= 64 * 8) with_steps<64, 1, 8>((nvec + 63) / 64, f);
  else if (nvec <= 128 * 8) with_steps<128, 5, 8>((nvec + 127) / 128, f);
  else if (nvec <= 256 * 8) with_steps<256, 5, 8>((nvec + 255) / 256, f);
  else with_steps<512, 5, 8>((nvec + 511) / 512, f);
}

// Threads per workgroup: four one-wavefront rows, else one row.
constexpr int row_block(int R) { return R == 64 ? 256 : R; }

__device__ __forceinline__ void unpack8(const uint4& v, float (&o)[8]) {
  const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(p[i] << 16);
    o[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint4 o;
  o.x = pack_bf16x2(v[0], v[1]);
  o.y = pack_bf16x2(v[2], v[3]);
  o.z = pack_bf16x2(v[4], v[5]);
  o.w = pack_bf16x2(v[6], v[7]);
  return o;
}
__device__ __forceinline__ uint4 ld16(const void* base, size_t vec) {
  const u32x4 v = reinterpret_cast<__attribute__((address_space(1))) const u32x4*>((gchar*)base)[vec];
  return __builtin_bit_cast(uint4, v);
}
__device__ __forceinline__ void st16(void* base, size_t vec, const uint4& v) {
  reinterpret_cast<__attribute__((address_space(1))) u32x4*>((gwchar*)base)[vec] =
      __builtin_bit_cast(u32x4, v);
}
__device__ __forceinline__ void st8(void* base, size_t off, uint32_t a, uint32_t b) {
  gstore8(base, off, uint2{a, b});
}

// Sums (or maxima) of NA values over the R threads of a row, the same in every thread and in a
// fixed order: a butterfly in each wavefront, then the wavefronts' results in order from LDS.
// red: NA * R / 64 values of its own for every call (no barrier protects a second use).
template <int R, int NA, class T, class Op>
__device__ __forceinline__ void row_reduce(T (&v)[NA], T* red, Op op) {
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v[i] = op(v[i], __shfl_xor(v[i], o));
  if constexpr (R > 64) {
    constexpr int W = R / 64;
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NA; ++i) red[i * W + wv] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      v[i] = red[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] = op(v[i], red[i * W + w]);
    }
  }
}
struct SumOp {
  template <class T> __device__ T operator()(T a, T b) const { return a + b; }
};
struct MaxOp {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// Magnitudes are compared as the bits of |v|: their unsigned order is the magnitudes' order with
// infinity above every number and NaN above infinity, so a maximum never drops a NaN.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// Largest value of each aligned group of 4 (or 16) lanes, in every lane of the group.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));  // quad_perm [1,0,3,2]
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));  // quad_perm [2,3,0,1]
  if (LANES == 16) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, false));  // row_half_mirror
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xf, 0xf, false));  // row_mirror
  }
  return m;
}

// Symmetric int8 rows: s = fp32(amax / 127) (1 when amax is 0 or the quotient underflows to 0; NaN
// when amax is not finite, so that whatever is multiplied by it shows it), q = round(v / s) to
// nearest, ties to even.  Both quotients go through float64: amax / 127 is then correctly rounded to
// fp32 (53 >= 2 * 24 + 2); v * (1 / s) differs from the exact quotient by 2^-52 of it and is rounded
// to a whole number from there (through fp32, amax / 2 over s = 63.4999999 would come out as 64).  A
// quotient that is exactly a half step needs an s of few bits, and fp32(amax / 127) of a bf16 amax
// has few bits only as a power of two, whose reciprocal is exact.
__device__ __forceinline__ float i8_scale(uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return __uint_as_float(0x7FC00000u);
  const float s = float(double(__uint_as_float(amax_bits)) / 127.0);
  return s == 0.0f ? 1.0f : s;
}
// Four codes in a dword.  |v| <= amax, so |v / s| <= 127 (1 + 2^-24): the rounding cannot reach 128.
__device__ __forceinline__ uint32_t i8_pack4(const float* v, double inv) {
  uint32_t p = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p |= (uint32_t(int(__builtin_rint(double(v[i]) * inv))) & 0xFFu) << (8 * i);
  return p;
}

}  // namespace moe

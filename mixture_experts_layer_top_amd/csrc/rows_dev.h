// Pieces of the row kernels (norm, int8 row quantisation, combine gradient): a row of d bf16 or fp32
// values is spread over R threads, 8 consecutive values (one 16-byte bf16 vector) per thread and
// step, V steps, and stays in registers between the passes over it.
#pragma once

#include "common.h"
#include "i8_codec.h"

namespace moe {

// Longest row: 512 threads x 8 steps x 8 values.
constexpr int kMaxRow = 32768;

// Threads (R) and steps (V) for a row of nvec 8-value vectors: one wavefront while 8 steps are
// enough (no barrier), then the fewest wavefronts; V is the row's own step count, so no step is
// empty.  Few rows (`few`: a decode batch leaves most CUs idle) take a wavefront per 64 or 128 vectors
// instead: a row's latency is then one or two loads deep.  Calls f with both as integral constants.
// nvec <= kMaxRow / 8.
template <int R, int V, int VMAX, class F>
inline void with_steps(int v, F&& f) {
  if constexpr (V < VMAX) {
    if (v > V) return with_steps<R, V + 1, VMAX>(v, f);
  }
  f(std::integral_constant<int, R>{}, std::integral_constant<int, V>{});
}
template <class F>
inline void with_row_shape(int nvec, bool few, F&& f) {
  if (few && nvec > 64) {
    if (nvec <= 256) with_steps<256, 1, 1>(1, f);
    else if (nvec <= 512) with_steps<512, 1, 1>(1, f);
    else if (nvec <= 1024) with_steps<512, 2, 2>(2, f);
    else if (nvec <= 4096) with_steps<1024, 2, 4>((nvec + 1023) / 1024, f);
    return;
  }
  if (nvec <= 64 * 8) with_steps<64, 1, 8>((nvec + 63) / 64, f);
  else if (nvec <= 128 * 8) with_steps<128, 5, 8>((nvec + 127) / 128, f);
  else if (nvec <= 256 * 8) with_steps<256, 5, 8>((nvec + 255) / 256, f);
  else with_steps<512, 5, 8>((nvec + 511) / 512, f);
}
// (Four rows per CU.  The norm with e4m3 rows of 7168, this shape against the other: 1 row 3.5 and 5.4 us, 512
// 7.4 and 9.5, 768 9.2 and 10.6, 1024 11.1 and 12.4; the int8 quantisation 2.6 and 3.6, 4.1 and 5.1, 4.9
// and 5.4, 5.9 and 5.9; at 2048 rows of 2048 4.5 and 4.2.)
constexpr int kFewRows = 1024;

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
// The same for rows that are read or written once: non-temporal, so that they push nothing out of L2.
__device__ __forceinline__ uint4 ld16_once(const void* base, size_t vec) {
  const u32x4 v = __builtin_nontemporal_load(
      reinterpret_cast<__attribute__((address_space(1))) const u32x4*>((gchar*)base) + vec);
  return __builtin_bit_cast(uint4, v);
}
__device__ __forceinline__ void st16_once(void* base, size_t vec, const uint4& v) {
  gstore16_nt(base, vec * 16, v);
}
__device__ __forceinline__ void st8(void* base, size_t off, uint32_t a, uint32_t b) {
  gstore8(base, off, uint2{a, b});
}

// One lane exchange inside rows of 16 lanes (DPP), for values of 4 or 8 bytes.
template <int CTRL, class T>
__device__ __forceinline__ T dpp16(T v) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
  } else {
    return __builtin_bit_cast(
        T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
  }
}
template <class T>
__device__ __forceinline__ T read_lane(T v, int lane) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}
// Over aligned groups of 16 lanes, in every lane: neighbours, pairs, mirrored halves, mirrored rows.
template <class T, class Op>
__device__ __forceinline__ T reduce16(T v, Op op) {
  v = op(v, dpp16<0xb1>(v));   // quad_perm [1,0,3,2]
  v = op(v, dpp16<0x4e>(v));   // quad_perm [2,3,0,1]
  v = op(v, dpp16<0x141>(v));  // row_half_mirror
  return op(v, dpp16<0x140>(v));  // row_mirror
}

// Sums (or maxima) of NA values over the R threads of a row, the same in every thread and in a
// fixed order: rows of 16 lanes, the four rows of a wavefront, then the wavefronts through LDS.
// red: NA * R / 64 values of its own for every call (no barrier protects a second use).
template <int R, int NA, class T, class Op>
__device__ __forceinline__ void row_reduce(T (&v)[NA], T* red, Op op) {
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    v[i] = reduce16(v[i], op);
    v[i] = op(op(read_lane(v[i], 0), read_lane(v[i], 16)), op(read_lane(v[i], 32), read_lane(v[i], 48)));
  }
  if constexpr (R > 64) {
    constexpr int W = R / 64;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < NA; ++i) red[i * W + wv] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NA; ++i) {  // (W <= 16: lane l of each row of 16 takes wavefront l's, or 0)
      const int l = lane & 15;
      v[i] = l < W ? red[i * W + l] : T(0);
      v[i] = read_lane(reduce16(v[i], op), 0);
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
  if (LANES == 16) return reduce16(m, MaxOp{});
  m = max(m, dpp16<0xb1>(m));
  return max(m, dpp16<0x4e>(m));
}

}  // namespace moe

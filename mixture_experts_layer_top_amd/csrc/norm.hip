// RMS norm in front of the layer, with the residual's addition and an 8-bit output, its gradient,
// and the int8 row quantisation.
//
//   h = bf16(x + r) (h = x without a residual), n = h / sqrt(mean(h^2) + eps), y = n * w
//   outputs: h, bf16(y), and y in the activation format of the experts' weights (from the fp32 y,
//   one rounding): e4m3 with an fp32 scale per 128 channels, e4m3 with an E8M0 scale per 32, or
//   int8 with an fp32 scale per row.
// gradient (g = dy * w, dh the gradient that arrives at h on the residual path):
//   dx = (g - n * mean(g * n)) / sqrt(mean(h^2) + eps) + dh, for x and for r alike
//   dw[c] = sum_t dy[t][c] * n[t][c]
//
// All of it is bound by HBM: a row is read once into registers, both passes over it (the sum of
// squares, then the scaling) run from there, and the 8-bit output costs no second read of y.  The
// sum of squares is held in fp64 across a row, over fp32 chains of eight; a row whose squares leave
// fp32's range (row_in_range) is summed again in fp64 from its registers.  Forward with a residual and e4m3
// rows: 8192 x 7168 98 us (5.4 TB/s, a copy's rate), 1 x 7168 3.4 us.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "mx_codec.h"
#include "rows_dev.h"

namespace moe {

namespace {

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

template <int FMT, int R, int V>
__global__ __launch_bounds__(row_block(R)) void rmsnorm_kernel(
    const void* x, const void* res, const void* __restrict__ w, float eps, double inv_d, int T,
    int nvec, void* h_out, void* y, uint8_t* q, void* qs) {
  __shared__ double red[2][R / 64];
  __shared__ uint32_t redm[R / 64];
  const int row = R == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (R == 64 && row >= T) return;  // (whole wavefronts; no barrier in this form)
  const int i = R == 64 ? threadIdx.x & 63 : threadIdx.x;
  const size_t base = (size_t)row * nvec;
  uint4 hv[V], rv[V], wr[V];
#pragma unroll
  for (int s = 0; s < V; ++s) hv[s] = ld16(x, base + min(i + R * s, nvec - 1));
  if (res) {
#pragma unroll
    for (int s = 0; s < V; ++s) rv[s] = ld16(res, base + min(i + R * s, nvec - 1));
  }
#pragma unroll
  for (int s = 0; s < V; ++s) wr[s] = ld16(w, min(i + R * s, nvec - 1));
  double sum[1] = {0.0};
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const bool in = i + R * s < nvec;
    float h[8];
    unpack8(hv[s], h);
    if (res) {
      float r[8];
      unpack8(rv[s], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] += r[j];
      hv[s] = pack8(h);
      unpack8(hv[s], h);
    }
    if (in) {
      if (h_out) st16(h_out, base + i + R * s, hv[s]);
      float p = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) p = fmaf(h[j], h[j], p);
      sum[0] += (double)p;
    }
  }
  row_reduce<R>(sum, red[0], SumOp{});
  float rstd = row_rstd(sum[0], inv_d, eps);
  if (!row_in_range(sum[0], inv_d, eps)) {  // (the same in all threads of the row)
    sum[0] = 0.0;
#pragma unroll
    for (int s = 0; s < V; ++s)
      if (i + R * s < nvec) add_squares(hv[s], sum[0]);
    row_reduce<R>(sum, red[1], SumOp{});
    bool small;
    rstd = wide_rstd(sum[0], inv_d, eps, small);
    if (small) {
#pragma unroll
      for (int s = 0; s < V; ++s) hv[s] = enlarged(hv[s]);
    }
  }
  auto yvec = [&](int s, float (&v)[8]) {
    float wv[8];
    unpack8(wr[s], wv);
    unpack8(hv[s], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * wv[j];
  };
  Scale row_scale(1.0f);
  bool bad_row = false;
  if (FMT == kNormI8) {
    uint32_t m[1] = {0u};
#pragma unroll
    for (int s = 0; s < V; ++s) {
      float v[8];
      yvec(s, v);
      if (i + R * s < nvec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[0] = max(m[0], abs_bits(v[j]));
      }
    }
    row_reduce<R>(m, redm, MaxOp{});
    const float sc = i8_scale(m[0]);
    bad_row = m[0] >= kInfBits;  // (scale NaN, codes 0)
    row_scale = Scale(bad_row ? 1.0f : sc);
    if (i == 0) static_cast<float*>(qs)[row] = sc;
  }
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int idx = i + R * s;
    float v[8];
    yvec(s, v);
    uint32_t m = 0u;
    if (FMT == kNormFp8 || FMT == kNormMx) {
      // (the 16 or 4 lanes of a scale group are in or out together: d % 128 == 0, d % 32 == 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
      m = group_max<FMT == kNormFp8 ? 16 : 4>(m);
    }
    if (idx >= nvec) continue;
    if (y) st16(y, base + idx, pack8(v));
    if (FMT == kNormI8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = bad_row ? 0.f : v[j];
      uint32_t c[2];
      i8_pack<2, false>(v, row_scale, c);
      st8(q, (base + idx) * 8, c[0], c[1]);
    }
    if (FMT == kNormFp8 || FMT == kNormMx) {
      const bool bad = m >= kInfBits;
      if (FMT == kNormFp8) {
        float sc = __uint_as_float(m) / 448.0f;
        if (sc == 0.0f || bad) sc = 1.0f;
        if ((idx & 15) == 0) static_cast<float*>(qs)[base / 16 + idx / 16] = sc;
        const Scale f(sc);
        // (a subnormal scale holds few bits: amax over it may reach 670, and saturates)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(f.div(v[j]), -448.0f, 448.0f);
      } else {
        const int X = bad ? 127 : mx_scale_code(__uint_as_float(m));
        if ((idx & 3) == 0) gstore_u8(static_cast<uint8_t*>(qs), base / 4 + idx / 4, X);
        const float f = mx_inv_scale(X);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
      }
      uint32_t p[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) p[j] = e4m3_pack4(v + 4 * j);
      if (bad) p[0] = p[1] = 0x7F7F7F7Fu;  // NaN codes
      st8(q, (base + idx) * 8, p[0], p[1]);
    }
  }
}

// x [T][d] bf16 or fp32 -> int8 rows and their scales.  A thread takes 16 bytes of x per load (8 bf16
// values or 4 fp32), so that a wavefront's loads are whole lines in both.  The fp32 rows are a scratch
// of the experts, read here for the last time, past the caches: 8192 x 14336 98 us (6.0 TB/s), 114
// with plain loads; 512 x 2048 4.8 us either way.
template <bool F32, int R, int V>
__global__ __launch_bounds__(row_block(R)) void quant_i8_kernel(const void* __restrict__ x, int T,
                                                                int nvec, uint8_t* __restrict__ q,
                                                                float* __restrict__ qs) {
  constexpr int N = F32 ? 4 : 8, L = F32 ? 2 * V : V;
  __shared__ uint32_t redm[R / 64];
  const int row = R == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (R == 64 && row >= T) return;
  const int i = R == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int n = F32 ? 2 * nvec : nvec;
  const size_t base = (size_t)row * n;
  uint4 a[L];
#pragma unroll
  for (int s = 0; s < L; ++s) {
    const size_t idx = base + min(i + R * s, n - 1);
    a[s] = F32 ? ld16_once(x, idx) : ld16(x, idx);
  }
  auto vec = [&](int s, float (&v)[N]) {
    if constexpr (F32) {
      const uint32_t p[4] = {a[s].x, a[s].y, a[s].z, a[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(p[j]);
    } else {
      unpack8(a[s], v);
    }
  };
  uint32_t m[1] = {0u};  // (clamped loads repeat a value of the row: the maximum is unchanged)
#pragma unroll
  for (int s = 0; s < L; ++s) {
    float v[N];
    vec(s, v);
#pragma unroll
    for (int j = 0; j < N; ++j) m[0] = max(m[0], abs_bits(v[j]));
  }
  row_reduce<R>(m, redm, MaxOp{});
  const float sc = i8_scale(m[0]);
  const bool bad = m[0] >= kInfBits;
  const Scale f(bad ? 1.0f : sc);
  if (i == 0) qs[row] = sc;
#pragma unroll
  for (int s = 0; s < L; ++s) {
    if (i + R * s >= n) continue;
    float v[N];
    vec(s, v);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = bad ? 0.f : v[j];
    const size_t at = (base + i + R * s) * N;
    uint32_t c[N / 4];
    i8_pack<N / 4, !F32>(v, f, c);
    if constexpr (F32) gstore4(q, at, c[0]);
    else st8(q, at, c[0], c[1]);
  }
}

// Norm gradient: every workgroup takes rows blockIdx.x, + gridDim.x, ... and keeps its share of dw
// in registers; part [gridDim.x][d] receives it (summed by dw_reduce_kernel, in a fixed order).
// Up to 4096 channels the next row is loaded while this one is reduced (two rows do not fit the
// registers beyond that).  Both kernels, T x d: 4096 x 4096 with dh 29.4 us (4.6 TB/s; without
// the second row in flight and with 8 columns a workgroup in the sum 30.5 where it took 28.3), 8192 x 7168
// with dh 94.8 (4.96), 777 x 7168 15.3 (21.3 where it took 15.2).
template <int R, int V>
__global__ __launch_bounds__(R) void rmsnorm_grad_kernel(
    const void* dy, const void* dh, const void* h, const void* __restrict__ w, float eps,
    double inv_d, int T, int nvec, void* dx, float* __restrict__ part) {
  __shared__ double red[4][2 * R / 64];
  const int i = threadIdx.x;
  float dw[V][8];
#pragma unroll
  for (int s = 0; s < V; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[s][j] = 0.f;
  // the row's vectors, and the next row's in flight while this one is reduced and written
  struct Row { uint4 h[V], g[V], a[V]; };
  auto load = [&](Row& r, int row) {
    const size_t base = (size_t)row * nvec;
#pragma unroll
    for (int s = 0; s < V; ++s) {
      const size_t idx = base + min(i + R * s, nvec - 1);
      r.h[s] = ld16(h, idx);
      r.g[s] = ld16(dy, idx);
      if (dh) r.a[s] = ld16(dh, idx);
    }
  };
  uint4 wr[V];
#pragma unroll
  for (int s = 0; s < V; ++s) wr[s] = ld16(w, min(i + R * s, nvec - 1));
  constexpr bool kAhead = V <= 2;  // (more vectors a thread: no registers for a second row)
  Row cur, nxt;
  if (kAhead) load(cur, blockIdx.x);
  int turn = 0;
  for (int row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
    const bool more = row + (int)gridDim.x < T;
    // (dx may be dy or dh: a row's own vectors are all loaded before it is written, and no other row's
    // are written by this call before their workgroup has loaded them)
    if (!kAhead) load(cur, row);
    else if (more) load(nxt, row + gridDim.x);
    double sum[2] = {0.0, 0.0};
#pragma unroll
    for (int s = 0; s < V; ++s) {
      float a[8], g[8], wv[8];
      unpack8(cur.h[s], a);
      unpack8(cur.g[s], g);
      unpack8(wr[s], wv);
      float p = 0.f, c = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p = fmaf(a[j], a[j], p);
        c = fmaf(g[j] * wv[j], a[j], c);
      }
      if (i + R * s < nvec) {
        sum[0] += (double)p;
        sum[1] += (double)c;
      }
    }
    // (two buffers in turn: a wavefront that is a row ahead writes the other one)
    row_reduce<R>(sum, red[turn], SumOp{});
    // (unpacked anew behind the sums: values kept across the branch below would take a third more
    // registers, and with up to three vectors a wavefront's place)
#pragma unroll
    for (int s = 0; s < V && V < 4; ++s) {
      cur.h[s] = opaque(cur.h[s]);
      cur.g[s] = opaque(cur.g[s]);
      wr[s] = opaque(wr[s]);
    }
    float rstd = row_rstd(sum[0], inv_d, eps);
    float c = float(sum[1] * inv_d) * rstd * rstd;
    float up = 1.0f;
    const double gn = fabs(sum[1]) * inv_d;
    if (!row_in_range(sum[0], inv_d, eps) || !(gn < __builtin_inf()) || (gn < 0x1p-100 && gn > 0.0)) {
      // (the row's sums in fp64, as in the forward kernel; the same in all threads.  A sum of 0, which rows
      // without a gradient have, stays: its products are 0, or below 2^-150 each)
      sum[0] = sum[1] = 0.0;
#pragma unroll
      for (int s = 0; s < V; ++s) {
        if (i + R * s >= nvec) continue;
        add_squares(cur.h[s], sum[0]);
        add_products(cur.h[s], cur.g[s], wr[s], sum[1]);
      }
      row_reduce<R>(sum, red[2 + turn], SumOp{});
      bool small;
      rstd = wide_rstd(sum[0], inv_d, eps, small);
      if (small) {
        up = kSmallRow;
#pragma unroll
        for (int s = 0; s < V; ++s) cur.h[s] = enlarged(cur.h[s]);
      }
      c = float(sum[1] * inv_d * (double)up * (double)rstd * (double)rstd);
    }
#pragma unroll
    for (int s = 0; s < V; ++s) {
      float a[8], g[8], wv[8], add[8], o[8];
      unpack8(cur.h[s], a);
      unpack8(cur.g[s], g);
      unpack8(wr[s], wv);
      if (dh) unpack8(cur.a[s], add);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[s][j] = fmaf(g[j], a[j] * rstd, dw[s][j]);
        o[j] = rstd * fmaf(-c, a[j], g[j] * wv[j]) * up;
        if (dh) o[j] += add[j];
      }
      if (i + R * s < nvec) st16(dx, (size_t)row * nvec + i + R * s, pack8(o));
    }
    if (kAhead && more) cur = nxt;
  }
  if (!part) return;
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int idx = i + R * s;
    if (idx >= nvec) continue;
    float* p = part + ((size_t)blockIdx.x * nvec + idx) * 8;
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      gstore16(p + j, 0, make_uint4(__float_as_uint(dw[s][j]), __float_as_uint(dw[s][j + 1]),
                                    __float_as_uint(dw[s][j + 2]), __float_as_uint(dw[s][j + 3])));
  }
}

// dw[c] = sum_b part[b][c]: 32 columns per workgroup (whole 128-byte lines), its 32 groups of 8 threads
// take every 32nd partial, then the groups' sums in order.
__global__ __launch_bounds__(256) void dw_reduce_kernel(const float* __restrict__ part, int nb, int d,
                                                        float* __restrict__ dw) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, col = blockIdx.x * 32 + c * 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < d) {  // (d % 8 == 0)
#pragma unroll 4
    for (int b = r; b < nb; b += 32) {
      const uint4 v = ld16(part, ((size_t)b * d + col) / 4);
      s[0] += __uint_as_float(v.x);
      s[1] += __uint_as_float(v.y);
      s[2] += __uint_as_float(v.z);
      s[3] += __uint_as_float(v.w);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[r][c * 4 + j] = s[j];
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + (int)threadIdx.x < d) {
    float v = 0.f;
    for (int b = 0; b < 32; ++b) v += red[b][threadIdx.x];
    dw[blockIdx.x * 32 + threadIdx.x] = v;
  }
}

}  // namespace

hipError_t launch_rmsnorm(const void* x, const void* res, const void* w, float eps, int T, int d,
                          int fmt, void* h_out, void* y, void* q, void* qs, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int nvec = d / 8;
  with_row_shape(nvec, T <= kFewRows, [&](auto Rc, auto Vc) {
    constexpr int R = decltype(Rc)::value, V = decltype(Vc)::value;
    const unsigned grid = R == 64 ? ((unsigned)T + 3) / 4 : (unsigned)T;
    auto go = [&](auto F) {
      rmsnorm_kernel<decltype(F)::value, R, V><<<grid, row_block(R), 0, s>>>(
          x, res, w, eps, 1.0 / d, T, nvec, h_out, y, static_cast<uint8_t*>(q), qs);
    };
    if (fmt == kNormFp8) go(std::integral_constant<int, kNormFp8>{});
    else if (fmt == kNormMx) go(std::integral_constant<int, kNormMx>{});
    else if (fmt == kNormI8) go(std::integral_constant<int, kNormI8>{});
    else go(std::integral_constant<int, kNormBf16>{});
  });
  return hipGetLastError();
}

hipError_t launch_quant_i8(const void* x, bool f32, int T, int d, uint8_t* q, float* qs,
                           hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int nvec = d / 8;
  with_row_shape(nvec, T <= kFewRows, [&](auto Rc, auto Vc) {
    constexpr int R = decltype(Rc)::value, V = decltype(Vc)::value;
    const unsigned grid = R == 64 ? ((unsigned)T + 3) / 4 : (unsigned)T;
    if (f32) quant_i8_kernel<true, R, V><<<grid, row_block(R), 0, s>>>(x, T, nvec, q, qs);
    else quant_i8_kernel<false, R, V><<<grid, row_block(R), 0, s>>>(x, T, nvec, q, qs);
  });
  return hipGetLastError();
}

// Partial sums of dw: one per workgroup, each 8 d bytes of traffic beside a row's 6 or 8 d.  At 1, 3 and
// 6 rows per workgroup: 777 x 4096 13.4, 12.3, 13.4 us; 333 x 4096 9.8, 9.9, 12.5; 1500 x 2048 11.1,
// 11.9, 12.4.
int rmsnorm_grad_parts(int T) {
  return T <= 64 ? T : std::min(kNormGradBlocks, std::max(64, (T + kNormGradRows - 1) / kNormGradRows));
}

hipError_t launch_rmsnorm_grad(const void* dy, const void* dh, const void* h, const void* w,
                               float eps, int T, int d, void* dx, float* dw, float* part,
                               hipStream_t s) {
  const int nvec = d / 8, nb = rmsnorm_grad_parts(T);
  if (T > 0) {
    auto go = [&](auto Rc, auto Vc) {
      constexpr int R = decltype(Rc)::value, V = decltype(Vc)::value;
      rmsnorm_grad_kernel<R, V><<<nb, R, 0, s>>>(dy, dh, h, w, eps, 1.0 / d, T, nvec, dx,
                                                 dw ? part : nullptr);
    };
    if (nvec <= 64) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 128) go(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 1024) with_steps<256, 1, 4>((nvec + 255) / 256, go);
    else with_steps<512, 3, 4>((nvec + 511) / 512, go);
  }
  if (dw) dw_reduce_kernel<<<(d + 31) / 32, 256, 0, s>>>(part, nb, d, dw);
  return hipGetLastError();
}

}  // namespace moe

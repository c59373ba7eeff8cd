// Gradient of the norms around a block (the forward pass is the norm kernel's, norm.hip).
//
//   u = x / sqrt(mean(x^2) + eps) * post,  h = rs * r + bs * gate * u,  y = h / sqrt(mean(h^2) + eps) * pre
// with dy at y and dh at h:
//   H = dh + r2 (dy pre - n2 mean(dy pre n2))             n2 = h r2, r2 = 1 / sqrt(mean(h^2) + eps)
//   dr = rs H,  dgate = bs H u,  g1 = bs gate post H      n1 = x r1, r1 likewise
//   dx = r1 (g1 - n1 mean(g1 n1))  (without a norm behind the block: bs gate H)
//   dpre[c] = sum_t dy n2,  dpost[c] = sum_t bs gate H n1,  dgate[c] = sum_t bs H u for a gate per channel
// A gate per channel is the same in all rows, so both of the last two come from one sum, of H n1.
//
// Bound by HBM: x, h, dy and dh are read once and dx, dr written once, 12 bytes a value; H stays in fp32
// registers between the two norms. 8192 x 7168 takes 156 us (4.5 TB/s; a copy runs at 5.1), with a gate per token
// 190 us (16 bytes a value, 4.9 TB/s). Few rows are bound by their chain of loads and two reductions instead:
// 8.1 us for one row of 7168. Loading the next row ahead, loads past the caches and more or fewer workgroups than
// four wavefronts per SIMD gave nothing.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "norm_dev.h"

namespace moe {

namespace {

// 1 / sqrt(mean(v^2) + eps) of a row from its sum of squares, which is summed again in fp64 where it left
// fp32's range; a small row's values are enlarged (norm_dev.h), `up` is then kSmallRow.
template <int R, int V>
__device__ __forceinline__ float rstd_of(uint4 (&v)[V], double sum, double inv_d, float eps, int i, int nvec,
                                         double* red, float& up) {
  up = 1.0f;
  if (row_in_range(sum, inv_d, eps)) return row_rstd(sum, inv_d, eps);
  double s[1] = {0.0};
#pragma unroll
  for (int q = 0; q < V; ++q)
    if (i + R * q < nvec) add_squares(v[q], s[0]);
  row_reduce<R>(s, red, SumOp{});
  bool small;
  const float r = wide_rstd(s[0], inv_d, eps, small);
  if (small) {
    up = kSmallRow;
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = enlarged(v[q]);
  }
  return r;
}

// Whether fp32 products may have left their range on the way to this sum (a sum of 0, which rows without a
// gradient have, stays).
__device__ __forceinline__ bool out_of_range(double sum, double inv_d) {
  const double m = fabs(sum) * inv_d;
  return !(m < __builtin_inf()) || (m < 0x1p-100 && m > 0.0);
}

// sum += sum_j n[j] * x[j] in fp64, a value at a time in a loop that turns both (they end as they began): a
// path that must not cost the other one registers.
__device__ __forceinline__ void add_row_products(float (&n)[8], uint4 x, double& sum) {
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    sum = fma((double)n[0], (double)bf16_lo(x.x), sum);
    const float f = n[0];
#pragma unroll
    for (int c = 0; c < 7; ++c) n[c] = n[c + 1];
    n[7] = f;
    x = make_uint4((x.x >> 16) | (x.y << 16), (x.y >> 16) | (x.z << 16), (x.z >> 16) | (x.w << 16),
                   (x.w >> 16) | (x.x << 16));
  }
}

// Value j of a vector.
__device__ __forceinline__ float value(const uint4& v, int j) {
  const uint32_t p = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return j & 1 ? bf16_hi(p) : bf16_lo(p);
}

// The sum of a vector's squares, two at a time from their packed form.
__device__ __forceinline__ float squares(const uint4& v) {
  const uint32_t p[4] = {v.x, v.y, v.z, v.w};
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t b = __builtin_bit_cast(bf16x2_t, p[i]);
    sum = __builtin_amdgcn_fdot2_f32_bf16(b, b, sum, false);
  }
  return sum;
}

// A row's sums in fp64, the same in every thread and in a fixed order: row_reduce's, but that all rows of 16
// lanes pass theirs on through LDS, and the r-th row of each wavefront joins those of value r: one exchange among
// lanes for all values (4096 x 2048 33.6 us; with row_reduce in fp64 37.0, in fp32 32.9).  red: NA * R / 16 values
// of its own for every call.
template <int R, int NA>
__device__ __forceinline__ void row_sums(double (&v)[NA], double* red) {
  static_assert(NA <= 4, "a row of lanes per value");
  if constexpr (R == 64) {
    row_reduce<R>(v, red, SumOp{});
  } else {
    constexpr int W = R / 16;
    const int lane = threadIdx.x & 63, l = lane & 15;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      v[i] = reduce16(v[i], SumOp{});
      if (l == 0) red[i * W + (threadIdx.x >> 4)] = v[i];
    }
    __syncthreads();
    const double* mine = red + min(lane >> 4, NA - 1) * W;
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < W; j += 16)
      if (W >= 16 || l < W) s += mine[j + l];
    s = reduce16(s, SumOp{});
#pragma unroll
    for (int i = 0; i < NA; ++i) v[i] = read_lane(s, 16 * i);
  }
}

// ROWS: a gate per token and channel, [T][d].
template <int R, int V, bool ROWS>
__global__ __launch_bounds__(R, 4) void block_grad_kernel(BlockGrad a, double inv_d, int nvec) {
  __shared__ double red[2][4][R / 16];  // a row's four sums, in fp64 over fp32 chains of eight
  __shared__ double wide[2][3][R / 64];
  const int i = threadIdx.x;
  // Sums over the thread's rows, of H n1 and of dy n2. Beside two vectors of a row and of its gate the registers do
  // not hold the latter: they take 64 KB of LDS per CU at every R, which four wavefronts per SIMD leave free.
  constexpr bool kLds = ROWS && V == 2;
  __shared__ float lds_sum[kLds ? V * 8 * R : 1];
  float sA[V][8], sP[kLds ? 1 : V][8];
  auto pre_sum = [&](int s, int j) -> float& {
    if constexpr (kLds) return lds_sum[(s * 8 + j) * R + i];
    else return sP[s][j];
  };
#pragma unroll
  for (int s = 0; s < V; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j) sA[s][j] = pre_sum(s, j) = 0.f;
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  int turn = 0;
  for (int row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    // (a uniform address per row and array, and lane offsets that are opaque, since the compiler would keep
    // their sums with every array's address instead: 20 registers a vector)
    const size_t base = (size_t)row * nvec * 16;
    auto rows = [&](const void* p, uint32_t off) { return gload16(static_cast<const char*>(p) + base, off); };
    auto put = [&](char* p, uint32_t off, const uint4& v) {
      if (a.once) gstore16_nt(p, off, v);
      else gstore16(p, off, v);
    };
    uint4 h[V], g[V], x[V], add[V], gt[V], wp[V], wq[V];
    uint32_t at[V];
#pragma unroll
    for (int s = 0; s < V; ++s) {
      at[s] = min(i + R * s, nvec - 1) * 16;
      asm volatile("" : "+v"(at[s]));
      const uint32_t c = at[s];
      h[s] = rows(a.h, c);
      g[s] = rows(a.dy, c);
      x[s] = rows(a.x, c);
      // (what is absent is 0 or 1: no branches below)
      add[s] = a.dh ? rows(a.dh, c) : make_uint4(0, 0, 0, 0);
      gt[s] = ROWS ? rows(a.in.gate, c) : a.in.gate ? gload16(a.in.gate, c) : ones;
      wp[s] = gload16(a.pre, c);
      if (!ROWS) wq[s] = a.in.post ? gload16(a.in.post, c) : ones;
    }
    double sum[3] = {0.0, 0.0, 0.0};
#pragma unroll
    for (int s = 0; s < V; ++s) {
      float c = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c = fmaf(value(g[s], j) * value(wp[s], j), value(h[s], j), c);
        if (j & 1) __builtin_amdgcn_sched_barrier(0);  // (few unpacked values at a time)
      }
      if (i + R * s < nvec) {
        sum[0] += (double)squares(h[s]);
        sum[1] += (double)c;
        sum[2] += (double)squares(x[s]);
      }
    }
    // (two buffers in turn: a wavefront that is a row ahead writes the other one)
    row_sums<R>(sum, red[turn][0]);
    double gh = sum[1];
    if (!row_in_range(sum[0], inv_d, a.eps) || out_of_range(gh, inv_d)) {
      double c[1] = {0.0};
#pragma unroll
      for (int s = 0; s < V; ++s)
        if (i + R * s < nvec) add_products(h[s], g[s], wp[s], c[0]);
      row_reduce<R>(c, wide[turn][0], SumOp{});
      gh = c[0];
    }
    float up2, up1 = 1.0f, r1 = 1.0f;
    const float r2 = rstd_of<R, V>(h, sum[0], inv_d, a.eps, i, nvec, wide[turn][1], up2);
    const float c2 = float(gh * inv_d * (double)up2 * (double)r2 * (double)r2);
    if (a.in.post) r1 = rstd_of<R, V>(x, sum[2], inv_d, a.eps, i, nvec, wide[turn][2], up1);
    // (unpacked anew behind the sums: values kept across the branches would not fit the registers)
#pragma unroll
    for (int s = 0; s < V; ++s) {
      h[s] = opaque(h[s]);
      g[s] = opaque(g[s]);
      x[s] = opaque(x[s]);
      if (!ROWS) wp[s] = opaque(wp[s]);
    }
    float n[V][8];  // the gradient that reaches the first norm (or x)
    double back[1] = {0.0};
#pragma unroll
    for (int s = 0; s < V; ++s) {
      const bool in = i + R * s < nvec;
      if (ROWS) {  // (no registers for them before)
        __builtin_amdgcn_sched_barrier(0);
        wp[s] = gload16(a.pre, at[s]);
        wq[s] = a.in.post ? gload16(a.in.post, at[s]) : ones;
      }
      uint32_t dr[4], dg[4];
      float q = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // (two values at a time: few live ones)
        float r[2], t[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * w + e;
          const float hv = value(h[s], j), gv = value(g[s], j), gate = value(gt[s], j), post = value(wq[s], j);
          pre_sum(s, j) = fmaf(gv, hv * r2, pre_sum(s, j));
          const float H = fmaf(r2 * fmaf(-c2, hv, gv * value(wp[s], j)), up2, value(add[s], j));
          const float n1 = value(x[s], j) * r1, bH = a.in.bs * H;
          r[e] = a.in.rs * H;
          if (ROWS) t[e] = bH * n1 * post;
          sA[s][j] = fmaf(ROWS ? gate * H : H, n1, sA[s][j]);
          n[s][j] = bH * gate * post;
          q = fmaf(n[s][j], value(x[s], j), q);
        }
        // (the sums are taken here: moved to the row's end they would keep all their operands)
        asm volatile("" : "+v"(sA[s][2 * w]), "+v"(sA[s][2 * w + 1]));
        if (!kLds) asm volatile("" : "+v"(pre_sum(s, 2 * w)), "+v"(pre_sum(s, 2 * w + 1)));
        dr[w] = pack_bf16x2(r[0], r[1]);
        if (ROWS) dg[w] = pack_bf16x2(t[0], t[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (in) {
        const uint32_t c = at[s];
        put(static_cast<char*>(a.dres) + base, c, make_uint4(dr[0], dr[1], dr[2], dr[3]));
        if (ROWS && a.dgate_rows)
          put(static_cast<char*>(a.dgate_rows) + base, c, make_uint4(dg[0], dg[1], dg[2], dg[3]));
        back[0] += (double)q;
      }
    }
#pragma unroll
    for (int s = 0; s < V; ++s) x[s] = opaque(x[s]);
    float c1 = 0.f;
    if (a.in.post) {
      row_sums<R>(back, red[turn][3]);
      double gx[1] = {back[0]};
      if (out_of_range(gx[0], inv_d)) {
        gx[0] = 0.0;
#pragma unroll
        for (int s = 0; s < V; ++s)
          if (i + R * s < nvec) add_row_products(n[s], x[s], gx[0]);
        row_reduce<R>(gx, wide[turn][0], SumOp{});
      }
      // (of a small row, x and the sum hold `up` once, r1 its inverse)
      c1 = float(gx[0] * inv_d * (double)r1 * (double)r1);
    }
#pragma unroll
    for (int s = 0; s < V; ++s) {
      float xv[8], o[8];
      unpack8(x[s], xv);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = a.in.post ? r1 * fmaf(-c1, xv[j], n[s][j]) * up1 : n[s][j];
      if (i + R * s < nvec) put(static_cast<char*>(a.dx) + base, at[s], pack8(o));
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int idx = i + R * s;
    if (idx >= nvec) continue;
    float* p = a.part + ((size_t)blockIdx.x * 2 * nvec + idx) * 8;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      gstore16(p + j, 0, make_uint4(__float_as_uint(sA[s][j]), __float_as_uint(sA[s][j + 1]),
                                    __float_as_uint(sA[s][j + 2]), __float_as_uint(sA[s][j + 3])));
      gstore16(p + (size_t)nvec * 8 + j, 0,
               make_uint4(__float_as_uint(pre_sum(s, j)), __float_as_uint(pre_sum(s, j + 1)),
                          __float_as_uint(pre_sum(s, j + 2)), __float_as_uint(pre_sum(s, j + 3))));
    }
  }
}

// The workgroups' sums [nb][2][d] in a fixed order (norm_dev.h), then the factors that all rows share.
__global__ __launch_bounds__(256) void block_grad_sum_kernel(BlockGrad a, int nb, int d) {
  __shared__ float red[32][33];
  sum_parts(a.part, nb, 2 * d, red);
  const int at = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || at >= 2 * d) return;
  float v = 0.f;
  for (int b = 0; b < 32; ++b) v += red[b][threadIdx.x];
  if (at >= d) {
    if (a.dpre) a.dpre[at - d] = v;
    return;
  }
  auto channel = [&](const void* p) { return bf16_to_f32(static_cast<const uint16_t*>(p)[at]); };
  if (a.dpost) a.dpost[at] = a.in.bs * (a.in.gate && !a.in.gate_rows ? channel(a.in.gate) * v : v);
  if (a.dgate) a.dgate[at] = a.in.bs * (a.in.post ? channel(a.in.post) * v : v);
}

}  // namespace

// A row takes two reductions one behind the other, and a workgroup's sums 16 d bytes beside its 12 or 16 d: at 1, 2, 3
// and 4 rows per workgroup, 200 x 4096 12.5, 13.0, 14.6, 16.8 us; 333 x 4096 with a gate per token 15.5, 14.9, 17.7,
// 20.2; 777 x 7168 31.7, 29.8, 31.2, 29.6; 777 x 4096 with a gate per token 22.3, 21.0, 22.8, 23.8.  (Up to 1024
// workgroups for long batches: 2048 x 7168 57 us, 50 with 512.)
int block_grad_parts(int T) { return norm_grad_parts(T, kBlockGradRows); }

hipError_t launch_block_grad(BlockGrad a, int d, hipStream_t s) {
  // Outputs pass the caches by when a call's rows are more than the 256 MB last-level cache holds (8192 x 7168 154
  // us, 158 kept).
  a.once = (int64_t)a.T * d * (a.in.gate_rows ? 16 : 12) > (int64_t)256 << 20;
  const int nvec = d / 8, nb = block_grad_parts(a.T);
  if (a.T > 0) {
    auto go = [&](auto Rc, auto Vc) {
      constexpr int R = decltype(Rc)::value, V = decltype(Vc)::value;
      auto* kernel = a.in.gate_rows ? &block_grad_kernel<R, V, true> : &block_grad_kernel<R, V, false>;
      kernel<<<nb, R, 0, s>>>(a, 1.0 / d, nvec);
    };
    if (nvec <= 64) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 128) go(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 512) with_steps<256, 1, 2>((nvec + 255) / 256, go);
    else if (nvec <= 1024) go(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  }
  if (a.dpre || a.dpost || a.dgate) block_grad_sum_kernel<<<(2 * d + 31) / 32, 256, 0, s>>>(a, nb, d);
  return hipGetLastError();
}

}  // namespace moe

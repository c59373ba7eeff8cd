// The way back of the sort by expert: gradients of combine and route (permute's is the combine
// without weights, combine.hip).
//
//   combine   out[t] = sum_j w[t][j] * y[row(t, j)]   (row = slot_dst)
//     dy[row(t, j)] = bf16(w[t][j] * dout[t]),  dw[t][j] = sum_c dout[t][c] * y[row(t, j)][c]
//   route     w = softmax over the k selected logits
//     dlogits[t][e] = sum over the slots j of expert e of w_j (dw_j - sum_i w_i dw_i), else 0
//
// The combine gradient is bound by HBM: y is read once, dy written once, and each token's dout is
// held in registers for its k rows.  8192 tokens x 8 rows of 7168: 385 us (5.2 TB/s).  The route
// gradient is bound by its launch up to some thousand tokens (4096 x 384 4.2 us) and then by its 4-byte
// stores: 8192 x 384 6.9, and 2.4 for every further 4096 x 384 (2.6 TB/s).
#include <type_traits>

#include "kernels.h"
#include "rows_dev.h"

namespace moe {

namespace {

constexpr int64_t kLastLevelCache = 256 << 20;
// Tokens up to which a row takes more wavefronts (with_row_shape): 4 rows of 7168 each, 1 token 4.7 us
// against 6.5, 256 7.2 against 8.8, 512 12.7 against 13.4, 1024 22.1 either way.
constexpr int kFewTokens = 512;

// ONCE: y and dy pass the caches by.  Rows that the 256 MB last-level cache holds are better left in
// it, for this kernel and for what reads dy next (1024 tokens x 8 x 7168, 250 MB: 39 us kept, 48
// passed by), larger ones only push each other out (1500 tokens 76 and 72 us, 8192 406 and 385).
template <int R, int V, bool ONCE>
__global__ __launch_bounds__(row_block(R)) void combine_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ y, const int32_t* __restrict__ slot_dst,
    const float* __restrict__ w, int T, int k, int nvec, void* __restrict__ dy,
    float* __restrict__ dw) {
  __shared__ float red[kMaxTopK * R / 64];
  const int t = R == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (R == 64 && t >= T) return;  // (whole wavefronts; no barrier in this form)
  const int i = R == 64 ? threadIdx.x & 63 : threadIdx.x;
  uint4 g[V];
#pragma unroll
  for (int s = 0; s < V; ++s) g[s] = ld16(dout, (size_t)t * nvec + min(i + R * s, nvec - 1));
  float dot[kMaxTopK];
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    dot[j] = 0.f;
    if (j >= k) continue;
    const size_t base = (size_t)slot_dst[(size_t)t * k + j] * nvec;
    const float wj = dy ? w[(size_t)t * k + j] : 0.f;
    uint4 yv[V];
    if (dw) {
#pragma unroll
      for (int s = 0; s < V; ++s) {
        const size_t idx = base + min(i + R * s, nvec - 1);
        yv[s] = ONCE ? ld16_once(y, idx) : ld16(y, idx);
      }
    }
#pragma unroll
    for (int s = 0; s < V; ++s) {
      if (i + R * s >= nvec) continue;
      float a[8];
      unpack8(g[s], a);
      if (dw) {
        float b[8];
        unpack8(yv[s], b);
#pragma unroll
        for (int c = 0; c < 8; ++c) dot[j] = fmaf(a[c], b[c], dot[j]);
      }
      if (dy) {
#pragma unroll
        for (int c = 0; c < 8; ++c) a[c] *= wj;
        if (ONCE) st16_once(dy, base + i + R * s, pack8(a));
        else st16(dy, base + i + R * s, pack8(a));
      }
    }
  }
  if (!dw) return;
  row_reduce<R>(dot, red, SumOp{});
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < k && i == j) dw[(size_t)t * k + j] = dot[j];
}

// 2^lg lanes per token (E <= 64: the fewest that cover E), each writing every 2^lg-th expert.
__global__ __launch_bounds__(256) void route_grad_kernel(const int32_t* __restrict__ ids,
                                                         const float* __restrict__ w,
                                                         const float* __restrict__ dw, int T, int E,
                                                         int k, int lg, float* __restrict__ dl) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = at >> lg;
  if (t >= T) return;
  int id[kMaxTopK];
  float v[kMaxTopK], u[kMaxTopK];
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    id[j] = -1;
    v[j] = u[j] = 0.f;
    if (j < k) {
      id[j] = ids[t * k + j];
      v[j] = w[t * k + j];
      u[j] = dw[t * k + j];
      s = fmaf(v[j], u[j], s);
    }
  }
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) v[j] *= u[j] - s;
  for (int e = (int)(at & ((1 << lg) - 1)); e < E; e += 1 << lg) {
    float o = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) o += id[j] == e ? v[j] : 0.f;
    dl[t * E + e] = o;
  }
}

}  // namespace

hipError_t launch_combine_grad(const void* dout, const void* y, const int32_t* slot_dst,
                               const float* w, int T, int k, int d, void* dy, float* dw,
                               hipStream_t s) {
  if (T == 0) return hipSuccess;
  const bool once = (int64_t)T * d * 2 * (1 + k * ((dy ? 1 : 0) + (dw ? 1 : 0))) > kLastLevelCache;
  with_row_shape(d / 8, T <= kFewTokens, [&](auto Rc, auto Vc) {
    constexpr int R = decltype(Rc)::value, V = decltype(Vc)::value;
    const unsigned grid = R == 64 ? ((unsigned)T + 3) / 4 : (unsigned)T;
    auto* kernel = once ? &combine_grad_kernel<R, V, true> : &combine_grad_kernel<R, V, false>;
    kernel<<<grid, row_block(R), 0, s>>>(dout, y, slot_dst, w, T, k, d / 8, dy, dw);
  });
  return hipGetLastError();
}

hipError_t launch_route_grad(const int32_t* ids, const float* w, const float* dw, int T, int E,
                             int k, float* dl, hipStream_t s) {
  if (T == 0) return hipSuccess;
  int lg = 0;
  while (lg < 6 && (1 << lg) < E) ++lg;
  const int64_t blocks = (((int64_t)T << lg) + 255) / 256;
  route_grad_kernel<<<(unsigned)blocks, 256, 0, s>>>(ids, w, dw, T, E, k, lg, dl);
  return hipGetLastError();
}

}  // namespace moe

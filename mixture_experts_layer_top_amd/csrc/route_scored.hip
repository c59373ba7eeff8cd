// Routing by scores: sigmoid, or softmax over all experts; a bias per expert that only the selection
// sees; groups of experts, of which the best are kept; weights renormalised over the selected and scaled.
// And its gradient.
//
//   s_e = sigmoid(l_e), or exp(l_e - max) / sum over all E
//   c_e = s_e + b_e; without a bias the logits' order, which is the scores' (both rise with l); -inf
//         where l_e is -inf
//   groups of E / G consecutive experts, valued by the sum of their 1 or 2 largest c; the `top` best stay
//   ids: the k largest c there, ties to the lower id; w_j = scale * s_j (/ sum_i s_i, 0 where that is 0)
// gradient, with w from the forward call and D = sum_i w_i dw_i:
//   sigmoid, renormalised  dl_j = (1 - s_j) w_j (dw_j - D / scale)      plain  (1 - s_j) w_j dw_j
//   softmax, renormalised  dl_j = w_j (dw_j - D / scale)                plain  dl_e = [selected] w_e dw_e - s_e D
//
// One wavefront per token, lane l holding experts l, l + 64, ...; each of the k rounds takes the largest
// remaining key, as in route_dev.h.  Keys are 64 bits wide: scores of different experts lie as near as
// 2^-30 to each other in some row of a large batch, and which of them is selected is a result.
#include "kernels.h"
#include "rows_dev.h"

namespace moe {

namespace {

// Unsigned order of the keys is the values' order, with 0 for "no candidate", NaN next above it, then
// -inf; +0 and -0 are one value.
__device__ __forceinline__ uint64_t key64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t k = (u >> 63) ? ~u : (u | (uint64_t(1) << 63));
  return v != v ? uint64_t(1) : k;
}

struct Max64 {
  __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  v = reduce16(v, Max64{});
  const Max64 m;
  return m(m(read_lane(v, 0), read_lane(v, 16)), m(read_lane(v, 32), read_lane(v, 48)));
}
__device__ __forceinline__ double wave_sum64(double v) {
  v = reduce16(v, SumOp{});
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = reduce16(v, [](float a, float b) { return fmaxf(a, b); });
  return fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)), fmaxf(read_lane(v, 32), read_lane(v, 48)));
}

constexpr float kInf = __builtin_inff();

// Scores of the wavefront's token in 64 bits (0 past E, and for a row without any finite logit).
template <int VPL>
__device__ __forceinline__ void scores64(const float (&l)[VPL], int E, int score, double (&s)[VPL]) {
  const int lane = threadIdx.x & 63;
  if (score == kScoreSigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    return;
  }
  float m = -kInf;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (lane + 64 * i < E) m = fmaxf(m, l[i]);
  m = wave_max(m);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    s[i] = lane + 64 * i < E && m != -kInf ? exp((double)l[i] - (double)m) : 0.0;
    sum += s[i];
  }
  sum = wave_sum64(sum);
#pragma unroll
  for (int i = 0; i < VPL; ++i) s[i] = sum == 0.0 ? 0.0 : s[i] / sum;
}

template <int VPL>
__global__ __launch_bounds__(256) void route_scored_kernel(const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int T, int E,
                                                           int k, Scoring p, int32_t* __restrict__ ids,
                                                           float* __restrict__ w) {
  __shared__ uint64_t s_key[4][64 * VPL];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wv;
  if (t >= T) return;  // (whole wavefronts; no barrier below)
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = logits[(size_t)t * E + min(e, E - 1)];
  }
  double s[VPL];
  scores64<VPL>(l, E, p.score, s);
  double c[VPL];
  uint64_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = bias ? s[i] + (double)bias[min(e, E - 1)] : p.groups > 1 && p.group_top > 1 ? s[i] : (double)l[i];
    if (l[i] == -kInf) c[i] = -__builtin_inf();
    key[i] = e < E ? key64(c[i]) : 0;
  }
  if (p.groups > 1) {
    const int size = E / p.groups;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s_key[wv][lane + 64 * i] = __builtin_bit_cast(uint64_t, c[i]);
    __builtin_amdgcn_wave_barrier();
    uint64_t gk = 0;
    if (lane < p.groups) {
      // (by keys, so that a NaN stays at the bottom)
      uint64_t k0 = 0, k1 = 0;
      double a = 0.0, b = 0.0;
      for (int j = 0; j < size; ++j) {
        const double v = __builtin_bit_cast(double, s_key[wv][lane * size + j]);
        const uint64_t kv = key64(v);
        if (kv > k0) {
          k1 = k0; b = a;
          k0 = kv; a = v;
        } else if (kv > k1) {
          k1 = kv; b = v;
        }
      }
      gk = key64(p.group_top > 1 ? a + b : a);
    }
    uint64_t keep = 0;
    for (int j = 0; j < p.top; ++j) {
      const uint64_t best = wave_max64(gk);
      const int g = __ffsll((unsigned long long)__ballot(gk == best)) - 1;
      keep |= uint64_t(1) << g;
      if (lane == g) gk = 0;
    }
    if (!bias) {  // (group values need the scores, the order inside them the logits)
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = key[i] == 0 ? 0 : key64((double)l[i]);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((keep >> (e / size)) & 1)) key[i] = 0;
    }
  }
  // lane j keeps the j-th selected expert and its score
  int my_id = 0;
  double my_s = 0.0;
  for (int j = 0; j < k; ++j) {
    uint64_t m = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = m > key[i] ? m : key[i];
    const uint64_t best = wave_max64(m);
    int id = -1;
    double sc = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint64_t hit = __ballot(key[i] == best);
      if (id < 0 && hit != 0) {
        const int at = __ffsll((unsigned long long)hit) - 1;
        id = 64 * i + at;
        sc = read_lane(s[i], at);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i == id) key[i] = 0;
    if (lane == j) {
      my_id = id;
      my_s = sc;
    }
  }
  if (p.renorm) {
    const double sum = wave_sum64(my_s);
    my_s = sum == 0.0 ? 0.0 : my_s / sum;
  }
  if (lane < k) {
    ids[(size_t)t * k + lane] = my_id;
    w[(size_t)t * k + lane] = float(my_s * (double)p.scale);
  }
}

// 2^lg lanes per token, as the softmax's gradient in grad.hip; WHOLE: a wavefront per token, since
// every expert's score takes part.
template <bool WHOLE>
__global__ __launch_bounds__(256) void route_scored_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int T, int E, int k, int lg, Scoring p, float* __restrict__ dl) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = at >> lg;
  if (t >= T) return;
  int id[kMaxTopK];
  float v[kMaxTopK], u[kMaxTopK];
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    id[j] = -1;
    v[j] = u[j] = 0.f;
    if (j < k) {
      id[j] = ids[t * k + j];
      v[j] = w[t * k + j];
      u[j] = dw[t * k + j];
      dot = fmaf(v[j], u[j], dot);
    }
  }
  const float off = p.renorm ? dot / p.scale : 0.f;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    v[j] *= u[j] - off;
    if (p.score == kScoreSigmoid && j < k) {
      const float l = (unsigned)id[j] < (unsigned)E ? logits[t * E + id[j]] : 0.f;
      const float e = expf(-fabsf(l));  // (at most 1, whatever l)
      v[j] *= (l > 0.f ? e : 1.0f) / (1.0f + e);  // 1 - s
    }
  }
  const int e0 = (int)(at & ((1 << lg) - 1));
  if constexpr (WHOLE) {
    float l[8], m = -kInf, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      l[i] = e0 + 64 * i < E ? logits[t * E + e0 + 64 * i] : -kInf;
      m = fmaxf(m, l[i]);
    }
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      l[i] = m == -kInf ? 0.f : expf(l[i] - m);
      sum += l[i];
    }
    sum = reduce16(sum, SumOp{});
    sum = (read_lane(sum, 0) + read_lane(sum, 16)) + (read_lane(sum, 32) + read_lane(sum, 48));
    const float f = sum == 0.f ? 0.f : dot / sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + 64 * i;
      if (e >= E) continue;
      float o = -l[i] * f;
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) o += id[j] == e ? v[j] : 0.f;
      dl[t * E + e] = o;
    }
  } else {
    for (int e = e0; e < E; e += 1 << lg) {
      float o = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) o += id[j] == e ? v[j] : 0.f;
      dl[t * E + e] = o;
    }
  }
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, int E, int k,
                               const Scoring& p, int32_t* ids, float* w, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const unsigned grid = ((unsigned)T + 3) / 4;
  auto* kernel = E <= 64 ? &route_scored_kernel<1> : E <= 128 ? &route_scored_kernel<2>
                 : E <= 256 ? &route_scored_kernel<4> : &route_scored_kernel<8>;
  kernel<<<grid, 256, 0, s>>>(logits, bias, T, E, k, p, ids, w);
  return hipGetLastError();
}

hipError_t launch_route_scored_grad(const float* logits, const int32_t* ids, const float* w,
                                    const float* dw, int T, int E, int k, const Scoring& p, float* dl,
                                    hipStream_t s) {
  if (T == 0) return hipSuccess;
  const bool whole = p.score == kScoreSoftmax && !p.renorm;
  int lg = whole ? 6 : 0;
  while (lg < 6 && (1 << lg) < E) ++lg;
  const int64_t blocks = (((int64_t)T << lg) + 255) / 256;
  auto* kernel = whole ? &route_scored_grad_kernel<true> : &route_scored_grad_kernel<false>;
  kernel<<<(unsigned)blocks, 256, 0, s>>>(logits, ids, w, dw, T, E, k, lg, p, dl);
  return hipGetLastError();
}

}  // namespace moe

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
// 16 lanes per token sort the experts in fp32 (route_scored_kernel); what fp32 cannot decide, scores that lie as
// near as 2^-30 in some row of a large batch and rows with masked or non-finite logits, is decided in 64 bits,
// since which expert is selected is a result: among the token's candidates, or by a wavefront over the whole row
// (route_exact).  Weights are worked out in 64 bits and rounded once.
//
// Bound by one token's chain of some thousand dependent instructions, which two wavefronts per SIMD (8192 tokens)
// do not hide, not by HBM: 8192 tokens of 256 experts in 8 groups take 8.3 to 12.9 us, by how many need 64 bits, without
// groups and bias 5.5 (moe_route's wavefront per token 9.7), where their 8.9 MB take 2 us; 32768 of 384 21 us (2.5
// TB/s), one token 5.0.  Groups that 16 lanes do not share out go to route_exact at once: 60 experts in 6 groups 12
// us, 380 in 2, whose groups two lanes of 64 walk, 92.
// The gradient writes all of dlogits and reads no more than k values per token, but for a softmax over all
// experts: 8192 x 256 4.5 us and 5.9.
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

// One token by the whole wavefront, compared in 64 bits.  s_key: 64 * VPL keys of LDS of its own (groups).
template <int VPL>
__device__ __forceinline__ void route_exact(const float* __restrict__ logits, const float* __restrict__ bias,
                                            int t, int E, int k, const Scoring& p, uint64_t* s_key,
                                            int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & 63;
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
    for (int i = 0; i < VPL; ++i) s_key[lane + 64 * i] = __builtin_bit_cast(uint64_t, c[i]);
    __builtin_amdgcn_wave_barrier();
    uint64_t gk = 0;
    if (lane < p.groups) {
      // (by keys, so that a NaN stays at the bottom)
      uint64_t k0 = 0, k1 = 0;
      double a = 0.0, b = 0.0;
      for (int j = 0; j < size; j += 4) {
        double v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __builtin_bit_cast(double, s_key[lane * size + min(j + q, size - 1)]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t kv = j + q < size ? key64(v[q]) : 0;
          if (kv > k0) {
            k1 = k0; b = a;
            k0 = kv; a = v[q];
          } else if (kv > k1) {
            k1 = kv; b = v[q];
          }
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

template <int VPL>
__global__ __launch_bounds__(64) void route_exact_kernel(const float* __restrict__ logits,
                                                         const float* __restrict__ bias, int E, int k,
                                                         Scoring p, int32_t* __restrict__ ids,
                                                         float* __restrict__ w) {
  __shared__ uint64_t s_key[64 * VPL];
  route_exact<VPL>(logits, bias, blockIdx.x, E, k, p, s_key, ids, w);
}

// ------------------------------------------------------------------------------------------------
// 16 lanes per token
//
// Lane i of a token holds experts i v .. i v + v - 1 (v = ceil(E / 16)) and their c in fp32.  A key is c's
// place below the row's largest, 1 to 2^23 - 1, above the expert's complement, 511 - e, in 9 bits: unsigned order is
// c's order and ties go to the lower id, so one register carries an expert through the sort, and 0 is no expert.
// Each lane keeps its eight largest keys in order (one med3 per place and key), then four exchanges with other lanes
// merge the lists (the larger of each with the other's reversed, and a bitonic sort of eight).
//
// fp32 and 23 bits do not decide everything.  Where two of the first k + 1 keys are nearer than their errors (a row
// in some hundred), the first nine are compared again in 64 bits, a lane each.  Where that cannot help (the
// ninth and tenth are near too, or the last group that stays and the first that does not), and where anything
// infinite, masked or NaN is among them, the token is routed again by route_exact.
// ------------------------------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t from(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float from(float v) { return __uint_as_float(from<CTRL>(__float_as_uint(v))); }

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  return max(min(a, b), min(max(a, b), c));
}
// Descending order: larger first.
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t m = max(a, b);
  b = min(a, b);
  a = m;
}
// The eight largest of two lanes' lists, in order, in both lanes.
template <int CTRL>
__device__ __forceinline__ void merge8(uint32_t (&v)[8]) {
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = max(v[j], from<CTRL>(v[7 - j]));
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & d)) order(m[j], m[j + d]);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = m[j];
}
// The two largest of two lanes' pairs a >= b.
template <int CTRL>
__device__ __forceinline__ void merge2(float& a, float& b) {
  const float x = from<CTRL>(a), y = from<CTRL>(b);
  b = fmaxf(fminf(a, x), fmaxf(b, y));
  a = fmaxf(a, x);
}
__device__ __forceinline__ float max16(float v) {
  return reduce16(v, [](float a, float b) { return fmaxf(a, b); });
}

constexpr float kPlaces = 0x1p23f;  // of a key

template <int V, bool VEC>
__global__ __launch_bounds__(64) void route_scored_kernel(const float* __restrict__ logits,
                                                          const float* __restrict__ bias, int T, int E,
                                                          int k, Scoring p, int32_t* __restrict__ ids,
                                                          float* __restrict__ w) {
  constexpr int VPL = V <= 4 ? 1 : V <= 8 ? 2 : V <= 16 ? 4 : 8;
  __shared__ uint64_t s_key[64 * VPL];
  const int lane = threadIdx.x, li = lane & 15;
  const int tok = blockIdx.x * 4 + (lane >> 4);
  const int t = min(tok, T - 1);  // (a token past the last is the last again, and not written)
  const int v = VEC ? V : (E + 15) >> 4, e0 = li * v;
  const size_t row = (size_t)t * E;
  float l[V], c[V];
  auto load4 = [&](const float* from, float* to) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint4 q = gload16(from, (e0 + i) * 4);
      to[i] = __uint_as_float(q.x);
      to[i + 1] = __uint_as_float(q.y);
      to[i + 2] = __uint_as_float(q.z);
      to[i + 3] = __uint_as_float(q.w);
    }
  };
  if (VEC) {
    load4(logits + row, l);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = e0 + i;
      l[i] = i < v && e < E ? logits[row + min(e, E - 1)] : -kInf;
    }
  }
  // scores, and a softmax's largest logit and 1 / sum
  float top = -kInf, inv = 1.0f;
  double inv64 = 1.0;
  if (p.score == kScoreSoftmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = max16(top);
    if (p.renorm) {  // (for the selection only)
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += __expf(l[i] - top);
      inv = 1.0f / reduce16(sum, SumOp{});
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += exp((double)l[i] - (double)top);  // (-inf past E)
      inv64 = 1.0 / reduce16(sum, SumOp{});
      inv = (float)inv64;
    }
  }
  const bool scored = bias || (p.groups > 1 && p.group_top > 1);
  if (!scored) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = p.score == kScoreSoftmax ? __expf(l[i] - top) * inv
                                               : __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
      c[i] = l[i] == -kInf ? -kInf : s;
    }
    if (bias) {
      float b[V];
      if (VEC) {
        load4(bias, b);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = bias[min(e0 + i, E - 1)];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] += b[i];
    }
  }
  // a sigmoid's fp32 value is within 2^-22 (its slope makes up for the exponential's argument), a softmax's within
  // 2^-18 of the largest one, 1 / sum (its exponentials and up to 36 additions); c adds |c| 2^-24
  const float tol_s = !scored ? 0.f : p.score == kScoreSoftmax ? inv * 0x1p-18f : 0x1p-21f;
  bool kept = true, unsure = false;
  if (p.groups > 1) {  // (16 / groups lanes hold a group)
    const int lg = 16 / p.groups;
    float a = -kInf, b = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b = fmaxf(b, fminf(a, c[i]));
      a = fmaxf(a, c[i]);
    }
    if (lg >= 2) merge2<0xb1>(a, b);
    if (lg >= 4) merge2<0x4e>(a, b);
    if (lg >= 8) merge2<0x141>(a, b);
    const float g = p.group_top > 1 ? a + b : a;
    const float size = fabsf(a) + (p.group_top > 1 ? fabsf(b) : 0.f);
    const float far = 2.0f * tol_s + max16(size < kInf ? size : 0.f) * (scored ? 0x1p-22f : 0.f);
    int above = 0, near = 0;
    auto against = [&](float o) {
      const float d = o - g;
      above += d > far ? 1 : 0;
      near += !(fabsf(d) > far) ? 1 : 0;  // (or not to be compared: two groups masked whole)
    };
#define MOE_ROT(n) if (p.groups == 16 || (n) % lg == 0) against(from<0x120 + (n)>(g));
    MOE_ROT(1) MOE_ROT(2) MOE_ROT(3) MOE_ROT(4) MOE_ROT(5) MOE_ROT(6) MOE_ROT(7) MOE_ROT(8)
    MOE_ROT(9) MOE_ROT(10) MOE_ROT(11) MOE_ROT(12) MOE_ROT(13) MOE_ROT(14) MOE_ROT(15)
#undef MOE_ROT
    kept = above + near < p.top;
    unsure = !kept && above < p.top;
    if (!bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l[i];
    }
  }
  // keys: places below the largest c that stays
  float high = -kInf;
#pragma unroll
  for (int i = 0; i < V; ++i) high = fmaxf(high, c[i]);
  high = max16(kept ? high : -kInf);
  // (values further below the largest than the span have place 1.  Far from 0 base is rounded, by more than what
  // it is above high - span: the largest ones then share the last place.  A place is off by half a step of c - base
  // and its rounding down: 3 between two without errors of their own are more than enough)
  const float span = bias ? 2.0f : 16.0f, scale = kPlaces / span, base = high - span * (1.0f - 0x1p-20f);
  // (up to all places: sums past 2^21 lie more than a million apart, and still may be out of order)
  const float off = (bias ? 2.0f * tol_s + fabsf(high) * 0x1p-22f : 0.f) * scale;
  const int apart = 2 + (int)fminf(off + 1.0f, kPlaces);
  uint32_t best[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) best[j] = 0u;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = e0 + i;
    const uint32_t place = (uint32_t)fminf(fmaxf((c[i] - base) * scale, 1.0f), kPlaces - 1.0f);  // (NaN: 1)
    key[i] = kept && (VEC || (i < v && e < E)) ? (place << 9) + (uint32_t)(511 - e) : 0u;
#pragma unroll
    for (int j = 7; j > 0; --j)
      if (j <= i) best[j] = med3(key[i], best[j - 1], best[j]);
    best[0] = max(best[0], key[i]);
  }
  merge8<0xb1>(best);
  merge8<0x4e>(best);
  merge8<0x141>(best);
  merge8<0x140>(best);
  uint32_t next = 0u;  // the largest that is not among them
#pragma unroll
  for (int i = 0; i < V; ++i) next = max(next, key[i] < best[7] ? key[i] : 0u);
  next = max(next, from<0xb1>(next));
  next = max(next, from<0x4e>(next));
  next = max(next, from<0x141>(next));
  next = max(next, from<0x140>(next));
  // lane j keeps the j-th, lane 8 the one behind them
  uint32_t mine = li == 8 ? next : 0u;
  bool gap = false, close = false;  // a gap at or behind the k-th; two of the first k + 1 too near to tell
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t after = j < 7 ? best[j + 1] : next;
    const bool apart_here = after == 0u || (int)(best[j] >> 9) - (int)(after >> 9) >= apart;
    if (j < k) {
      unsure |= (int)(best[j] >> 9) <= apart;  // (place 1: clamped, masked or NaN, or too near to what is)
      close |= !apart_here;
    }
    if (j >= k - 1) gap |= apart_here;
    if (j == li) mine = best[j];
  }
  int id = mine ? 511 - (int)(mine & 511u) : 0, rank = li < 8 ? li : 16;
  if (__ballot(close)) {
    // candidates again, in 64 bits: right among them if a gap divides them from the rest
    uint32_t last = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) last = max(last, key[i] < next ? key[i] : 0u);
    last = max(last, from<0xb1>(last));
    last = max(last, from<0x4e>(last));
    last = max(last, from<0x141>(last));
    last = max(last, from<0x140>(last));
    gap |= last == 0u || (int)(next >> 9) - (int)(last >> 9) >= apart;
    unsure |= close && !gap;
    const bool in = mine >= 2u << 9;
    double v64 = logits[row + min(id, E - 1)];
    if (bias) {
      if (p.score == kScoreSoftmax) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += exp((double)l[i] - (double)top);  // (-inf past E)
        v64 = exp(v64 - (double)top) / reduce16(sum, SumOp{});
      } else {
        v64 = 1.0 / (1.0 + exp(-v64));
      }
      v64 += (double)bias[min(id, E - 1)];
    }
    if (!in) v64 = -__builtin_inf();
    const int no = in ? id : 1024 + li;
    int above = 0;
    auto against = [&](double o, int n) { above += o > v64 || (o == v64 && n < no) ? 1 : 0; };
#define MOE_ROT(n) against(dpp16<0x120 + (n)>(v64), dpp16<0x120 + (n)>(no));
    MOE_ROT(1) MOE_ROT(2) MOE_ROT(3) MOE_ROT(4) MOE_ROT(5) MOE_ROT(6) MOE_ROT(7) MOE_ROT(8)
    MOE_ROT(9) MOE_ROT(10) MOE_ROT(11) MOE_ROT(12) MOE_ROT(13) MOE_ROT(14) MOE_ROT(15)
#undef MOE_ROT
    if (close) rank = above;
  }
  const bool chosen = rank < k;
  // scores, their renormalisation and scale in 64 bits; what even they do not hold, by route_exact
  const float lj = logits[row + min(id, E - 1)];
  double s;
  if (p.score == kScoreSoftmax) {
    const double x = (double)lj - (double)(p.renorm ? max16(chosen ? lj : -kInf) : top);
    s = exp(x) * inv64;
    unsure |= chosen && !(x > -700.0);
  } else {
    const double e = exp(-fabs((double)lj));
    s = (lj > 0.f ? 1.0 : e) / (1.0 + e);
    unsure |= chosen && !(lj > -700.0f);
  }
  if (p.renorm) s = s / reduce16(chosen ? s : 0.0, SumOp{});
  // (unsure is a group's, a token's: any of its lanes)
  const uint64_t ask = __ballot(unsure);
  const bool redo = (ask >> (lane & 48)) & 0xFFFF;
  if (tok < T && chosen && !redo) {
    ids[(size_t)t * k + rank] = id;
    w[(size_t)t * k + rank] = float(s * (double)p.scale);
  }
  if (ask) {
    for (int q = 0; q < 4; ++q)
      if (((ask >> (16 * q)) & 0xFFFF) && (int)blockIdx.x * 4 + q < T)
        route_exact<VPL>(logits, bias, blockIdx.x * 4 + q, E, k, p, s_key, ids, w);
  }
}

// Gradient, 16 lanes per token: lane j works out slot j's, and every lane then has all slots' (id, value) by
// row broadcasts and writes its share of the row.  V > 0: every expert's score takes part (a softmax over
// all), the logits of a lane's V experts stay in registers.  VEC: a lane has experts 64 c + 4 li .. + 3 (whole 16-byte
// vectors, E % 4 == 0), else 16 c + li.
template <int V, bool VEC>
__global__ __launch_bounds__(256) void route_scored_grad_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int T, int E, int k, Scoring p, float* __restrict__ dl) {
  const int li = threadIdx.x & 15;
  const int tok = (int)(((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4);
  const int t = min(tok, T - 1);  // (all lanes of a wavefront take part in the sums)
  const size_t row = (size_t)t * E, slot = (size_t)t * k + min(li, k - 1);
  constexpr int N = VEC ? 4 : 1, C = V / N;  // experts per step, steps
  auto at = [&](int c) { return VEC ? 64 * c + 4 * li : 16 * c + li; };
  float l[V ? V : 1], top = -kInf;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (VEC) {
      const uint4 q = gload16(logits + row, min(at(c), E - 4) * 4);
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < N; ++i) l[V ? c * N + i : 0] = at(c) < E ? __uint_as_float(u[i]) : -kInf;
    } else {
      l[V ? c : 0] = at(c) < E ? logits[row + min(at(c), E - 1)] : -kInf;
    }
  }
  const int id = ids[slot];
  const float u = dw[slot];
  float v = li < k ? w[slot] : 0.f;
  const float dot = reduce16(li < k ? v * u : 0.f, SumOp{});
  v *= li < k ? u - (p.renorm ? dot / p.scale : 0.f) : 0.f;
  if (!V && p.score == kScoreSigmoid) {
    const float lj = (unsigned)id < (unsigned)E ? logits[row + id] : 0.f;
    const float e = expf(-fabsf(lj));  // (at most 1, whatever the logit)
    v *= (lj > 0.f ? e : 1.0f) / (1.0f + e);  // 1 - s
  }
  float f = 0.f;  // of all experts: - s_e * dot
  if (V) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = max16(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = top == -kInf ? 0.f : expf(l[i] - top);
      sum += (double)l[i];
    }
    sum = reduce16(sum, SumOp{});
    f = sum == 0.0 ? 0.f : -dot / (float)sum;
  }
  int sid[kMaxTopK];
  float sv[kMaxTopK];
#define MOE_SLOT(j)                                                                                  \
  sid[j] = __builtin_amdgcn_update_dpp(0, id, 0x150 + j, 0xf, 0xf, false);                           \
  sv[j] = from<0x150 + j>(v);                                                                        \
  if (j >= k) sid[j] = -1;
  MOE_SLOT(0) MOE_SLOT(1) MOE_SLOT(2) MOE_SLOT(3) MOE_SLOT(4) MOE_SLOT(5) MOE_SLOT(6) MOE_SLOT(7)
#undef MOE_SLOT
  if (tok >= T) return;
  auto step = [&](int c, const float* mine) {
    float o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      o[i] = V ? mine[i] * f : 0.f;
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) o[i] += sid[j] == at(c) + i ? sv[j] : 0.f;
    }
    if (at(c) >= E) return;
    if constexpr (VEC)
      gstore16(dl + row, at(c) * 4, make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                                               __float_as_uint(o[3])));
    else dl[row + at(c)] = o[0];
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) step(c, l + c * N);
  } else {
    for (int c = 0; 16 * N * c < E; ++c) step(c, nullptr);
  }
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, int E, int k,
                               const Scoring& p, int32_t* ids, float* w, hipStream_t s) {
  if (T == 0) return hipSuccess;
  if (p.groups > 1 && (E % 16 || 16 % p.groups)) {  // (groups that lanes do not share out)
    auto* kernel = E <= 64 ? &route_exact_kernel<1> : E <= 128 ? &route_exact_kernel<2>
                   : E <= 256 ? &route_exact_kernel<4> : &route_exact_kernel<8>;
    kernel<<<(unsigned)T, 64, 0, s>>>(logits, bias, E, k, p, ids, w);
    return hipGetLastError();
  }
  // Whole vectors wherever a lane's experts are some of them (8192 tokens, with and without: 192 experts 6.0 us and 8.5,
  // 320 8.0 and 13.8, 448 9.5 and 17.3).
  using Kernel = decltype(&route_scored_kernel<4, true>);
  static constexpr Kernel kVec[] = {
      &route_scored_kernel<4, true>,  &route_scored_kernel<8, true>,  &route_scored_kernel<12, true>,
      &route_scored_kernel<16, true>, &route_scored_kernel<20, true>, &route_scored_kernel<24, true>,
      &route_scored_kernel<28, true>, &route_scored_kernel<32, true>};
  const bool vec = E % 64 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  const Kernel kernel = vec        ? kVec[E / 64 - 1]
                        : E <= 64  ? &route_scored_kernel<4, false>
                        : E <= 128 ? &route_scored_kernel<8, false>
                        : E <= 256 ? &route_scored_kernel<16, false> : &route_scored_kernel<32, false>;
  kernel<<<((unsigned)T + 3) / 4, 64, 0, s>>>(logits, bias, T, E, k, p, ids, w);
  return hipGetLastError();
}

hipError_t launch_route_scored_grad(const float* logits, const int32_t* ids, const float* w,
                                    const float* dw, int T, int E, int k, const Scoring& p, float* dl,
                                    hipStream_t s) {
  if (T == 0) return hipSuccess;
  const bool whole = p.score == kScoreSoftmax && !p.renorm;
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dl)) % 16 == 0;
  auto* kernel = !whole     ? vec ? &route_scored_grad_kernel<0, true> : &route_scored_grad_kernel<0, false>
                 : E <= 128 ? vec ? &route_scored_grad_kernel<8, true> : &route_scored_grad_kernel<8, false>
                 : E <= 256 ? vec ? &route_scored_grad_kernel<16, true> : &route_scored_grad_kernel<16, false>
                            : vec ? &route_scored_grad_kernel<32, true> : &route_scored_grad_kernel<32, false>;
  kernel<<<((unsigned)T + 15) / 16, 256, 0, s>>>(logits, ids, w, dw, T, E, k, p, dl);
  return hipGetLastError();
}

}  // namespace moe

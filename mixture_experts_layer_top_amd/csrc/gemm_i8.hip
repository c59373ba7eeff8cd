// Matrix products of int8 rows and int8 weights with one fp32 scale per row (token) and per weight
// row (output channel): the experts' grouped gate/up and down GEMMs, and one dense product.
//
//   acc[row][n] = sum_k qx[row][k] * qw[n][k]          (int32, exact: K <= 32768 keeps it below 2^30)
//   v[row][n] = float(acc) * sx[row] * sw[n]
//   gate/up: h = SiLU(v_gate) * v_up in fp32 (quantised per row before the down GEMM, norm.hip: a
//            row's scale needs all of its d_ff columns, which no tile has alone)
//   down, dense: y = bf16(v)
//
// The scales are constant along K, so the K loops are MFMAs and loads only, and integer sums do not
// depend on their order: results are the same bits whatever the tile family.  Two families, as for
// bf16:
//  * stream (light experts, small dense products): a workgroup's 4 wavefronts split K over 16 weight
//    rows (K >= kStreamSplitK) or 32, up to 64 token rows per pass; weights go straight from HBM
//    into MFMA registers, 1 KB contiguous per load in the tiled layout (moe_fp8_tile).
//  * mfma (mfma_tile.h): 256 weight rows by 32 to 256 token rows staged through LDS; dense, 4096 rows
//    of K = 4096 by 14336 channels, 217-230 us (2.1-2.2 POP/s, the library's rate), of K = 14336 by 4096 193
//    (2.49): the clock falls to 1.6-1.7 GHz under this load, and MFMAs fill 0.67 of the CUs' busy cycles at
//    K = 4096, where an epilogue follows every 32 K-steps, and 0.83 at K = 14336.  8 experts of 4096 x 14336,
//    8192 rows: 930-945 + 470 us (2.04-2.06).
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "mfma_tile.h"
#include "rows_dev.h"
#include "stream_dev.h"

namespace moe {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// 16 bytes per lane and operand, loaded alike for both (row l % 32 or l % 16, the lane group's 16
// bytes of K), so the K order inside the instruction does not matter.  C as the bf16 MFMAs.
struct ElemI8 {
  using Frag = i32x4;
  using Acc = i32x16;
  static constexpr int kBytes = 1;
  static constexpr bool kTiledW = true;
  static constexpr bool kOddSteps = true;  // K % 128 == 0: any number of 128-wide K-steps
  static __device__ __forceinline__ Frag frag(const uint4& v) { return __builtin_bit_cast(i32x4, v); }
  static __device__ __forceinline__ Acc mfma(const Frag& a, const Frag& b, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};

__device__ __forceinline__ i32x4 mfma16_i8(const uint4& a, const uint4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ float4 gload_f32x4(const float* p, uint32_t i) {
  return __builtin_bit_cast(float4, gload16(p, i * 4));
}

// ------------------------------------------------------------------------------------------------
// streaming tiles
// ------------------------------------------------------------------------------------------------

// Rows [m0, m0 + rows) (rows <= 16 * MQ) by the 16 weight rows of each wavefront group from n0.  XL: the
// rows' codes lie in LDS, xl bytes apart from xs, and their scales in sxs (MQ = 1); they are read only
// after `staged` has run, behind the first weight loads.
template <int MQ, bool GU, int WK, bool XL = false, class Staged = void (*)()>
__device__ __forceinline__ void stream_tile_i8(const Seg& sg, int m0, int rows, int n0, int* red,
                                               const uint8_t* xs = nullptr, int xl = 0,
                                               const float* sxs = nullptr, Staged staged = nullptr) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int grp = wv / WK, kw = wv % WK;
  n0 += 16 * grp;
  const int K = sg.K, N = sg.N, nkb = K / 128;
  const uint32_t woff = (uint32_t)(n0 >> 4) * (uint32_t)(nkb * 2048) + lane * 16;
  int src[MQ];
  uint32_t xoff[MQ];
#pragma unroll
  for (int q = 0; q < MQ; ++q) {
    int r = q * 16 + r16;
    r = r < rows ? r : rows - 1;  // padded columns re-read a valid row; never stored
    const int gr = sg.row0 + m0 + r;
    src[q] = XL ? r : sg.tok ? gload_i32(sg.tok, gr) : gr;
    xoff[q] = (uint32_t)src[q] * (uint32_t)(XL ? xl : K) + kg * 32;
  }
  i32x4 acc0[MQ], acc1[MQ];
#pragma unroll
  for (int q = 0; q < MQ; ++q) acc0[q] = acc1[q] = i32x4{0, 0, 0, 0};
  constexpr int U = XL || (MQ == 1 && !GU) ? 4 : 2;  // 128-wide chunks per batch
  struct Batch { uint4 a0[U][2], a1[U][2], b[XL ? 1 : U][MQ][2]; };
  // this wavefront's chunks: kw, kw + WK, ... (the group's wavefronts read adjacent units)
  const int nc = (nkb - kw + WK - 1) / WK;
  auto load = [&](Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)min(kw + WK * (i + u), nkb - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bt.a0[u][h] = gload16_nt(sg.w0, woff + kb * 2048 + h * 1024);
        if (GU) bt.a1[u][h] = gload16_nt(sg.w1, woff + kb * 2048 + h * 1024);
        if (!XL) {
#pragma unroll
          for (int q = 0; q < MQ; ++q) bt.b[XL ? 0 : u][q][h] = gload16(sg.a, xoff[q] + kb * 128 + h * 16);
        }
      }
    }
  };
  auto compute = [&](const Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= nc) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < MQ; ++q) {
          const uint4 b = XL ? *reinterpret_cast<const uint4*>(
                                   xs + xoff[q] + (uint32_t)(kw + WK * (i + u)) * 128 + h * 16)
                             : bt.b[XL ? 0 : u][q][h];
          acc0[q] = mfma16_i8(bt.a0[u][h], b, acc0[q]);
          if (GU) acc1[q] = mfma16_i8(bt.a1[u][h], b, acc1[q]);
        }
    }
  };
  Batch b0, b1;
  if (nc > 0) load(b0, 0);
  if constexpr (XL) staged();
  for (int i = 0; i < nc; i += 2 * U) {
    if (i + U < nc) load(b1, i + U);
    compute(b0, i);
    if (i + 2 * U < nc) load(b0, i + 2 * U);
    if (i + U < nc) compute(b1, i + U);
  }
  // split-K sums: wavefronts kw > 0 of a group park theirs in LDS, wavefront 0 adds them
  constexpr int NV = MQ * 4 * (GU ? 2 : 1);
  if (WK > 1) __syncthreads();  // red[] may still be read by the previous tile
  if (WK > 1 && kw > 0) {
    int* dst = red + ((grp * (WK - 1) + kw - 1) * NV) * 64 + lane;
#pragma unroll
    for (int q = 0; q < MQ; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dst[(q * 4 + j) * 64] = acc0[q][j];
        if (GU) dst[(MQ * 4 + q * 4 + j) * 64] = acc1[q][j];
      }
  }
  if (WK > 1) __syncthreads();
  if (kw != 0) return;
#pragma unroll
  for (int w = 0; w < WK - 1; ++w) {
    const int* sp = red + ((grp * (WK - 1) + w) * NV) * 64 + lane;
#pragma unroll
    for (int q = 0; q < MQ; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc0[q][j] += sp[(q * 4 + j) * 64];
        if (GU) acc1[q][j] += sp[(MQ * 4 + q * 4 + j) * 64];
      }
  }
  // lane holds weight rows n0 + 4 kg + j of token column r16 of each group q
  const float4 s0 = gload_f32x4(sg.s0, n0 + 4 * kg);
  const float4 s1 = GU ? gload_f32x4(sg.s1, n0 + 4 * kg) : s0;
  const float c0[4] = {s0.x, s0.y, s0.z, s0.w}, c1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int q = 0; q < MQ; ++q) {
    const int r = q * 16 + r16;
    if (r >= rows) continue;
    const float sx = XL ? sxs[src[q]] : gload_f32(sg.as, src[q]);
    const size_t at = (size_t)(sg.row0 + m0 + r) * N + n0 + 4 * kg;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = float(acc0[q][j]) * sx * c0[j];
      if (GU) v[j] = swiglu(v[j], float(acc1[q][j]) * sx * c1[j]);
    }
    if (GU)
      gstore16(sg.out, at * 4, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                          __float_as_uint(v[2]), __float_as_uint(v[3])));
    else
      gstore8(sg.out, at * 2, uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
  }
}

template <int MQMAX, bool GU, int WK>
__device__ __forceinline__ void stream_rows_i8(const Seg& sg, int m0, int rows, int n0, int* red) {
  for (int sub = 0; sub < rows; sub += 16 * MQMAX) {
    const int r = min(16 * MQMAX, rows - sub);
    if (MQMAX == 1 || r <= 16) stream_tile_i8<1, GU, WK>(sg, m0 + sub, r, n0, red);
    else if (MQMAX == 2 || r <= 32) stream_tile_i8<MQMAX >= 2 ? 2 : 1, GU, WK>(sg, m0 + sub, r, n0, red);
    else stream_tile_i8<MQMAX, GU, WK>(sg, m0 + sub, r, n0, red);
  }
}

// Persistent, as the bf16 streaming kernel.
template <bool GU, int MQMAX>
__global__ __launch_bounds__(256) void gemm_stream_i8(const Seg* __restrict__ segs,
                                                      int32_t* __restrict__ meta) {
  __shared__ int slot;
  __shared__ int seg_base[kSegCap];
  __shared__ int red[3 * MQMAX * 4 * 2 * 64];
  const int nseg = meta[0], ntiles = meta[1];
  if ((int)blockIdx.x >= ntiles) return;
  for (int i = threadIdx.x; i < nseg; i += 256) seg_base[i] = segs[i].tile_base;
  __syncthreads();
  int t = blockIdx.x;
  for (;;) {
    const Seg& sg = segs[__builtin_amdgcn_readfirstlane(find_seg_lds(seg_base, nseg, t))];
    const int local = t - sg.tile_base;
    const int mt = local % sg.mtiles, nt = local / sg.mtiles;
    const int m0 = mt * kStreamMaxRows;
    const int rows = min(kStreamMaxRows, sg.rows - m0);
    if (sg.tn == 16) stream_rows_i8<MQMAX, GU, 4>(sg, m0, rows, nt * 16, red);
    else stream_rows_i8<MQMAX, GU, 2>(sg, m0, rows, nt * 32, red);
    t = gridDim.x + __builtin_amdgcn_readfirstlane(pop_tile(&meta[kMetaQueue], &slot));
    if (t >= ntiles) break;
  }
}

// The dense product's streaming form: 16 * NR weight rows by 16 * MQ token rows per workgroup, whose 4
// wavefronts split K (interleaved chunks; the sums meet in LDS).  A wavefront's weight blocks share its
// token fragments and the other way round, so the traffic between L2 and the CUs, which bounds all but the
// smallest batches (some 40 GB/s per CU with all of them loading, with twice the loads in flight too),
// falls with both.  7168 x 7168: 16 tokens 12 us (4.3 TB/s of weights), 64 19, 128 27; 2048 x 7168: 64
// tokens 7.8, 256 13.3.
template <int MQ, int NR>
__global__ __launch_bounds__(256) void gemm_stream_i8_dense(Seg sg) {
  constexpr int U = MQ * NR == 1 ? 4 : MQ * NR <= 4 ? 2 : 1;  // 128-wide chunks per batch
  constexpr int NV = MQ * NR * 4;                            // sums per lane
  __shared__ int red[3 * NV * 64];
  const int lane = threadIdx.x & 63, kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = sg.K, N = sg.N, nkb = K / 128;
  // (the tiles of one weight block on one XCD, whose L2 they share)
  const int tile = sg.mtiles == 1 ? blockIdx.x
                                  : (blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
  if (tile >= sg.mtiles * sg.ntiles) return;
  const int m0 = (tile % sg.mtiles) * (16 * MQ), rows = min(16 * MQ, sg.rows - m0);
  const int n0 = (tile / sg.mtiles) * (16 * NR);
  uint32_t woff[NR], xoff[MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)  // (a block past N re-reads the last one; never stored)
    woff[j] = (uint32_t)min((n0 >> 4) + j, (N >> 4) - 1) * (uint32_t)(nkb * 2048) + lane * 16;
#pragma unroll
  for (int q = 0; q < MQ; ++q)  // (a row past the last re-reads it; never stored)
    xoff[q] = (uint32_t)(m0 + min(q * 16 + r16, rows - 1)) * (uint32_t)K + kg * 32;
  i32x4 acc[NR][MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int q = 0; q < MQ; ++q) acc[j][q] = i32x4{0, 0, 0, 0};
  struct Batch { uint4 w[U][NR][2], x[U][MQ][2]; };
  const int nc = (nkb - kw + 3) / 4;  // this wavefront's chunks: kw, kw + 4, ...
  auto load = [&](Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)min(kw + 4 * (i + u), nkb - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < NR; ++j)
          bt.w[u][j][h] = sg.mtiles == 1 ? gload16_nt(sg.w0, woff[j] + kb * 2048 + h * 1024)
                                         : gload16(sg.w0, woff[j] + kb * 2048 + h * 1024);
#pragma unroll
        for (int q = 0; q < MQ; ++q) bt.x[u][q][h] = gload16(sg.a, xoff[q] + kb * 128 + h * 16);
      }
    }
  };
  auto compute = [&](const Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= nc) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int q = 0; q < MQ; ++q) acc[j][q] = mfma16_i8(bt.w[u][j][h], bt.x[u][q][h], acc[j][q]);
    }
  };
  Batch b0, b1;
  if (nc > 0) load(b0, 0);
  for (int i = 0; i < nc; i += 2 * U) {
    if (i + U < nc) load(b1, i + U);
    compute(b0, i);
    if (i + 2 * U < nc) load(b0, i + 2 * U);
    if (i + U < nc) compute(b1, i + U);
  }
  // every wavefront parks its sums but those of the pieces (j, q) it finishes itself: piece p goes to
  // wavefront p % 4, slot order (p, wavefront)
  constexpr int P = NR * MQ;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 4 == kw) continue;
    int* dst = red + (p * 3 + (kw < p % 4 ? kw : kw - 1)) * 256 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i * 64] = acc[p / MQ][p % MQ][i];
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 4 != kw) continue;
    const int j = p / MQ, q = p % MQ;
    const int* src = red + p * 3 * 256 + lane;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][q][i] += src[w * 256 + i * 64];
    const int r = q * 16 + r16, n = n0 + 16 * j + 4 * kg;
    if (r >= rows || n >= N) continue;
    const float4 s4 = gload_f32x4(sg.s0, n);
    const float c[4] = {s4.x, s4.y, s4.z, s4.w};
    const float sx = gload_f32(sg.as, m0 + r);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = float(acc[j][q][i]) * sx * c[i];
    gstore8(sg.out, ((size_t)(m0 + r) * N + n) * 2, uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
  }
}

// ------------------------------------------------------------------------------------------------
// small batches (kernels.h: kSmallI8Tokens)
//
// A decode step's experts hold a few rows each, and the launches around the weights' stream weigh as
// much as a part of it: the selection kernel (one workgroup, 8-10 us) and the rows' quantisation (5 us)
// beside 37 + 24 us of weights at one token (DeepSeek-V3-shaped layer; 61 us in all, 82 with them).
// Here every workgroup finds the experts that hold rows by itself, from the counts, and a down tile
// quantises its expert's rows of h into LDS while its first weights are on their way.  Same tiles, same
// sums, same bits.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void small_list(const int32_t* counts, int E, int (&s_exp)[kSmallI8Rows],
                                           int& s_n) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const bool has = e < E && gload_i32(counts, e) > 0;
      const uint64_t m = __ballot(has);
      const int at = n + __popcll(m & ((1ull << lane) - 1));
      if (has && at < kSmallI8Rows) s_exp[at] = e;
      n += __popcll(m);
    }
    if (lane == 0) s_n = min(n, kSmallI8Rows);
  }
  __syncthreads();
}

template <bool GU, int WK>
__global__ __launch_bounds__(256) void gemm_small_i8(SmallI8 a) {
  constexpr int TN = 64 / WK;  // output columns per workgroup
  __shared__ int s_exp[kSmallI8Rows];
  __shared__ int s_n;
  __shared__ int red[(WK > 1 ? 3 : 1) * 4 * 2 * 64];
  __shared__ float s_sx[16];
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];  // down: up to 16 rows of codes
  small_list(a.counts, a.E, s_exp, s_n);
  const int per = a.N / TN, ntiles = s_n * per, xl = a.K + 16;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const int e = __builtin_amdgcn_readfirstlane(s_exp[t / per]);
    Seg sg = {};
    sg.a = a.x;
    sg.as = a.xs;
    sg.tok = a.tok;
    sg.w0 = static_cast<const uint8_t*>(a.w0) + (size_t)e * a.N * a.K;
    sg.w1 = static_cast<const uint8_t*>(a.w1) + (size_t)e * a.N * a.K;
    sg.s0 = a.s0 + (size_t)e * a.N;
    sg.s1 = a.s1 + (size_t)e * a.N;
    sg.out = a.out;
    sg.N = a.N;
    sg.K = a.K;
    sg.row0 = __builtin_amdgcn_readfirstlane(gload_i32(a.offsets, e));
    // (never more rows than the batch has, whatever the counts say: the codes' LDS is sized for them)
    const int rows = min(__builtin_amdgcn_readfirstlane(gload_i32(a.counts, e)), a.rows);
    const int n0 = (t % per) * TN;
    for (int m0 = 0; m0 < rows; m0 += 16) {
      const int r = min(16, rows - m0);
      if constexpr (GU) {
        stream_tile_i8<1, true, WK>(sg, m0, r, n0, red);
      } else {
        const float* h = a.h + (size_t)(sg.row0 + m0) * a.K;
        stream_tile_i8<1, false, WK, true>(sg, m0, r, n0, red, s_x, xl, s_sx, [&] {
          __syncthreads();  // (the last tile's readers are done)
          // a wavefront per row: its largest magnitude, then its codes (as quant_i8_kernel)
          for (int i = wv; i < r; i += 4) {
            const float* row = h + (size_t)i * a.K;
            uint32_t m[1] = {0u};
            for (int c = lane * 4; c < a.K; c += 256) {
              const uint4 v = ld16(row + c, 0);
              m[0] = max(max(m[0], max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu)),
                         max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu));
            }
            row_reduce<64>(m, static_cast<uint32_t*>(nullptr), MaxOp{});
            const float sc = i8_scale(m[0]);
            const bool bad = m[0] >= kInfBits;
            const Scale f(bad ? 1.0f : sc);
            if (lane == 0) s_sx[i] = sc;
            for (int c = lane * 4; c < a.K; c += 256) {
              const uint4 u = ld16(row + c, 0);
              float v[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                            __uint_as_float(u.w)};
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = bad ? 0.f : v[j];
              i8_pack<1, false>(v, f, reinterpret_cast<uint32_t*>(s_x + i * xl + c));
            }
          }
          __syncthreads();
        });
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// LDS-staged MFMA tiles
// ------------------------------------------------------------------------------------------------

// What the epilogue needs of a claimed tile.
struct I8Cur {
  int m0, rows, n0, nk, N, row0;
  void* out;
  const float* as;
  const float* s0;
  const float* s1;
  const int32_t* tok;
};

// Epilogue through LDS (as the bf16 tiles'): the tile goes into the idle ring as [token row][column],
// fp32 h (gate/up, 128 columns) or bf16 y (256 columns), 512 bytes of output per row and 16 of
// padding, then out in 16-byte chunks of whole rows.  TB: token blocks of a short tile (8: full).
template <bool GU, int TB>
__device__ __forceinline__ void i8_store(const i32x16 (&acc)[4][4], const I8Cur& c) {
  constexpr bool kFull = TB == 8;
  constexpr int RS = 512 + 16;
  static_assert(256 * RS <= kRingBytes, "an output tile fits the ring");
  const uint32_t tid = tid_here();
  const int lane = tid & 63, wv = tid >> 6;
  const int l32 = lane & 31, khalf = lane >> 5;
  const int wm = kFull ? wv & 1 : 0, wn = kFull ? wv >> 1 : wv;
  constexpr int NB = kFull ? 4 : TB;           // token blocks of this wavefront
  constexpr int NA = GU ? (kFull ? 2 : 1) : (kFull ? 4 : 2);  // its 32-column output blocks
  const int cw = wn * 32 * NA;                 // its first output column
  const int t0 = (kFull ? wm * 128 : 0) + l32;  // its token rows: t0 + 32 b
  float sx[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int gr = c.row0 + c.m0 + min(t0 + 32 * b, c.rows - 1);
    sx[b] = gload_f32(c.as, c.tok ? gload_i32(c.tok, gr) : gr);
  }
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    // (one block's scales at a time: all of them together would not fit beside the accumulators)
    __builtin_amdgcn_sched_barrier(0);
    // lane holds C[8 q + 4 khalf + s][l32] of each 32x32 block (rows = weights)
    const int col = cw + a * 32 + 4 * khalf;
    float4 w0[4], w1[GU ? 4 : 1];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = min(c.n0 + col + 8 * q, c.N - 4);  // (columns past N are not stored)
      w0[q] = gload_f32x4(c.s0, n);
      if (GU) w1[GU ? q : 0] = gload_f32x4(c.s1, n);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint8_t* row = g_ring + (t0 + 32 * b) * RS;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float s0[4] = {w0[q].x, w0[q].y, w0[q].z, w0[q].w};
        float v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = float(acc[a][b][q * 4 + s]) * sx[b] * s0[s];
        if (GU) {
          const float4 u = w1[GU ? q : 0];
          const float s1[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int s = 0; s < 4; ++s)
            v[s] = swiglu(v[s], float(acc[a + NA][b][q * 4 + s]) * sx[b] * s1[s]);
          *reinterpret_cast<float4*>(row + (col + 8 * q) * 4) = float4{v[0], v[1], v[2], v[3]};
        } else {
          *reinterpret_cast<uint2*>(row + (col + 8 * q) * 2) =
              uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
      }
    }
  }
  __syncthreads();
  constexpr int H = kFull ? 256 : TB * 32;
  constexpr int VB = GU ? 4 : 2;  // bytes per value
  const int ch = tid & 31;
  const int col = c.n0 + ch * (16 / VB);
  const int nr = c.rows < H ? c.rows : H;
  if (col < c.N) {  // (down: the last tile of a row may be part full, in multiples of 16 columns)
    for (int t = tid >> 5; t < nr; t += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(g_ring + t * RS + ch * 16);
      gstore16(c.out, ((size_t)(c.row0 + c.m0 + t) * c.N + col) * VB, v);
    }
  }
}

template <bool GU>
__device__ __forceinline__ void i8_run(MfmaTile<GU, ElemI8>& tile, int h, const I8Cur& c) {
  if (h == BM) {
    tile.run_full(c.nk);
    i8_store<GU, 8>(tile.acc, c);
  } else if (h == 128) {
    tile.template run_short<4>(c.nk);
    i8_store<GU, 4>(tile.acc, c);
  } else if (h == 64) {
    tile.template run_short<2>(c.nk);
    i8_store<GU, 2>(tile.acc, c);
  } else {
    tile.template run_short<1>(c.nk);
    i8_store<GU, 1>(tile.acc, c);
  }
}

template <bool GU>
__device__ __forceinline__ I8Cur i8_cur(const Seg& sg, int m0, int rows, int nt) {
  I8Cur c;
  c.m0 = m0;
  c.rows = rows;
  c.n0 = nt * (GU ? kMfmaBNGateUp : kMfmaBNDown);
  c.nk = sg.K / 128;
  c.N = sg.N;
  c.row0 = sg.row0;
  c.out = sg.out;
  c.as = sg.as;
  c.s0 = sg.s0;
  c.s1 = sg.s1;
  c.tok = sg.tok;
  return c;
}

// Persistent: one workgroup per CU takes tiles from the per-XCD queues in the list's order (the
// selection kernel's, as for bf16).
template <bool GU>
__global__ __launch_bounds__(256, 1) void gemm_mfma_i8(const Seg* __restrict__ segs,
                                                       int32_t* __restrict__ meta) {
  __shared__ int slot;
  __shared__ int seg_base[kSegCap];
  const int ntiles = meta[1];
  if (ntiles == 0) return;
  const int nseg = meta[0], ntiles0 = meta[kMetaClass0], order = meta[kMetaOrder];
  // positions [0, sbase) are whole tiles, then come 2^lgs pieces of 256 >> lgs token rows of each tile
  const int sbase = meta[kMetaSplitBase], S = meta[kMetaSplitS], lgs = S == 4 ? 2 : S == 2 ? 1 : 0;
  int pref, b0, b1;
  two_class_split((int)gridDim.x, ntiles0, ntiles - ntiles0, pref, b0, b1);
  b0 = __builtin_amdgcn_readfirstlane(b0);
  b1 = __builtin_amdgcn_readfirstlane(b1);
  const int chunk = __builtin_amdgcn_readfirstlane(max(1, (int)gridDim.x / kXcds) *
                                                   (order == kOrderMix ? 2 : 1));
  for (int i = threadIdx.x; i < nseg; i += blockDim.x) seg_base[i] = segs[i].tile_base;
  __syncthreads();
  MfmaTile<GU, ElemI8> tile;
  // A list of at most one position per workgroup is handed out without the queues, whose ends every
  // workgroup would look for in turn (some 10 us): XCD x takes an equal run of positions.
  const int npos = sbase + ((ntiles - sbase) << lgs), per = (npos + kXcds - 1) / kXcds;
  const bool once = npos <= (int)gridDim.x && per <= (int)gridDim.x / kXcds && order != kOrderTwoClass;
  const int mine = blockIdx.x / kXcds < per ? blockIdx.x % kXcds * per + blockIdx.x / kXcds : npos;
  int q = 0;
  for (bool first = true;; first = false) {
    if (once && (!first || mine >= npos)) return;
    // (opaque moves: the reciprocals of the queue's divisions are computed here, not held across
    // the K loops)
    const int nt_ = opaque_s(ntiles), nt0_ = opaque_s(ntiles0), ch_ = opaque_s(chunk);
    int t, piece = 0, hrows = BM;
    if (order == kOrderTwoClass) {  // (never split)
      t = pop_tile_two_class(meta + kMetaQueue, meta + kMetaQueue1, nt0_, nt_ - nt0_, opaque_s(b0),
                             opaque_s(b1), pref, &slot, q);
      if (t < 0) return;
    } else {
      const int sb_ = opaque_s(sbase);
      int pos = once ? mine
                     : pop_tile_xcd(meta + kMetaQueue, sb_ + ((nt_ - sb_) << lgs), ch_, &slot, q);
      if (pos < 0) return;
      if (pos >= sb_) {
        hrows = BM >> lgs;
        piece = (pos - sb_) & ((1 << lgs) - 1);
        pos = sb_ + ((pos - sb_) >> lgs);
      }
      t = order == kOrderLongestFirst ? pos : interleave_tile(pos, nt0_, nt_);
    }
    const Seg& sg = segs[__builtin_amdgcn_readfirstlane(find_seg_lds(seg_base, nseg, t))];
    const int local = t - sg.tile_base;
    const int m0 = local % sg.mtiles * BM + piece * hrows;
    if (m0 >= sg.rows) continue;  // (a piece past the tile's rows)
    const I8Cur c = i8_cur<GU>(sg, m0, min(hrows, sg.rows - m0), local / sg.mtiles);
    tile.setup(sg, c.m0, c.rows, c.n0, 0);
    const int h = __builtin_amdgcn_readfirstlane(tile.bm);
    tile.prologue(c.nk);
    i8_run<GU>(tile, h, c);  // (the pop's barriers keep the next tile's loads behind its stores)
  }
}

// Tile t of a dense product in an order that keeps 32 consecutive tiles (one round of an XCD's CUs)
// near a square: runs of kDenseGM m-tiles per weight tile.
constexpr int kDenseGM = 8;
__device__ __forceinline__ void dense_tile(int t, int mtiles, int ntiles, int& mt, int& nt) {
  const int per = kDenseGM * ntiles, g = t / per, r = t - g * per;
  const int gm = min(kDenseGM, mtiles - g * kDenseGM);
  nt = r / gm;
  mt = g * kDenseGM + r - nt * gm;
}

// The dense product: whole tiles [0, full), a multiple of the grid, then what is left over as pieces
// of H = 256 >> lgs token rows, so that the last round is shorter instead of half empty (full = 0: the
// product has less than a round of whole tiles, and all of it is pieces).  XCD x takes an equal run of
// the whole tiles and of the pieces.
__global__ __launch_bounds__(256, 1) void gemm_mfma_i8_dense(Seg sg, int full, int pieces, int lgs) {
  sg.tok = nullptr;
  sg.row0 = 0;
  MfmaTile<false, ElemI8> tile;
  const int x = blockIdx.x % kXcds, step = gridDim.x / kXcds;
  const int nfull = full / kXcds, n = nfull + (pieces + kXcds - 1) / kXcds;
  for (int i = blockIdx.x / kXcds; i < n; i += step) {
    // (opaque: the decode's reciprocals are computed here, not held across the K loop)
    const int mt_ = opaque_s(sg.mtiles), nt_ = opaque_s(sg.ntiles), lgs_ = opaque_s(lgs);
    const int H = BM >> lgs_;
    int mt, nt, m0, rows;
    if (i < nfull) {
      dense_tile(x * nfull + i, mt_, nt_, mt, nt);
      m0 = mt * BM;
      rows = min(BM, sg.rows - m0);
    } else {
      const int q = x * (n - nfull) + i - nfull;
      if (q >= pieces) return;
      if (full) {
        dense_tile(full + (q >> lgs_), mt_, nt_, mt, nt);
        m0 = mt * BM + (q & ((1 << lgs_) - 1)) * H;
        if (m0 >= sg.rows) continue;  // (an m-tile of fewer rows)
      } else {
        dense_tile(q, (sg.rows + H - 1) >> (8 - lgs_), nt_, mt, nt);
        m0 = mt * H;
      }
      rows = min(H, sg.rows - m0);
    }
    const I8Cur c = i8_cur<false>(sg, m0, rows, nt);
    tile.setup(sg, c.m0, c.rows, c.n0, 0);
    const int h = __builtin_amdgcn_readfirstlane(tile.bm);
    tile.prologue(c.nk);
    i8_run<false>(tile, h, c);
    __syncthreads();  // (the ring's rows are stored before the next tile's loads overwrite them)
  }
}

template <bool GU>
void launch_stream_i8(const Seg* ss, int32_t* ms, int num_cus, int64_t max_rows, hipStream_t s) {
  const int g = 4 * num_cus;
  if (max_rows <= 16) gemm_stream_i8<GU, 1><<<g, 256, 0, s>>>(ss, ms);
  else if (max_rows <= 32) gemm_stream_i8<GU, 2><<<g, 256, 0, s>>>(ss, ms);
  else gemm_stream_i8<GU, 4><<<g, 256, 0, s>>>(ss, ms);
}

}  // namespace

hipError_t launch_gemms_i8(const SelectOut& o, int g, int num_cus, int64_t max_rows, bool stream,
                           bool mfma, hipStream_t s) {
  const Seg* ss = o.segs + (size_t)(g * kNumFam + kFamStream) * kSegCap;
  int32_t* ms = o.meta + (g * kNumFam + kFamStream) * kMetaStride;
  const Seg* sm = o.segs + (size_t)(g * kNumFam + kFamMfma) * kSegCap;
  int32_t* mm = o.meta + (g * kNumFam + kFamMfma) * kMetaStride;
  if (g == kGemmGateUp) {
    if (stream) launch_stream_i8<true>(ss, ms, num_cus, max_rows, s);
    if (mfma) gemm_mfma_i8<true><<<num_cus, 256, 0, s>>>(sm, mm);
  } else {
    if (stream) launch_stream_i8<false>(ss, ms, num_cus, max_rows, s);
    if (mfma) gemm_mfma_i8<false><<<num_cus, 256, 0, s>>>(sm, mm);
  }
  return hipGetLastError();
}

hipError_t launch_small_i8(const SmallI8& a, bool gate_up, int num_cus, hipStream_t s) {
  const int g = num_cus * (gate_up ? 4 : 5);
  if (gate_up) {
    if (a.K >= kStreamSplitK) gemm_small_i8<true, 4><<<g, 256, 0, s>>>(a);
    else gemm_small_i8<true, 2><<<g, 256, 0, s>>>(a);
  } else {
    // (64 columns per workgroup whatever K: with 16 and K split over the wavefronts four times as many
    // quantise the same rows; 64 experts of 4096 x 4096, 8 tokens: 371 us against 526)
    gemm_small_i8<false, 1><<<g, 256, small_i8_lds(a.rows, a.K), s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const void* xq, const float* xs, int M, const void* wq, const float* ws,
                          int N, int K, void* y, int num_cus, hipStream_t s) {
  if (M == 0) return hipSuccess;
  Seg sg = {};
  sg.a = xq;
  sg.as = xs;
  sg.w0 = wq;
  sg.s0 = ws;
  sg.out = y;
  sg.rows = M;
  sg.N = N;
  sg.K = K;
  // A tile's time is mostly its rows' way from L2 (tokens and weights alike), which all CUs together draw
  // at 9 (streaming) to 12 TB/s (LDS DMA), so the choice is the tile of the fewest rows times rounds of
  // CUs; an MFMA tile's rows count three quarters.  Measured with each tile forced (us): 7168 x 7168,
  // 16 tokens 1x2 12.2 (1x1 15.7, 2x2 12.9), 64 tokens 2x4 19.4 (4x4 28, 2x2 24, MFMA 41), 128 tokens 4x4
  // 26.6 (2x4 30, MFMA 40), 192 tokens MFMA 40.3 (4x4 46.6); 2048 x 7168, 64 tokens 1x2 7.8 (2x2 10.9,
  // 1x1 11.8, 4x4 20), 160 tokens 2x4 13.2 (1x2 16.9, 2x2 18.6, 4x4 20), 384 tokens 4x4 20.5 (2x4 22, 2x2
  // 26, MFMA 27); 14336 x 4096, 48 tokens 4x4 17.9 (2x4 18.8), 96 tokens MFMA 26.1 (4x4 28).
  const int g = std::max(kXcds, num_cus / kXcds * kXcds);
  sg.ntiles = (N + kMfmaBNDown - 1) / kMfmaBNDown;
  sg.mtiles = (M + BM - 1) / BM;
  const int64_t tiles = (int64_t)sg.mtiles * sg.ntiles;
  const int full = (int)(tiles / g * g);
  int lgs = 0, pieces;
  if (full) {
    while (lgs < 3 && (tiles - full) * (2 << lgs) <= g) ++lgs;
    pieces = (int)(tiles - full) << lgs;
  } else {
    // the shortest tiles that still make one round (7168 x 7168, 512 tokens: 224 tiles of 64 rows 45 us,
    // 448 of 32 73)
    auto count = [&](int l) { return (int64_t)((M + (BM >> l) - 1) / (BM >> l)) * sg.ntiles; };
    while (lgs < 3 && count(lgs + 1) <= g) ++lgs;
    pieces = (int)count(lgs);
  }
  constexpr int kTiles[][2] = {{1, 1}, {1, 2}, {2, 2}, {2, 4}, {4, 4}};  // 16 token rows x 16 weight rows
  const int groups = (M + 15) / 16;
  int64_t best = (full ? (tiles + g - 1) / g * (BM + BNW) : (BM >> lgs) + BNW) * 12;
  int mq = 0, nr = 0;
  for (const auto& c : kTiles) {
    if (c[0] >= 2 * groups) continue;
    const int64_t wgs = (int64_t)((groups + c[0] - 1) / c[0]) * ((N / 16 + c[1] - 1) / c[1]);
    const int64_t cost = (wgs + num_cus - 1) / num_cus * (c[0] + c[1]) * 16 * 16;
    if (cost > best) continue;
    best = cost;
    mq = c[0];
    nr = c[1];
  }
  if (mq) {
    sg.mtiles = (groups + mq - 1) / mq;
    sg.ntiles = (N / 16 + nr - 1) / nr;
    const unsigned grid = ((unsigned)sg.mtiles * sg.ntiles + kXcds - 1) / kXcds * kXcds;
    if (mq == 4) gemm_stream_i8_dense<4, 4><<<grid, 256, 0, s>>>(sg);
    else if (mq == 2 && nr == 4) gemm_stream_i8_dense<2, 4><<<grid, 256, 0, s>>>(sg);
    else if (mq == 2) gemm_stream_i8_dense<2, 2><<<grid, 256, 0, s>>>(sg);
    else if (nr == 2) gemm_stream_i8_dense<1, 2><<<grid, 256, 0, s>>>(sg);
    else gemm_stream_i8_dense<1, 1><<<grid, 256, 0, s>>>(sg);
    return hipGetLastError();
  }
  gemm_mfma_i8_dense<<<g, 256, 0, s>>>(sg, full, pieces, lgs);
  return hipGetLastError();
}

}  // namespace moe

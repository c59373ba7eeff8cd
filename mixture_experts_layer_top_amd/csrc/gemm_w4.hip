// Products with 4-bit weights: y = x W^T of bf16 rows, W[n][k] = (code - zero) * scale with a scale (and a
// zero point) per `group` values of a weight row; one matrix, or the gate and up pair of a SwiGLU.
//
//   y[m][n] = bf16(sum over groups of scale[n][g] * sum_{k in g} x[m][k] * (code[n][k] - zero[n][g]))
// code - zero is a whole number of at most 8 bits, exact in bf16, so a group's products are exact and
// summed in fp32 by the MFMA; the scale is applied to the group's fp32 sum.  Nothing is rounded but the sums
// themselves and the output.  (Weights scaled before the product would be rounded to bf16, 2^-9 each.)
#include "common.h"
#include "kernels.h"
#include "mfma_dev.h"
#include "rows_dev.h"

namespace moe {

namespace {

// Tiled layout, per 16 weight rows and unit of 128 columns (S = 128 / group groups):
//  codes   1 KB ordered [lane group 0..3][row][part 0..3] of dwords, part i of lane group g being values
//          32 i + 8 g .. + 7 (in the order of the row-major bytes): one 16-byte load gives a lane its operand of
//          four MFMAs, each of which covers 32 consecutive values, so that a group of 32 is one MFMA;
//  scales  [row / 4][group][row % 4]: the four rows of a lane's results, all groups, in one piece;
//  zeros   [row][group].
__global__ __launch_bounds__(256) void w4_tile_kernel(const uint32_t* __restrict__ src,
                                                      uint32_t* __restrict__ dst, int64_t n, int nkb) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  const int i = (int)(at & 3), row = (int)(at >> 2) & 15, g = (int)(at >> 6) & 3;
  const int64_t unit = at >> 8, blk = unit / nkb;
  const int kb = (int)(unit % nkb);
  dst[at] = src[((blk * 16 + row) * nkb + kb) * 16 + i * 4 + g];
}
// A thread per scale: groups = K / group of a row, S of them per unit.
__global__ __launch_bounds__(256) void w4_scale_tile_kernel(const uint16_t* __restrict__ src,
                                                            const uint8_t* __restrict__ zsrc,
                                                            uint16_t* __restrict__ dst,
                                                            uint8_t* __restrict__ zdst, int64_t n, int groups,
                                                            int S) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  const int64_t blk = at / (16 * groups);
  const int row = (int)(at / groups % 16), g = (int)(at % groups);
  const int64_t unit = (blk * (groups / S) + g / S) * (16 * S);
  dst[unit + (row >> 2) * (4 * S) + (g % S) * 4 + (row & 3)] = src[at];
  if (zsrc) zdst[unit + row * S + g % S] = zsrc[at];
}

// Four codes, one per byte in the low half (or the high half, HI), as signed bytes code - z: 128 + code - z
// never leaves a byte (z <= 127), and turning its top bit makes it two's complement.  zc = zero_bytes(z).
__device__ __forceinline__ uint32_t zero_bytes(uint32_t z) { return 0x80808080u - z * 0x01010101u; }

// Eight codes -> bf16 of code - z, in K order, exactly.  Without zero points (z = 8) the sign sits in the
// nibble's own top bit: the high half of a byte then is 16 (code - 8), and the 16 is left to the scale
// (kSymScale): the group's sum is 16 times as large, as far as fp32 goes as one with zero points of 127.  Either
// way a signed byte converts in one instruction and a pair packs in another.
constexpr float kSymScale = 0.0625f;
__device__ __forceinline__ float byte_f32(uint32_t w, int b) { return (float)(int8_t)(w >> (8 * b)); }
template <bool ZERO>
__device__ __forceinline__ bf16x8 decode8(uint32_t c, uint32_t zc) {
  uint32_t lo, hi;
  if (ZERO) {
    lo = ((c & 0x0F0F0F0Fu) + zc) ^ 0x80808080u;
    hi = (((c >> 4) & 0x0F0F0F0Fu) + zc) ^ 0x80808080u;
  } else {
    c ^= 0x88888888u;
    lo = (c << 4) & 0xF0F0F0F0u;
    hi = c & 0xF0F0F0F0u;
  }
  uint4 o;
  o.x = pack_bf16x2(byte_f32(lo, 0), byte_f32(hi, 0));
  o.y = pack_bf16x2(byte_f32(lo, 1), byte_f32(hi, 1));
  o.z = pack_bf16x2(byte_f32(lo, 2), byte_f32(hi, 2));
  o.w = pack_bf16x2(byte_f32(lo, 3), byte_f32(hi, 3));
  return as_bf16x8(o);
}

// A scale's 16 bits as a float.
__device__ __forceinline__ float scale_f32(uint32_t bits, bool fp16) {
  return fp16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : __uint_as_float(bits << 16);
}

// ------------------------------------------------------------------------------------------------
// few rows: 16 * NR weight rows (PAIR: 8 * NR of either matrix) by 16 * MQ rows of x per workgroup, whose W
// wavefronts split K (interleaved units; the sums meet in LDS in a fixed order)
//
// Weights go straight from HBM into registers, 1 KB per load, are decoded there and multiplied.  XL: all of x
// lies in LDS (few short rows): a wavefront then keeps nothing but weights in flight.  Bound by the latency of two or
// three loads in a row per wavefront and a launch, then by HBM: group 128, 1 x 7168 x 7168 10.7 us (2.6 TB/s),
// 1 x 14336 x 4096 10.8 (2.8); 64 x 7168 x 7168 23 us, 128 41: by L2, which gives x anew to every 64 weight rows.
// (16 wavefronts along K, or four units a batch instead of two: 12.9 and 10.3 us for 1 x 7168 x 7168, but group 32,
// 1 x 14336 x 4096 16.4 and 18.5 instead of 13.5.)
// ------------------------------------------------------------------------------------------------
constexpr int kXlBytes = 64 << 10;
constexpr int64_t xl_stride(int K) { return (int64_t)K * 2 + 64; }  // (rows start in different banks)

template <int MQ, int NR, int GROUP, bool PAIR, bool ZERO, int W, bool XL, bool FP16>
__device__ __forceinline__ void stream_w4(const W4Args& a, uint8_t* lds) {
  constexpr int S = 128 / GROUP, F = GROUP / 32;  // groups per unit, MFMAs per group
  constexpr int U = MQ == 1 ? 2 : 1;              // units per batch (by registers)
  constexpr bool HALF = PAIR && NR == 1;          // 8 rows of either matrix in one fragment, rows 8.. the second's
  constexpr int PC = PAIR && !HALF ? 2 : 1;       // accumulators per output
  constexpr int P = MQ * NR / PC;                 // outputs (16 x 16) per wavefront
  float* const red = reinterpret_cast<float*>(lds);  // [P][W - 1][PC * 4][64]
  uint8_t* const xl = lds + P * (W - 1) * PC * 1024;
  const int lane = threadIdx.x & 63, kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = a.K, nkb = K / 128, nblk = a.N / 16;
  const int m0 = (blockIdx.x % a.mtiles) * (16 * MQ), rows = min(16 * MQ, a.M - m0);
  const int n0 = (blockIdx.x / a.mtiles) * (HALF ? 8 : 16 * NR / PC);  // first weight row
  const int b0 = n0 / 16;                                             // and its 16-row block
  const int hn = HALF ? n0 % 16 + (r16 & 7) : r16, hs = HALF ? n0 % 16 / 4 + (kg & 1) : kg;
  uint32_t unit0[NR], xoff[MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)  // (a block past N re-reads the last one; never stored)
    unit0[j] = (uint32_t)min(b0 + j / PC, nblk - 1) * (uint32_t)nkb;
#pragma unroll
  for (int q = 0; q < MQ; ++q) {  // (a row past the last re-reads it; never stored)
    const int r = min(q * 16 + r16, rows - 1);
    xoff[q] = XL ? (uint32_t)(r * (int)xl_stride(K) + kg * 16) : ((uint32_t)(m0 + r) * (uint32_t)K + kg * 8) * 2;
  }
  f32x4 tot[NR][MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int q = 0; q < MQ; ++q) tot[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    uint4 w[U][NR], x[XL ? 1 : U][MQ][4];
    uint32_t s[U][NR][2 * S], z[ZERO ? U : 1][NR];
  };
  const int nc = (nkb - kw + W - 1) / W;  // this wavefront's units: kw, kw + W, ...
  auto load = [&](Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)min(kw + W * (i + u), nkb - 1);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        // (of a fragment of both matrices lane by lane; a scale is its result's row's, the rest its operand's)
        const int mc = HALF ? r16 >> 3 : PAIR ? j & 1 : 0, ms = HALF ? kg >> 1 : mc;
        const size_t unit = unit0[j] + kb;
        const char* codes = static_cast<const char*>(a.m[mc].codes) + unit * 1024;
        const uint32_t at = kg * 256 + hn * 16;
        bt.w[u][j] = a.mtiles == 1 ? gload16_nt(codes, at) : gload16(codes, at);
        const char* sc = static_cast<const char*>(a.m[ms].scales) + unit * (32 * S);
        if (S == 1) {
          const uint2 v = gload8(sc, hs * 8);
          bt.s[u][j][0] = v.x;
          bt.s[u][j][1] = v.y;
        } else {
#pragma unroll
          for (int g = 0; g < S / 2; ++g) {
            const uint4 v = gload16(sc, hs * (8 * S) + g * 16);
            bt.s[u][j][4 * g] = v.x;
            bt.s[u][j][4 * g + 1] = v.y;
            bt.s[u][j][4 * g + 2] = v.z;
            bt.s[u][j][4 * g + 3] = v.w;
          }
        }
        if (ZERO) {
          const uint8_t* z = a.m[mc].zeros + unit * (16 * S);
          bt.z[ZERO ? u : 0][j] = S == 1 ? gload_u8(z, hn) : S == 2 ? gload_u16(z, hn * 2) : gload4(z, hn * 4);
        }
      }
      if (!XL) {
#pragma unroll
        for (int q = 0; q < MQ; ++q)
#pragma unroll
          for (int f = 0; f < 4; ++f) bt.x[XL ? 0 : u][q][f] = gload16(a.x, xoff[q] + (kb * 128 + f * 32) * 2);
      }
    }
  };
  auto compute = [&](const Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= nc) break;
      const uint32_t kb = kw + W * (i + u);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const uint32_t c[4] = {bt.w[u][j].x, bt.w[u][j].y, bt.w[u][j].z, bt.w[u][j].w};
#pragma unroll
        for (int g = 0; g < S; ++g) {
          const W4Mat& m = a.m[HALF ? r16 >> 3 : PAIR ? j & 1 : 0];
          const uint32_t z = ZERO ? zero_bytes(m.zero(bt.z[ZERO ? u : 0][j] >> (8 * g))) : 0u;
          float sc[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sc[r] = scale_f32(bt.s[u][j][2 * g + (r >> 1)] >> (16 * (r & 1)) & 0xFFFF, FP16) *
                    (ZERO ? 1.0f : kSymScale);
          f32x4 acc[MQ];
#pragma unroll
          for (int q = 0; q < MQ; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < F; ++f) {
            const bf16x8 wf = decode8<ZERO>(c[g * F + f], z);
#pragma unroll
            for (int q = 0; q < MQ; ++q) {
              const uint4 xv = XL ? *reinterpret_cast<const uint4*>(xl + xoff[q] + kb * 256 + (g * F + f) * 64)
                                  : bt.x[XL ? 0 : u][q][g * F + f];
              acc[q] = mfma16(wf, as_bf16x8(xv), acc[q]);
            }
          }
#pragma unroll
          for (int q = 0; q < MQ; ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r) tot[j][q][r] = fmaf(sc[r], acc[q][r], tot[j][q][r]);
        }
      }
    }
  };
  Batch c0, c1;
  if constexpr (XL) {  // (one tile of rows: m0 = 0)
    // the first pieces of x, then both batches of weights behind them; the barrier waits for LDS alone
    constexpr int A = 2;
    const int per = K / 8, n = rows * per;  // 16-byte pieces of a row, of x
    auto place = [&](int i) { return reinterpret_cast<uint4*>(xl + (i / per) * (int)xl_stride(K) + (i % per) * 16); };
    uint4 v[A];
#pragma unroll
    for (int q = 0; q < A; ++q) v[q] = gload16(a.x, (uint32_t)min((int)threadIdx.x + q * 64 * W, n - 1) * 16);
    if (nc > 0) load(c0, 0);
    if (U < nc) load(c1, U);
#pragma unroll
    for (int q = 0; q < A; ++q)
      if ((int)threadIdx.x + q * 64 * W < n) *place(threadIdx.x + q * 64 * W) = v[q];
    for (int i = threadIdx.x + A * 64 * W; i < n; i += 64 * W) *place(i) = gload16(a.x, (uint32_t)i * 16);
    asm volatile("" ::: "memory");
    MOE_WAITCNT(63, 0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  } else {
    if (nc > 0) load(c0, 0);
  }
  for (int i = 0; i < nc; i += 2 * U) {
    if (i + U < nc && !(XL && i == 0)) load(c1, i + U);
    compute(c0, i);
    if (i + 2 * U < nc) load(c0, i + 2 * U);
    if (i + U < nc) compute(c1, i + U);
  }
  // every wavefront parks its sums but those of the outputs it finishes itself: output p goes to wavefront
  // p % W, slot order (p, wavefront)
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % W == kw) continue;
    float* dst = red + (p * (W - 1) + (kw < p % W ? kw : kw - 1)) * (PC * 256) + lane;
#pragma unroll
    for (int c = 0; c < PC; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[(c * 4 + r) * 64] = tot[p / MQ * PC + c][p % MQ][r];
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % W != kw) continue;
    const float* src = red + p * (W - 1) * (PC * 256) + lane;
    float v[PC][4];
#pragma unroll
    for (int c = 0; c < PC; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[c][r] = tot[p / MQ * PC + c][p % MQ][r];
#pragma unroll
        for (int w = 0; w < W - 1; ++w) v[c][r] += src[w * (PC * 256) + (c * 4 + r) * 64];
      }
    // lane holds weight rows 4 kg + r of row r16 of x
    const int r = p % MQ * 16 + r16, b = b0 + p / MQ;
    if (PAIR) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = swiglu(v[0][e], HALF ? __shfl_xor(v[0][e], 32) : v[PC - 1][e]);
    }
    if (r >= rows || b >= nblk || (HALF && kg >= 2)) continue;
    gstore8(a.y, ((size_t)(m0 + r) * a.N + b * 16 + 4 * hs) * 2,
            uint2{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3])});
  }
}

// ------------------------------------------------------------------------------------------------
// middling rows: 128 weight rows (PAIR: 64 of either matrix) by 16 * MQ = 64 or 128 rows of x per workgroup
//
// 8 wavefronts: two halves of K, each with its own units and its own ring of x in LDS, by four of 32 weight rows.  A
// stage is two units of either half (128 rows of x: one); loads run one stage ahead, x by global_load_lds, weights
// into registers as in the streaming tiles.  Group 128, 256 x 7168 x 7168 46 us, 512 71 us (0.57 and 0.74 PFLOP/s):
// bound by issue, decoding for 64 or 128 rows of x at a time, and by L2, one after the other where they do not
// overlap (256 rows without the loads 37 us, without the products 29, 10.6 TB/s).  Reading and decoding a piece ahead
// and interleaving it with the MFMAs gained 1 to 4% and spilled registers with groups of 32; four parts of K with 64
// weight rows each gained 3% and spilled alike.
// ------------------------------------------------------------------------------------------------
constexpr int kMidRing = 128 << 10;

template <int GROUP, bool PAIR, bool ZERO, int MQ, bool FP16>
__device__ __forceinline__ void mid_w4(const W4Args& a, int nblocks, uint8_t* ring) {
  constexpr int S = 128 / GROUP, F = GROUP / 32;
  constexpr int NR = 2, WK = 2, WN = 4, PC = PAIR ? 2 : 1, M = 16 * MQ;
  constexpr int kUnit = M * 256, U = kMidRing / (2 * WK * kUnit);  // bytes of x, units of a stage and half
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wv / WN, wn = wv % WN;
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = a.K, nkb = K / 128, nblk = a.N / 16, steps = (nkb + WK * U - 1) / (WK * U);
  // (every XCD takes an eighth of the tiles in a row, those of a weight block one behind the other: its L2 then
  // reads the block once)
  const int tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  if (tile >= nblocks * a.mtiles) return;
  const int m0 = tile % a.mtiles * M, b0 = tile / a.mtiles * (8 / PC) + wn * (NR / PC);
  uint32_t unit0[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j)  // (a block past N re-reads the last one; never stored)
    unit0[j] = (uint32_t)min(b0 + j / PC, nblk - 1) * (uint32_t)nkb;
  f32x4 tot[NR][MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int t = 0; t < MQ; ++t) tot[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    uint4 w[U][NR];
    uint32_t s[U][NR][2 * S], z[ZERO ? U : 1][NR];
  };
  auto load_x = [&](int i, int stage) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int l = wn * 8 + q, u = l / (M / 4), r4 = l % (M / 4);
      const int kb = min((i * WK + wk) * U + u, nkb - 1);
      const int row = 4 * r4 + (tid_here() >> 4 & 3), piece = (tid_here() & 15) ^ (row & 15);
      const uint32_t off = (uint32_t)min(m0 + row, a.M - 1) * (uint32_t)(K * 2) + piece * 16;
      dma16(static_cast<const char*>(a.x) + (size_t)kb * 256, off,
            (lds_void*)(ring + ((wk * 2 + stage) * U + u) * kUnit + r4 * 1024));
    }
  };
  auto load = [&](Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)min((i * WK + wk) * U + u, nkb - 1);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const W4Mat& m = a.m[PAIR ? j & 1 : 0];
        const size_t unit = unit0[j] + kb;
        bt.w[u][j] = gload16(static_cast<const char*>(m.codes) + unit * 1024, lane * 16);
        const char* sc = static_cast<const char*>(m.scales) + unit * (32 * S);
        if (S == 1) {
          const uint2 v = gload8(sc, kg * 8);
          bt.s[u][j][0] = v.x;
          bt.s[u][j][1] = v.y;
        } else {
#pragma unroll
          for (int g = 0; g < S / 2; ++g) {
            const uint4 v = gload16(sc, kg * (8 * S) + g * 16);
            bt.s[u][j][4 * g] = v.x;
            bt.s[u][j][4 * g + 1] = v.y;
            bt.s[u][j][4 * g + 2] = v.z;
            bt.s[u][j][4 * g + 3] = v.w;
          }
        }
        if (ZERO) {
          const uint8_t* z = m.zeros + unit * (16 * S);
          bt.z[ZERO ? u : 0][j] = S == 1 ? gload_u8(z, r16) : S == 2 ? gload_u16(z, r16 * 2) : gload4(z, r16 * 4);
        }
      }
    }
  };
  auto landed = [&](Batch& bt) {  // (a wait for registers behind the next stage's loads would wait for those too)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        uint4& w = bt.w[u][j];
        asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
#pragma unroll
        for (int g = 0; g < 2 * S; ++g) asm volatile("" : "+v"(bt.s[u][j][g]));
        if (ZERO) asm volatile("" : "+v"(bt.z[ZERO ? u : 0][j]));
      }
  };
  auto compute = [&](const Batch& bt, int i, int stage) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((i * WK + wk) * U + u >= nkb) break;
      uint32_t xa = ((wk * 2 + stage) * U + u) * kUnit + r16 * 256 + (kg ^ (r16 & 3)) * 16 + (r16 >> 2) * 64;
      asm volatile("" : "+v"(xa));
#pragma unroll
      for (int g = 0; g < S; ++g) {
        bf16x8 wf[NR][F];
        float sc[NR][4];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const uint32_t c[4] = {bt.w[u][j].x, bt.w[u][j].y, bt.w[u][j].z, bt.w[u][j].w};
          const uint32_t z = ZERO ? zero_bytes(a.m[PAIR ? j & 1 : 0].zero(bt.z[ZERO ? u : 0][j] >> (8 * g))) : 0u;
#pragma unroll
          for (int f = 0; f < F; ++f) wf[j][f] = decode8<ZERO>(c[g * F + f], z);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sc[j][r] = scale_f32(bt.s[u][j][2 * g + (r >> 1)] >> (16 * (r & 1)) & 0xFFFF, FP16) *
                       (ZERO ? 1.0f : kSymScale);
        }
        // (64 rows of x at a time: twice as many accumulators would not fit the registers beside the totals)
#pragma unroll
        for (int h = 0; h < MQ; h += 4) {
          f32x4 acc[NR][4];
#pragma unroll
          for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < F; ++f)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const bf16x8 xf = as_bf16x8(
                  *reinterpret_cast<const uint4*>(ring + ((xa ^ ((g * F + f) * 64)) + (h + t) * 4096)));
#pragma unroll
              for (int j = 0; j < NR; ++j) acc[j][t] = mfma16(wf[j][f], xf, acc[j][t]);
            }
#pragma unroll
          for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int r = 0; r < 4; ++r) tot[j][h + t][r] = fmaf(sc[j][r], acc[j][t][r], tot[j][h + t][r]);
          if (MQ > 4) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  Batch c0, c1;
  auto step = [&](Batch& now, Batch& next, int i, int stage) {
    MOE_WAITCNT(0, 15);  // this stage has landed
    landed(now);
    __syncthreads();  // for every wavefront; and all have read the other one
    load_x(min(i + 1, steps - 1), stage ^ 1);
    load(next, min(i + 1, steps - 1));
    compute(now, i, stage);
  };
  load_x(0, 0);
  load(c0, 0);
  for (int i = 0; i < steps; i += 2) {
    step(c0, c1, i, 0);
    if (i + 1 < steps) step(c1, c0, i + 1, 1);
  }
  MOE_WAITCNT(0, 15);
  __syncthreads();
  // every wavefront parks its sums but those of the tiles it finishes itself: tile t goes to wavefront t % WK
  auto slot = [&](int t, int from, int j) {
    const int at = (t * (WK - 1) + (from < t % WK ? from : from - 1)) * NR + j;
    return reinterpret_cast<f32x4*>(ring) + (wn * (MQ * (WK - 1) * NR) + at) * 64 + lane;
  };
#pragma unroll
  for (int t = 0; t < MQ; ++t)
#pragma unroll
    for (int j = 0; j < NR; ++j)
      if (t % WK != wk) *slot(t, wk, j) = tot[j][t];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MQ; ++t) {
    if (t % WK != wk) continue;
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int w = 0; w < WK; ++w)
        if (w != t % WK) tot[j][t] += *slot(t, w, j);
    // lane holds weight rows 4 kg + r of row r16 of x
    const int r = m0 + t * 16 + r16;
#pragma unroll
    for (int j = 0; j < NR; j += PC) {
      f32x4 v = tot[j][t];
      if (PAIR) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = swiglu(v[e], tot[j + PC - 1][t][e]);
      }
      const int b = b0 + j / PC;
      if (r < a.M && b < nblk)
        gstore8(a.y, ((size_t)r * a.N + b * 16 + 4 * kg) * 2, uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    }
  }
}
template <int GROUP, bool PAIR, bool ZERO, int MQ>
__global__ __launch_bounds__(512) void gemm_mid_w4(W4Args a, int nblocks) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kMidRing];
  if (a.fp16) mid_w4<GROUP, PAIR, ZERO, MQ, true>(a, nblocks, ring);
  else mid_w4<GROUP, PAIR, ZERO, MQ, false>(a, nblocks, ring);
}
template <int GROUP, bool PAIR, bool ZERO, int MQ>
hipError_t launch_mid(W4Args a, hipStream_t s) {
  a.mtiles = (a.M + 16 * MQ - 1) / (16 * MQ);
  const int nblocks = (a.N / 16 + (PAIR ? 3 : 7)) / (PAIR ? 4 : 8);
  gemm_mid_w4<GROUP, PAIR, ZERO, MQ><<<(unsigned)(a.mtiles * nblocks + 7) / 8 * 8, 512, 0, s>>>(a, nblocks);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------
// many rows: 256 weight rows (PAIR: 128 of either matrix) by 128 rows of x per workgroup
//
// Each of the 4 wavefronts holds 64 weight rows and all 128 rows of x: a weight is decoded by one wavefront,
// from registers, once for 128 rows, and only x goes through LDS as operands (global_load_lds, two stages of
// 128 columns).  A group's sums are four chained MFMAs from zero (one per 32 columns); the scale takes them to
// the totals while the next ones run.  Here x is the MFMA's first operand: a lane then holds one weight row per
// fragment, and one scale.  Bound by the SIMDs' issue: 4096 x 14336 x 4096, group 128, 395 to 433 us by the clock
// (1.1 to 1.2 PFLOP/s; the library's bf16 product of this size 406), MFMAs in 0.53 of the cycles and decoding and
// scaling in 0.53; group 32, whose scales are four times as many, 552.  Wave priorities and a stagger of the
// wavefronts gave nothing.
// ------------------------------------------------------------------------------------------------
constexpr int kTileM = 128;
constexpr int kXStage = kTileM * 256;  // bytes: rows of 16 pieces of 16 bytes, swizzled by the row

template <int GROUP, bool PAIR, bool ZERO>
__global__ __launch_bounds__(256, 2) void gemm_tile_w4(W4Args a) {
  constexpr int S = 128 / GROUP, F = GROUP / 32;
  constexpr int C = PAIR ? 2 : 4;  // consecutive weight rows of a lane
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * kXStage + 4 * 4096];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = a.K, nkb = K / 128;
  const int m0 = (blockIdx.x % a.mtiles) * kTileM;
  const int n0 = (blockIdx.x / a.mtiles) * (64 * C) + wv * (16 * C);
  // Row r of fragment j is weight row n0 + C r + j % C (of matrix j / 2 of a pair): a lane's results are
  // consecutive columns of y.  (Rows past N re-read the last ones; never stored.)
  const int nl = min(n0 + C * r16, a.N - C);
  // of the lane's 16 bytes of fragment 0 in the first unit; the next rows' follow
  const uint32_t woff = (uint32_t)(nl >> 4) * (uint32_t)(nkb * 1024) + kg * 256 + (nl & 15) * 16;
  f32x4 tot[4][8];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < 8; ++t) tot[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // 8 of the stage's 32 kilobytes: rows 32 wv + 4 q .. + 3 in load q
  auto load_x = [&](int kb, int stage) {
    const char* base = static_cast<const char*>(a.x) + (size_t)kb * 256;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = 32 * wv + 4 * q + (tid_here() >> 4 & 3);
      const int piece = (tid_here() & 15) ^ (row & 15);
      const uint32_t off = (uint32_t)min(m0 + row, a.M - 1) * (uint32_t)(K * 2) + piece * 16;
      dma16(base, off, (lds_void*)(ring + stage * kXStage + (32 * wv + 4 * q) * 256));
    }
  };
  // A wavefront's codes of a chunk, one kilobyte per fragment, as its lanes hold them.
  uint8_t* const codes = ring + 2 * kXStage + wv * 4096;
  auto load_codes = [&](int kb) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dma16(static_cast<const char*>(a.m[PAIR ? j >> 1 : 0].codes) + (size_t)kb * 1024 + (j % C) * 16, woff,
            (lds_void*)(codes + j * 1024));
  };
  // Scales (16 bits per row) and zero points (8) of a chunk wait in registers.
  uint32_t sc[S][2], zb[C * S / 4 ? C * S / 4 : 1][PAIR ? 2 : 1];
  auto load_scales = [&](int kb) {
    // (opaque: the compiler would keep a 64-bit address for each of these loads)
    uint32_t at = woff;
    asm volatile("" : "+v"(at));
    at = (at >> 10) * (16 * S);  // (16 rows of every group)
    const uint32_t e = at + ((nl & 15) >> 2) * (4 * S) + (nl & 3), ze = at + (nl & 15) * S;
#pragma unroll
    for (int c = 0; c < (PAIR ? 2 : 1); ++c) {
      const char* s = static_cast<const char*>(a.m[c].scales) + (size_t)kb * (32 * S);
#pragma unroll
      for (int g = 0; g < S; ++g) {
        if (PAIR) {
          sc[g][c] = gload4(s, (e + g * 4) * 2);
        } else {
          const uint2 v = gload8(s, (e + g * 4) * 2);
          sc[g][0] = v.x;
          sc[g][1] = v.y;
        }
      }
      if (ZERO) {
        const uint8_t* z = a.m[c].zeros + (size_t)kb * (16 * S);
        if (C * S == 2) {
          zb[0][c] = gload_u16(z, ze);
        } else {
#pragma unroll
          for (int i = 0; i < C * S / 4; ++i) zb[i][c] = gload4(z, ze + 4 * i);
        }
      }
    }
  };
  load_x(0, 0);
  load_codes(0);
  load_scales(0);
  for (int kb = 0; kb < nkb; ++kb) {
    const int st = kb & 1;
    MOE_WAITCNT(0, 15);  // this chunk has landed
    __syncthreads();     // for every wavefront; and all have read the other stage
    // (the last chunk loads itself again: without a branch the loop's body is one block)
    const int next = min(kb + 1, nkb - 1);
    load_x(next, st ^ 1);
    uint4 code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) code[j] = *reinterpret_cast<const uint4*>(codes + j * 1024 + lane * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)  // (in registers before the next chunk's take their place)
      asm volatile("" : "+v"(code[j].x), "+v"(code[j].y), "+v"(code[j].z), "+v"(code[j].w));
    load_codes(next);
    uint32_t xa = st * kXStage + r16 * 256 + (kg ^ (r16 & 3)) * 16 + (r16 >> 2) * 64;
    asm volatile("" : "+v"(xa));
#pragma unroll
    for (int g = 0; g < S; ++g) {
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b = sc[g][j >> 1] >> (16 * (j & 1));
        s[j] = (a.fp16 ? scale_f32(b & 0xFFFF, true) : scale_f32(b & 0xFFFF, false)) * (ZERO ? 1.0f : kSymScale);
      }
      bf16x8 wf[4][F];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
        const int zi = (j % C) * S + g;  // (row by row, its groups)
        const uint32_t z = ZERO ? zb[zi / 4][PAIR ? j >> 1 : 0] >> (8 * (zi % 4)) : 0u;
#pragma unroll
        for (int f = 0; f < F; ++f)
          wf[j][f] = decode8<ZERO>(c[g * F + f], ZERO ? zero_bytes(a.m[PAIR ? j >> 1 : 0].zero(z)) : 0u);
      }
      // (behind the last use of this chunk's; the loop's head waits for them)
      if (g == S - 1) load_scales(next);
      // row r16 of tile t, piece 4 f' + kg (f' = g F + f) at place (4 f' + kg) ^ r16
      auto read_x = [&](int t, int f) {
        return as_bf16x8(*reinterpret_cast<const uint4*>(ring + ((xa ^ ((g * F + f) * 64)) + t * 4096)));
      };
      // Operand f of tile t lies in slot (F t + f) mod X: a tile's first is read ahead, the rest as the tile before
      // has used its own up (with a whole second tile's the registers do not suffice).
      constexpr int X = F + 1;
      bf16x8 xf[X];
#pragma unroll
      for (int f = 0; f < F; ++f) xf[f] = read_x(0, f);
      f32x4 acc[2][2];
#pragma unroll
      for (int i = 0; i <= 16; ++i) {  // fragments 2 (i % 2) and + 1 of tile i / 2, and the totals of the ones before
        const int t = i >> 1, j = (i & 1) * 2;
        if (i < 16) {
          __builtin_amdgcn_sched_barrier(0);
          if (j == 0 && t < 7) {
#pragma unroll
            for (int f = 0; f < X - F; ++f) xf[(F * (t + 1) + f) % X] = read_x(t + 1, f);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[i & 1][e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < F; ++f) {
#pragma unroll
            for (int e = 0; e < 2; ++e) acc[i & 1][e] = mfma16(xf[(F * t + f) % X], wf[j + e][f], acc[i & 1][e]);
            if (j == 2 && t < 7 && f + X - F < F) xf[(F * (t + 1) + f + X - F) % X] = read_x(t + 1, f + X - F);
          }
        }
        if (i > 0) {
          const int u = (i - 1) >> 1, v = ((i - 1) & 1) * 2;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int r = 0; r < 4; ++r) tot[v + e][u][r] = fmaf(s[v + e], acc[(i - 1) & 1][e][r], tot[v + e][u][r]);
          }
          if (i < 16) {
#pragma unroll
            for (int q = 0; q < 2 * F; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 8 / (2 * F) ? 8 / (2 * F) : 1, 0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          // (the sums are taken here: moved behind the chunk's other MFMAs they would keep every acc)
          asm volatile("" : "+v"(tot[v][u]));
          asm volatile("" : "+v"(tot[v + 1][u]));
        }
      }
    }
  }
  MOE_WAITCNT(0, 15);  // (no load may still be on its way to LDS when the workgroup ends)
  // lane holds rows 4 kg + r of tile t, columns nl .. + C - 1
  if (n0 + C * r16 >= a.N) return;
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = m0 + t * 16 + kg * 4 + r;
      if (row >= a.M) continue;
      const size_t at = ((size_t)row * a.N + nl) * 2;
      if (PAIR)
        gstore4(a.y, at, pack_bf16x2(swiglu(tot[0][t][r], tot[2][t][r]), swiglu(tot[1][t][r], tot[3][t][r])));
      else
        gstore8(a.y, at, uint2{pack_bf16x2(tot[0][t][r], tot[1][t][r]), pack_bf16x2(tot[2][t][r], tot[3][t][r])});
    }
}

// (One loop per type of scale: with the choice inside it the sums would be taken behind a branch, where every
// accumulator has to be kept.)
template <int MQ, int NR, int GROUP, bool PAIR, bool ZERO, int W, bool XL>
__global__ __launch_bounds__(64 * W) void gemm_stream_w4(W4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  if (a.fp16) stream_w4<MQ, NR, GROUP, PAIR, ZERO, W, XL, true>(a, lds);
  else stream_w4<MQ, NR, GROUP, PAIR, ZERO, W, XL, false>(a, lds);
}

template <int MQ, int NR, int GROUP, bool PAIR, bool ZERO, int W, bool XL>
hipError_t launch_stream(W4Args a, hipStream_t s) {
  constexpr int rows = PAIR ? 8 * NR : 16 * NR;  // (of a matrix)
  a.mtiles = (a.M + 16 * MQ - 1) / (16 * MQ);
  const unsigned grid = (unsigned)a.mtiles * ((a.N + rows - 1) / rows);
  const int lds = MQ * NR * (W - 1) * 1024 + (XL ? a.M * (int)xl_stride(a.K) : 0);
  gemm_stream_w4<MQ, NR, GROUP, PAIR, ZERO, W, XL><<<grid, 64 * W, lds, s>>>(a);
  return hipGetLastError();
}
// More than 32 rows of x: the streaming tiles where the middling ones would not be enough workgroups; these with 64
// rows of x for up to one workgroup per CU, with 128 where that is no more than one (groups of 32: two), with 64 up to
// two; the MFMA tiles beyond.  Microseconds at rows x weight rows x columns (workgroups with 64 rows of x per CU): streaming
// and 64 rows, group 128, 128 x 7168 x 7168 (0.4) 41 and 45, 192 x 6144 x 4096 (0.6) 40 and 27, 256 x 7168 x 7168 (0.9)
// 79 and 46; group 64, 256 x 3584 x 4096 (0.4) 41 and 29; group 32 pair, 256 x 2048 x 7168 (0.5) 70 and 57.  64 rows,
// 128 and MFMA tiles, group 128, 256 x 7168 x 7168 (0.9) 47, 68 and 121, 512 (1.75) 88, 71 and 122, 1024 (3.5) 178,
// 135 and 124, 2048 x 2048 x 2048 (2) 38, 27 and 39; group 32 pair, 1024 x 2048 x 7168 (2) 118, 90 and 193, 2048 (4)
// 247, 187 and 213.  Up to 32 rows half of a middling tile or more would be idle: 24 x 28672 x 4096 (0.9) 27 and 31.
template <int GROUP, bool PAIR, bool ZERO>
hipError_t launch_tiles(W4Args a, int num_cus, hipStream_t s) {
  const int64_t blocks = a.N / 16 * (PAIR ? 2 : 1), mtiles = (a.M + 31) / 32;
  const int64_t mid64 = (mtiles + 1) / 2 * ((blocks + 7) / 8), mid128 = (mtiles + 3) / 4 * ((blocks + 7) / 8);
  if (a.M > 32 && mid64 > (GROUP == 128 ? num_cus / 2 : num_cus / 8 * 3)) {
    if (mid64 > num_cus && mid128 <= num_cus) return launch_mid<GROUP, PAIR, ZERO, 8>(a, s);
    if (mid64 <= 2 * num_cus) return launch_mid<GROUP, PAIR, ZERO, 4>(a, s);
    if (GROUP == 32 && mid128 <= 2 * num_cus) return launch_mid<GROUP, PAIR, ZERO, 8>(a, s);
    a.mtiles = (a.M + kTileM - 1) / kTileM;
    const int64_t grid = (int64_t)a.mtiles * ((a.N + (PAIR ? 127 : 255)) / (PAIR ? 128 : 256));
    gemm_tile_w4<GROUP, PAIR, ZERO><<<(unsigned)grid, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  if (a.M <= 16) {
    // x in LDS where it fits (1 x 7168 x 7168 11.2 us, 12.3 with x from L2; 16 rows of 7168 do not).  16 weight rows
    // a workgroup (of a pair 8 of either matrix) where that is no more than one per CU: pair 1 x 2048 x 7168 10.4 us,
    // 12.7 with 32, 1 x 3200 x 7168 13.8 and 13.1; one matrix, 16 x 2048 x 7168 10.8 and 12.8, 16 x 4096 x 7168 11.7
    // and 13.6, with groups of 32 12.4 and 15.0, 16 x 7168 x 7168 19.6 and 14.1.
    const bool narrow = blocks <= num_cus;
    if (a.M * xl_stride(a.K) <= kXlBytes) {
      if constexpr (PAIR) {
        if (!narrow) return launch_stream<1, 2, GROUP, PAIR, ZERO, 8, true>(a, s);
      }
      return launch_stream<1, 1, GROUP, PAIR, ZERO, 8, true>(a, s);
    }
    return narrow ? launch_stream<1, 1, GROUP, PAIR, ZERO, 8, false>(a, s)
                  : launch_stream<1, 2, GROUP, PAIR, ZERO, 8, false>(a, s);
  }
  // 64 weight rows a workgroup halve what is read of x, where there are workgroups for half the CUs (64 x 7168 x
  // 7168 23 us, 33 with 32; 64 x 2048 x 2048 8.9 and 7.4).  Groups of 128 only: the registers hold no more scales.
  if constexpr (GROUP == 128) {
    if (2 * mtiles * ((blocks + 3) / 4) >= num_cus) return launch_stream<2, 4, GROUP, PAIR, ZERO, 8, false>(a, s);
  }
  return launch_stream<2, 2, GROUP, PAIR, ZERO, 8, false>(a, s);
}
template <int GROUP>
hipError_t launch_group(const W4Args& a, int cus, hipStream_t s) {
  const bool zero = a.m[0].zeros;  // (of either matrix, kernels.h)
  if (a.m[1].codes)
    return zero ? launch_tiles<GROUP, true, true>(a, cus, s) : launch_tiles<GROUP, true, false>(a, cus, s);
  return zero ? launch_tiles<GROUP, false, true>(a, cus, s) : launch_tiles<GROUP, false, false>(a, cus, s);
}

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, int group, int num_cus, hipStream_t s) {
  return group == 32   ? launch_group<32>(a, num_cus, s)
         : group == 64 ? launch_group<64>(a, num_cus, s) : launch_group<128>(a, num_cus, s);
}

hipError_t launch_w4_tile(const W4Mat& src, int N, int K, int group, void* codes, void* scales, uint8_t* zeros,
                          hipStream_t s) {
  const int64_t nw = (int64_t)N * K / 8, ns = (int64_t)N * (K / group);
  w4_tile_kernel<<<(unsigned)((nw + 255) / 256), 256, 0, s>>>(static_cast<const uint32_t*>(src.codes),
                                                              static_cast<uint32_t*>(codes), nw, K / 128);
  w4_scale_tile_kernel<<<(unsigned)((ns + 255) / 256), 256, 0, s>>>(
      static_cast<const uint16_t*>(src.scales), src.zeros, static_cast<uint16_t*>(scales), zeros, ns, K / group,
      128 / group);
  return hipGetLastError();
}

}  // namespace moe

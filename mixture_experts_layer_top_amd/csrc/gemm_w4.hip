// Products with 4-bit weights: y = x W^T of bf16 rows, W[n][k] = (code - zero) * scale with a scale (and a
// zero point) per `group` values of a weight row; one matrix, or the gate and up pair of a SwiGLU.
//
//   y[m][n] = bf16(sum over groups of scale[n][g] * sum_{k in g} x[m][k] * (code[n][k] - zero[n][g]))
// code - zero is a whole number of at most 8 bits, exact in bf16, so a group's products are exact and
// summed in fp32 by the MFMA; the scale is applied to the group's fp32 sum.  Nothing is rounded but the sums
// themselves and the output.  (Weights scaled before the product would be rounded to bf16, 2^-9 each.)
#include "common.h"
#include "kernels.h"
#include "rows_dev.h"

namespace moe {

namespace {

// Tiled layout: per 16 weight rows and 128 values of K, 1 KB ordered [lane group 0..3][row][part 0..3] of
// dwords, part i of lane group g being values 32 i + 8 g .. + 7 (in the order of the row-major bytes): one
// 16-byte load gives a lane its operand of four MFMAs, each of which covers 32 consecutive values, so that a
// group of 32 is one MFMA.  Scales and zeros [block][group][row].
__global__ __launch_bounds__(256) void w4_tile_kernel(const uint32_t* __restrict__ src,
                                                      uint32_t* __restrict__ dst, int64_t n, int nkb) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  const int i = (int)(at & 3), row = (int)(at >> 2) & 15, g = (int)(at >> 6) & 3;
  const int64_t unit = at >> 8, blk = unit / nkb;
  const int kb = (int)(unit % nkb);
  dst[at] = src[((blk * 16 + row) * nkb + kb) * 16 + i * 4 + g];
}
template <class T>
__global__ __launch_bounds__(256) void w4_scale_tile_kernel(const T* __restrict__ src, T* __restrict__ dst,
                                                            int64_t n, int groups) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  const int row = (int)(at & 15);
  const int64_t unit = at >> 4, blk = unit / groups;
  dst[at] = src[(blk * 16 + row) * groups + unit % groups];
}

// Eight codes -> bf16 of code - z, in K order.
__device__ __forceinline__ bf16x8 decode8(uint32_t c, float z) {
  const uint32_t lo = c & 0x0F0F0F0Fu, hi = (c >> 4) & 0x0F0F0F0Fu;
  uint4 o;
  o.x = pack_bf16x2(float(lo & 255) - z, float(hi & 255) - z);
  o.y = pack_bf16x2(float((lo >> 8) & 255) - z, float((hi >> 8) & 255) - z);
  o.z = pack_bf16x2(float((lo >> 16) & 255) - z, float((hi >> 16) & 255) - z);
  o.w = pack_bf16x2(float(lo >> 24) - z, float(hi >> 24) - z);
  return as_bf16x8(o);
}

// A scale's 16 bits as a float.
__device__ __forceinline__ float scale_f32(uint32_t bits, bool fp16) {
  return fp16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : __uint_as_float(bits << 16);
}

// 16 * NR weight rows (PAIR: 8 * NR of either matrix) by 16 * MQ rows of x per workgroup, whose 4
// wavefronts split K (interleaved chunks of 128; the sums meet in LDS in a fixed order).
template <int MQ, int NR, int GROUP, bool PAIR>
__global__ __launch_bounds__(256) void gemm_stream_w4(W4Args a) {
  constexpr int S = 128 / GROUP, F = GROUP / 32;  // groups per chunk, MFMAs per group
  constexpr int U = MQ * NR <= 2 ? 2 : 1;         // chunks per batch
  constexpr int PC = PAIR ? 2 : 1;                // accumulators per output
  constexpr int P = MQ * NR / PC;                 // outputs (16 x 16) per wavefront
  __shared__ float red[P * 3 * PC * 4 * 64];
  const int lane = threadIdx.x & 63, kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = a.K, nkb = K / 128, nblk = a.N / 16;
  const int m0 = (blockIdx.x % a.mtiles) * (16 * MQ), rows = min(16 * MQ, a.M - m0);
  const int b0 = (blockIdx.x / a.mtiles) * (NR / PC);  // first 16-row block
  uint32_t blk[NR], xoff[MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)  // (a block past N re-reads the last one; never stored)
    blk[j] = (uint32_t)min(b0 + j / PC, nblk - 1);
#pragma unroll
  for (int q = 0; q < MQ; ++q)  // (a row past the last re-reads it; never stored)
    xoff[q] = ((uint32_t)(m0 + min(q * 16 + r16, rows - 1)) * (uint32_t)K + kg * 8) * 2;
  f32x4 tot[NR][MQ];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int q = 0; q < MQ; ++q) tot[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Batch {
    uint4 w[U][NR], x[U][MQ][4];
    uint2 s[U][NR][S];
    uint32_t z[U][NR][S];
  };
  const int nc = (nkb - kw + 3) / 4;  // this wavefront's chunks: kw, kw + 4, ...
  auto load = [&](Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kb = (uint32_t)min(kw + 4 * (i + u), nkb - 1);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const W4Mat& m = a.m[PAIR ? j & 1 : 0];
        const uint32_t unit = blk[j] * (uint32_t)nkb + kb;
        bt.w[u][j] = gload16(static_cast<const char*>(m.codes) + (size_t)unit * 1024, lane * 16);
#pragma unroll
        for (int g = 0; g < S; ++g) {
          bt.s[u][j][g] = gload8(m.scales, ((unit * S + g) * 16 + kg * 4) * 2);
          bt.z[u][j][g] = m.zeros ? gload_u8(m.zeros, (unit * S + g) * 16 + r16) : 8u;
        }
      }
#pragma unroll
      for (int q = 0; q < MQ; ++q)
#pragma unroll
        for (int f = 0; f < 4; ++f) bt.x[u][q][f] = gload16(a.x, xoff[q] + (kb * 128 + f * 32) * 2);
    }
  };
  auto compute = [&](const Batch& bt, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= nc) break;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const uint32_t c[4] = {bt.w[u][j].x, bt.w[u][j].y, bt.w[u][j].z, bt.w[u][j].w};
#pragma unroll
        for (int g = 0; g < S; ++g) {
          const float z = float(bt.z[u][j][g]);
          const uint2 sb = bt.s[u][j][g];
          const float sc[4] = {scale_f32(sb.x & 0xFFFF, a.fp16), scale_f32(sb.x >> 16, a.fp16),
                               scale_f32(sb.y & 0xFFFF, a.fp16), scale_f32(sb.y >> 16, a.fp16)};
          f32x4 acc[MQ];
#pragma unroll
          for (int q = 0; q < MQ; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < F; ++f) {
            const bf16x8 wf = decode8(c[g * F + f], z);
#pragma unroll
            for (int q = 0; q < MQ; ++q) acc[q] = mfma16(wf, as_bf16x8(bt.x[u][q][g * F + f]), acc[q]);
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
  if (nc > 0) load(c0, 0);
  for (int i = 0; i < nc; i += 2 * U) {
    if (i + U < nc) load(c1, i + U);
    compute(c0, i);
    if (i + 2 * U < nc) load(c0, i + 2 * U);
    if (i + U < nc) compute(c1, i + U);
  }
  // every wavefront parks its sums but those of the outputs it finishes itself: output p goes to wavefront
  // p % 4, slot order (p, wavefront)
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 4 == kw) continue;
    float* dst = red + (p * 3 + (kw < p % 4 ? kw : kw - 1)) * (PC * 256) + lane;
#pragma unroll
    for (int c = 0; c < PC; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[(c * 4 + r) * 64] = tot[p / MQ * PC + c][p % MQ][r];
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 4 != kw) continue;
    const float* src = red + p * 3 * (PC * 256) + lane;
    float v[PC][4];
#pragma unroll
    for (int c = 0; c < PC; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[c][r] = tot[p / MQ * PC + c][p % MQ][r];
#pragma unroll
        for (int w = 0; w < 3; ++w) v[c][r] += src[w * (PC * 256) + (c * 4 + r) * 64];
      }
    // lane holds weight rows 4 kg + r of row r16 of x
    const int r = p % MQ * 16 + r16, b = b0 + p / MQ;
    if (r >= rows || b >= nblk) continue;
    if (PAIR) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = swiglu(v[0][e], v[PC - 1][e]);
    }
    gstore8(a.y, ((size_t)(m0 + r) * a.N + b * 16 + 4 * kg) * 2,
            uint2{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3])});
  }
}

template <int GROUP, bool PAIR>
hipError_t launch_group(W4Args a, hipStream_t s) {
  constexpr int NR = 2;
  const int mq = a.M <= 16 ? 1 : 2;
  a.mtiles = (a.M + 16 * mq - 1) / (16 * mq);
  const int per = PAIR ? NR / 2 : NR;
  const unsigned grid = (unsigned)a.mtiles * ((a.N / 16 + per - 1) / per);
  auto* kernel = mq == 1 ? &gemm_stream_w4<1, NR, GROUP, PAIR> : &gemm_stream_w4<2, NR, GROUP, PAIR>;
  kernel<<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w4(const W4Args& a, int group, int num_cus, hipStream_t s) {
  (void)num_cus;
  const bool pair = a.m[1].codes != nullptr;
  if (group == 32) return pair ? launch_group<32, true>(a, s) : launch_group<32, false>(a, s);
  if (group == 64) return pair ? launch_group<64, true>(a, s) : launch_group<64, false>(a, s);
  return pair ? launch_group<128, true>(a, s) : launch_group<128, false>(a, s);
}

hipError_t launch_w4_tile(const W4Mat& src, int N, int K, int group, void* codes, void* scales, uint8_t* zeros,
                          hipStream_t s) {
  const int64_t nw = (int64_t)N * K / 8, ns = (int64_t)N * (K / group);
  w4_tile_kernel<<<(unsigned)((nw + 255) / 256), 256, 0, s>>>(static_cast<const uint32_t*>(src.codes),
                                                              static_cast<uint32_t*>(codes), nw, K / 128);
  const unsigned grid = (unsigned)((ns + 255) / 256);
  w4_scale_tile_kernel<uint16_t><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(src.scales),
                                                      static_cast<uint16_t*>(scales), ns, K / group);
  if (src.zeros) w4_scale_tile_kernel<uint8_t><<<grid, 256, 0, s>>>(src.zeros, zeros, ns, K / group);
  return hipGetLastError();
}

}  // namespace moe

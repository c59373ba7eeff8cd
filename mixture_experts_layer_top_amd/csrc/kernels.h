// Internal launch interface between the C ABI (api.cpp) and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Tile families of the expert GEMMs.
enum Family { kFamStream = 0, kFamMfma = 1, kNumFam = 2 };
enum Gemm { kGemmGateUp = 0, kGemmDown = 1 };

constexpr int kMaxTopK = 8;  // experts per token (the boundary rejects more)

constexpr int kStreamMaxRows = 64;  // rows per weight-streaming pass
// Automatic selection: an expert takes the weight-streaming family for a GEMM while its row
// count is at most the policy's threshold for that GEMM (select_policy.h), the LDS-tiled MFMA
// family above it.
// Few-tile rule (policies that use it): a GEMM whose MFMA tiles would fill fewer than
// kFewTileRounds5 / 5 rounds of CUs runs wholly on the streaming tiles when none of its MFMA
// experts holds more than kFewTileRows rows (one 16-row MFMA pass per weight load); a larger
// expert keeps the whole GEMM on MFMA.
constexpr int kFewTileRows = 16;
constexpr int kFewTileRounds5 = 8;
// int8 experts: MFMA tiles, unless a GEMM's would fill fewer than kInt8FewTileRounds5 / 5 rounds and no
// expert holds more rows than one streaming pass: then all stream (see kInt8Policy).
constexpr int kInt8FewTileRows = kStreamMaxRows;
constexpr int kInt8FewTileRounds5 = 1;
constexpr int kMfmaBM = 256;        // rows per full LDS-tiled MFMA tile
constexpr int kMfmaBNGateUp = 128;  // h columns per gate/up MFMA tile (128 gate + 128 up rows)
constexpr int kMfmaBNDown = 256;    // y columns per down MFMA tile
constexpr int kXcds = 8;            // MI355X: 8 XCDs, each with its own L2
// Weight-streaming tiles: the 4 wavefronts split K four ways when K is long (16 output columns
// per tile), otherwise two ways (32 output columns, 16 per pair of wavefronts).  Measured: one
// wavefront per 16 columns over the whole K, or a four-way split of a short K, streams slower.
constexpr int kStreamSplitK = 4096;
__host__ __device__ constexpr int stream_bn(int K) { return K >= kStreamSplitK ? 16 : 32; }
// Longest K whose one-row activations a streaming tile stages in LDS (16 KB).
constexpr int kStreamXlMaxK = 8192;
constexpr int kSegCap = 1040;       // segment slots per (gemm, family); >= 2 * (E + 1)
// fp8 experts of more than kFp8MfmaRows rows take the LDS-staged MFMA tiles in automatic mode (when
// the GEMM's MFMA tiles fill at least one round of CUs), the others the streaming tiles.
constexpr int kFp8MfmaRows = 128;
// The same for mxfp4 experts with mxfp8 activations (whose streaming passes hold 32 rows).
constexpr int kMxMfmaRows = 64;
// fp8 weight-streaming tiles: rows per pass (more rows take more passes, which re-read
// the weights from L2; with 32 the down kernel fits three wavefronts per SIMD, while the gate/up
// kernel, which holds two K blocks of gate and up weights in flight, needs 256 VGPRs and runs one
// wavefront per SIMD), h columns per gate/up tile (one whole 128-column requantisation block), y
// columns per down tile
constexpr int kStreamMaxRows8 = 32;
constexpr int kStream8BNGateUp = 128;
constexpr int kStream8BNDown = 64;

// One expert's share of one grouped GEMM: out[row0 + r][n] for r < rows, n < N, from activation
// rows (gathered through `tok` when it is not null) and the expert's [N][K] weights.
struct Seg {
  const void* a;        // activation base ([.][K], bf16 or e4m3)
  const int32_t* tok;   // row -> activation row (null: row0 + r)
  const float* as;      // fp8: activation scales [.][K/128]; int8: [.]
  const void* w0;       // gate (gate/up GEMM) or down weights, [N][K]
  const void* w1;       // up weights (gate/up GEMM), [N][K]
  const float* s0;      // fp8 block scales of w0, [N/128][K/128]; int8 channel scales [N]
  const float* s1;      // the same of w1
  const uint8_t* e0;    // mxfp4: E8M0 scales of w0, [N][K/32] (w0 then holds [N][K/2] bytes)
  const uint8_t* e1;    // mxfp4: E8M0 scales of w1
  const uint8_t* ae;    // mxfp8 activations: E8M0 scales [.][K/32] of the rows of `a`
  void* out;            // output base [.][N] (bf16; e4m3 for the fp8 and mxfp8 gate/up GEMMs, fp32
                        // for the int8 one)
  float* outs;          // fp8 gate/up: output scales [.][N/128]
  uint8_t* oute;        // mxfp8 gate/up: output E8M0 scales [.][N/32]
  int32_t row0, rows, N, K;
  int32_t tile_base, mtiles, ntiles, expert;
  int32_t tn;           // output columns per tile
};

// Index of the segment holding tile t: the last one whose first tile (base[], in LDS) is <= t.
__device__ __forceinline__ int find_seg_lds(const int* base, int nseg, int t) {
  int lo = 0, hi = nseg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Last-round split of an MFMA GEMM: when its tiles leave a last round of CUs partly idle, the
// tiles of that round are split two or four ways in K, and every piece writes its fp32 partial sums
// to a slot of split_part.  A separate epilogue kernel, launched after the MFMA kernel, adds each
// split tile's slots in piece order (so results do not depend on which piece finished first) and
// stores the tile.
constexpr int kSplitMaxPieces = 256;  // partial-sum slots (one round of CUs)
constexpr int kSplitSlotFloats = 256 * 256;  // one full tile's accumulators
constexpr int kSplitMaxRounds = 3;    // longest-first order and split: fewer whole rounds than this
constexpr int kSplitMaxS = 4;         // pieces per split tile: 2 or 4

// Where the selection kernel writes its results (all inside the caller's workspace).
struct SelectOut {
  Seg* segs;           // [2 gemms][kNumFam][E + 1]
  int32_t* meta;       // [2 gemms][kNumFam][kMetaStride] (layout below)
  float* split_part;   // [kSplitMaxPieces][kSplitSlotFloats] partial sums (bf16 only, else null:
                       // no split; the two GEMMs run one after the other and share it)
};

// Everything the selection kernel needs to describe the two GEMMs.
struct SelectArgs {
  const int32_t* counts;   // [E]
  const int32_t* offsets;  // [E + 1]
  int E, T, k, d, f, f_sh, has_shared, config, fp8;
  int w4;                  // mxfp4 expert weights (streaming tiles)
  int i8;                  // int8 weights and rows, one scale per row and per output channel
  const void* hq; const void* h_shq;  // int8: the quantised rows of h and h_sh (the down GEMM's)
  int mx8;                 // with mxfp8 activations (x and h quantised per 32; else bf16)
  const uint8_t* e_gate; const uint8_t* e_up; const uint8_t* e_down;  // their E8M0 scales
  const uint8_t* xe;       // mx8: E8M0 scales of the gate/up activations [.][d/32]
  uint8_t* he;             // mx8: E8M0 scales of h [T*k][f/32]
  int num_cus;              // compute units of the device (one MFMA-tile round)
  const void* x;           // gate/up activations (bf16 x, or e4m3 xq)
  const float* xs;         // fp8 activation scales
  const int32_t* tok;      // row -> token, for routed rows (null: rows are already permuted)
  const void* w_gate; const void* w_up; const void* w_down;
  const float* s_gate; const float* s_up; const float* s_down;
  const void* sh_gate; const void* sh_up; const void* sh_down;
  const float* s_sh_gate; const float* s_sh_up; const float* s_sh_down;
  void* h; float* hs;      // routed gate/up output [T*k][f] (+ fp8 scales [T*k][f/128])
  void* h_sh; float* hs_sh;  // shared gate/up output [T][f_sh]
  void* y; void* y_sh;     // down outputs [T*k][d], [T][d]
  float* out_eeff;         // optional: the live effective expert count (bf16 selection)
  int32_t* out_policy;     // optional: the policy the selection applied (-1: a family was forced)
};

// ints per (gemm, family): nseg, ntiles, then kXcds queue counters (the stream family uses the
// first), zeroed by the selection kernel before each GEMM, then the number of class-0 tiles (which
// come first in tile order; see select_dev.h), then (MFMA family) the first queue position whose
// tile is split in K and the pieces per split tile (positions [0, base) are whole tiles, and each
// tile of [base, ntiles) takes S consecutive positions), then the ordering mode, then kXcds more
// queue counters (the class-1 queues of the two-class order), also zeroed before each GEMM.
constexpr int kMetaStride = 32;
constexpr int kMetaQueue = 2;
constexpr int kMetaClass0 = kMetaQueue + kXcds;
constexpr int kMetaSplitBase = kMetaClass0 + 1;
constexpr int kMetaSplitS = kMetaClass0 + 2;
constexpr int kMetaOrder = kMetaClass0 + 3;  // tile order of an MFMA list (select_dev.h)
constexpr int kMetaQueue1 = kMetaOrder + 1;
enum TileOrder { kOrderMix = 0, kOrderTwoClass = 1, kOrderLongestFirst = 2 };
constexpr int kLongK = 4096;  // K from which an MFMA list takes the two-class order
static_assert(kMetaQueue1 + kXcds <= kMetaStride, "meta layout");
// Two-class order: relative CU time of a class-1 (short) tile against a class-0 (full-height) one,
// in twentieths, which sets how many of an XCD's CUs start on each class.
constexpr int kTwoClassW0 = 20, kTwoClassW1 = 11;

hipError_t launch_route(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                        hipStream_t s);
int permute_nchunk(int n);
hipError_t launch_permute(const int32_t* ids, int T, int E, int k, int32_t* counts,
                          int32_t* offsets, int32_t* perm_src, int32_t* slot_dst, int32_t* tok,
                          int32_t* rank_ws, int32_t* hist_ws, hipStream_t s);
hipError_t launch_gather(const void* x, const float* xs, const int32_t* perm_src, int n, int k,
                         int row_bytes, int nb, void* xp, float* xps, hipStream_t s);
hipError_t launch_select(const SelectArgs& a, const SelectOut& o, hipStream_t s);
// Decode front end (route + permute + select in one workgroup) when T*k <= 2048.
bool front_small_fits(int T, int k);
hipError_t launch_front_small(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                              int32_t* counts, int32_t* offsets, int32_t* perm_src,
                              int32_t* slot_dst, int32_t* tok, const SelectArgs& sa,
                              const SelectOut& so, hipStream_t s);
// Launches the persistent kernel of each tile family of one GEMM (kGemmGateUp or kGemmDown) that
// may hold tiles (the other's queue is empty).  max_rows bounds the rows of any one expert, max_k
// the GEMM's K over all its segments.
// Row-major weight bytes [rows][row_bytes] -> tiled layout in chunks of cb bytes per row
// (rows % 16 == 0, row_bytes % cb == 0; cb = 64 for MXFP4, 128 for fp8).
hipError_t launch_weight_tile(const void* src, void* dst, int64_t rows, int64_t row_bytes, int cb,
                              hipStream_t s);
// w4: mxfp4 weights (streaming tiles only; mfma must be false).  maybe_split: the MFMA list may
// hold tiles split in K (the host's bound), so the split epilogue kernel follows the MFMA kernel.
hipError_t launch_gemms_bf16(const SelectOut& o, int gemm, int num_cus, int64_t max_rows,
                             int max_k, bool stream, bool mfma, bool maybe_split, hipStream_t s,
                             bool w4);
// fp8: the streaming kernel and/or the LDS-staged MFMA kernel of one GEMM (each launched only when
// its list may hold tiles).
hipError_t launch_gemms_fp8(const SelectOut& o, int gemm, int num_cus, int64_t max_rows,
                            bool stream, bool mfma, hipStream_t s);
void launch_mfma_fp8(const Seg* segs, int32_t* meta, int gemm, int num_cus, hipStream_t s);
// MXFP4 weights with MXFP8 activations (streaming tiles on the scaled f8f6f4 MFMA); max_rows
// bounds any expert's rows, K is the GEMM's (d for gate/up, f for down).
hipError_t launch_gemms_mx(const SelectOut& o, int gemm, int num_cus, int64_t max_rows, int K,
                           bool stream, bool mfma, hipStream_t s);
void launch_mfma_mx(const Seg* segs, int32_t* meta, int gemm, int num_cus, hipStream_t s);
// x [T][d] bf16 -> MXFP8: xq [T][d] e4m3, xe [T][d/32] E8M0 (smallest scale with no saturation).
hipError_t launch_quant_act_mx(const void* x, int T, int d, uint8_t* xq, uint8_t* xe,
                               hipStream_t s);

// Single-token decode (T = 1, bf16 weights, no shared expert, d <= kStreamXlMaxK): one kernel routes
// the token in every workgroup (the k selected experts are then known without a dispatch step),
// runs the gate/up GEMM on streaming tiles, and from workgroup 0 writes the routing, the
// histogram, the permutation and the down GEMM's streaming segments, which the down kernel then
// takes as the selection kernel would have written them.
struct Decode1Args {
  const float* logits;  // [E]
  int E, k, d, f;
  const void* x;        // [d] bf16
  const void* w_gate; const void* w_up; const void* w_down;
  void* h;              // [k][f] bf16
  void* y;              // [k][d] bf16
  int32_t* ids; float* w;                 // [k]
  int32_t* counts; int32_t* offsets;      // [E], [E + 1]
  int32_t* perm_src; int32_t* slot_dst;   // [k]
  int32_t* tok;                           // [k]
  int32_t* sync;                          // fused launch: kFusedSyncInts counters (zero on entry)
  void* out;                              // fused launch: [d] bf16
};
constexpr int kFusedSyncInts = 9216;  // the fused single-token launch's counters (36 KB)
hipError_t launch_decode1_bf16(const Decode1Args& a, const SelectOut& o, int num_cus,
                               hipStream_t s);
// The whole single-token layer (routing, gate/up, down, combine) in one launch (MOE_CONFIG_FUSED;
// bf16, no shared expert, d and f <= kStreamXlMaxK).
hipError_t launch_decode1_fused(const Decode1Args& a, int num_cus, hipStream_t s);
// (w null: every weight 1)
hipError_t launch_combine(const void* y, const int32_t* slot_dst, const float* w, int T, int k,
                          int d, const void* shared_y, void* out, hipStream_t s);
hipError_t launch_quant_act(const void* x, int T, int d, uint8_t* xq, float* xs, hipStream_t s);

// int8 weights and rows: one grouped GEMM (each kernel launched only when its list may hold tiles),
// one dense product [M][K] x [N][K] -> bf16 [M][N] (tiled weights, N % 16 == 0, K % 128 == 0), and
// the rows' quantisation (bf16, or fp32 when f32; d % 8 == 0, d <= 32768).
hipError_t launch_gemms_i8(const SelectOut& o, int gemm, int num_cus, int64_t max_rows, bool stream,
                           bool mfma, hipStream_t s);
// The experts' products of few tokens, without a selection: gate/up writes fp32 h, down quantises its
// rows of h itself, every workgroup anew, which costs as much as its weights from some 16 rows.  So at most
// kSmallI8Tokens tokens whose codes fit kSmallI8Lds bytes of LDS, or twice as many when an expert holds at
// most 4 rows on average and d_ff <= kSmallI8WideK.  Measured against the lists (us): 64 experts, d 7168,
// d_ff 2048, k 8: 1 token 60 and 90, 16 365 and 407, 32 449 and 468; d 2048, d_ff 1024: 32 tokens 75
// and 125; 16 experts of 4096 x 4096, k 8: 1 token 73 and 85, 16 165 and 164, 24 198 and 164; 8 experts,
// d 4096, d_ff 7168, k 8: 1 token 122 and 139, 8 166 and 140.
constexpr int kSmallI8Tokens = 16;
constexpr int kSmallI8Rows = 2 * kSmallI8Tokens * kMaxTopK;
constexpr int kSmallI8Lds = 66 << 10;
constexpr int kSmallI8WideK = 2048;
constexpr int small_i8_lds(int rows, int K) { return (rows < 16 ? rows : 16) * (K + 16); }
struct SmallI8 {
  const int32_t* counts; const int32_t* offsets;
  const int32_t* tok;                   // row -> row of x (null: itself)
  const void* x; const float* xs;       // gate/up: int8 rows and scales
  const float* h;                       // down: fp32 rows
  const void* w0; const void* w1;       // gate and up, or down (w1 null)
  const float* s0; const float* s1;
  void* out;                            // fp32 h, or bf16 y
  int E, N, K, rows;
};
hipError_t launch_small_i8(const SmallI8& a, bool gate_up, int num_cus, hipStream_t s);
hipError_t launch_gemm_i8(const void* xq, const float* xs, int M, const void* wq, const float* ws,
                          int N, int K, void* y, int num_cus, hipStream_t s);
hipError_t launch_quant_i8(const void* x, bool f32, int T, int d, uint8_t* q, float* qs,
                           hipStream_t s);

// What a block's output passes before the residual is added (null pointers: no such step).
struct BlockIn {
  const void* post;  // weight of the norm behind the block, [d]
  const void* gate;  // [d], or [T][d] with gate_rows
  int gate_rows;
  float rs, bs;
};
// RMS norm (fmt: 0 bf16 only, 1 e4m3 per 128, 2 e4m3 with E8M0 per 32, 3 int8 rows) and its gradient
// (part: rmsnorm_grad_parts(T) rows of d partial sums, unused when dw is null).
// b: a block norm (x is the block's output, res the residual, which it needs), else null.
hipError_t launch_rmsnorm(const void* x, const void* res, const void* w, float eps, int T, int d,
                          int fmt, void* h_out, void* y, void* q, void* qs, hipStream_t s,
                          const BlockIn* b = nullptr);
constexpr int kNormGradBlocks = 512;
constexpr int kNormGradRows = 3;     // per workgroup, until there are that many
constexpr int kNormGradChain = 128;  // and no more than these: more workgroups then
int norm_grad_parts(int T, int rows);
int rmsnorm_grad_parts(int T);
hipError_t launch_rmsnorm_grad(const void* dy, const void* dh, const void* h, const void* w,
                               float eps, int T, int d, void* dx, float* dw, float* part,
                               hipStream_t s);

// Gradients of combine and route (permute's is launch_combine without weights).
hipError_t launch_combine_grad(const void* dout, const void* y, const int32_t* slot_dst,
                               const float* w, int T, int k, int d, void* dy, float* dw,
                               hipStream_t s);
hipError_t launch_route_grad(const int32_t* ids, const float* w, const float* dw, int T, int E,
                             int k, float* dl, hipStream_t s);

// Gradient of the block norm: in.gate_rows as in the forward call, dgate_rows [T][d] bf16 then (else dgate
// [d]); part: block_grad_parts(T) rows of 2 d partial sums, null when dpre, dpost and dgate are.
struct BlockGrad {
  const void* dy; const void* dh; const void* x; const void* h;
  const void* pre;
  BlockIn in;
  float eps;
  int T;
  void* dx; void* dres; void* dgate_rows;
  float* dpre; float* dpost; float* dgate;
  float* part;
  int once;  // (the launch's)
};
constexpr int kBlockGradRows = 2;  // as kNormGradRows
int block_grad_parts(int T);
hipError_t launch_block_grad(BlockGrad a, int d, hipStream_t s);

// Routing by scores.
enum ScoreFn { kScoreSoftmax = 0, kScoreSigmoid = 1 };
constexpr int kMaxGroups = 64;
struct Scoring {
  int score, groups, top, group_top, renorm;
  float scale;
};
hipError_t launch_route_scored(const float* logits, const float* bias, int T, int E, int k,
                               const Scoring& p, int32_t* ids, float* w, hipStream_t s);
hipError_t launch_route_scored_grad(const float* logits, const int32_t* ids, const float* w,
                                    const float* dw, int T, int E, int k, const Scoring& p, float* dl,
                                    hipStream_t s);

// 4-bit weights: x [M][K] bf16 by one matrix, or by the gate and up pair (m[1].codes not null), tiled.
// A kernel that takes zero points takes them of both matrices: one without them has the other's pointer, read but
// not looked at, and all_zero (its zero point, 8) in their place.
struct W4Mat {
  const void* codes; const void* scales; const uint8_t* zeros;
  uint32_t zero_mask, all_zero;  // (0xFF and 0, or 0 and 8)
  __device__ uint32_t zero(uint32_t z) const { return (z & zero_mask) | all_zero; }
};
struct W4Args {
  const void* x;
  W4Mat m[2];
  void* y;
  int M, N, K;
  int fp16;    // the scales' type (else bf16)
  int mtiles;  // (the launch's)
};
hipError_t launch_gemm_w4(const W4Args& a, int group, int num_cus, hipStream_t s);
hipError_t launch_w4_tile(const W4Mat& src, int N, int K, int group, void* codes, void* scales, uint8_t* zeros,
                          hipStream_t s);

}  // namespace moe

// The LDS-staged MFMA tile shared by the bf16 and int8 expert GEMMs: 256 weight rows by 32 to 256
// token rows, its memory pipeline and its K loop.  Everything in it moves 16-byte pieces of rows
// through LDS; the element type (EL) only names the MFMA, the accumulator and the bytes per element:
// a 128-byte K-step is 64 bf16 or 128 int8 values, and either 32x32 MFMA takes 16 bytes per lane.
#pragma once

#include "common.h"
#include "kernels.h"
#include "mfma_dev.h"

namespace moe {

struct ElemBf16 {
  using Frag = bf16x8;
  using Acc = f32x16;
  static constexpr int kBytes = 2;
  static constexpr bool kTiledW = false;  // row-major weights
  static constexpr bool kOddSteps = false;  // K % 128 == 0: an even number of 64-wide K-steps
  static __device__ __forceinline__ Frag frag(const uint4& v) { return as_bf16x8(v); }
  static __device__ __forceinline__ Acc mfma(const Frag& a, const Frag& b, const Acc& c) {
    return mfma32(a, b, c);
  }
};

constexpr int BM = kMfmaBM;
constexpr int BNW = 256;                  // weight rows per tile
constexpr int LROWS = BM + BNW;           // LDS rows per stage of a full tile

// ------------------------------------------------------------------------------------------------
// Memory pipeline: K-steps of 64 (128-byte LDS rows) through a ring of stages; each stage holds the
// tile's token rows, then its 256 weight rows.  Global data goes straight into LDS
// (global_load_lds_dwordx4, no staging registers), every instruction moving 8 whole 128-byte lines.
// Rows keep 8 chunks of 16 B XOR-swizzled by (row >> 1) & 7, so the 16 lanes a ds_read_b128 serves
// together (16 rows, one chunk index) cover all 64 banks.
//
// Full tiles: two stages of 64 KB.  Waits are explicit (vmcnt) around a plain barrier so prefetches
// stay in flight.  Step kt
// on stage S: substeps 0..2 run while substeps 1..3 are read; wait until this wavefront's reads are
// done and every load it issued has landed; barrier (stage S^1 complete, stage S free); half the
// loads for step kt+2 into stage S while substep 3 runs and substep 0 of stage S^1 is read, the
// other half during substep 1 of step kt+1.
//
// Short tiles: NS stages (three; four for 32-row tiles) at a run-time stage index, so that NS - 1
// steps of loads stay in flight while one stage is read.  Step kt reads stage kt % NS; before the
// barrier it waits until the loads of step kt+1 have landed (later ones may still fly), then loads
// step kt+NS into the stage it just finished.
// ------------------------------------------------------------------------------------------------
constexpr int BK64 = 64;
constexpr int ROWB64 = 128;
constexpr int STAGE64 = LROWS * ROWB64;            // 64 KB
constexpr int DMA64 = STAGE64 / (256 * 16);        // 16 loads per thread per stage
constexpr int kShortStages = 3;
constexpr int kRingBytes = kShortStages * (128 + BNW) * ROWB64;  // 144 KB (>= 2 full stages)
// LDS stages of a short tile of TB token blocks: as many as the ring holds (32-row tiles: four
// 36 KB stages, three K-steps of loads in flight; 64- and 128-row tiles: three).
template <int TB> constexpr int kStagesFor = kRingBytes / ((TB * 32 + BNW) * ROWB64) >= 4 ? 4 : 3;
static_assert(kStagesFor<1> * (32 + BNW) * ROWB64 <= kRingBytes, "32-row stages fit the ring");
// Tile height for a tile holding `rows` token rows (the shortest that fits).
__device__ __forceinline__ int tile_height(int rows) {
  return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : kMfmaBM;
}
static_assert(kRingBytes >= 2 * STAGE64, "ring holds two full-tile stages");
__shared__ __attribute__((aligned(1024))) uint8_t g_ring[kRingBytes];
template <int S> __device__ __forceinline__ uint8_t* stage64_ptr() { return g_ring + S * STAGE64; }

// Fragment reads: a wavefront's A (weight) and B (token) fragments sit in 32-row blocks starting at
// multiples of 32 rows, so a lane's swizzle (row >> 1) & 7 = (lane % 32 >> 1) & 7 is the same in
// every block.  Each read address is then a per-lane base for the k-substep (row 32*blk + lane%32,
// chunk 2*kk + lane/32) plus a block offset that is a compile-time constant, which the LDS read
// instruction carries as its immediate: 4 bases per operand instead of one register per fragment.
__device__ __forceinline__ int frag_lane_off(int kk) {
  const int lane = threadIdx.x & 63, l32 = lane & 31;
  return l32 * ROWB64 + (((kk * 2 + (lane >> 5)) ^ ((l32 >> 1) & 7)) << 4);
}
// The same for weights in the tiled layout, whose LDS bytes keep it: per 16-row block 2 KB ordered
// [half][lane group][row][16 bytes], chunk c of a row being half c & 1 of lane group c >> 1.  A read of
// chunks 2 kk (lanes 0..31) and 2 kk + 1 (lanes 32..63) of 32 rows is four runs of 256 bytes, free of
// bank conflicts without a swizzle.
__device__ __forceinline__ int frag_lane_off_tiled(int kk) {
  const int lane = threadIdx.x & 63;
  return ((lane >> 4) & 1) * 2048 + (lane >> 5) * 1024 + kk * 256 + (lane & 15) * 16;
}
// byte offset of weight block a of a full tile (gate/up: gate blocks 0, 1 then up blocks 2, 3)
template <bool GU>
__device__ __forceinline__ constexpr int full_a_blk(int a) {
  return GU ? ((a & 1) * 32 + (a >> 1) * 128) * ROWB64 : a * 32 * ROWB64;
}

template <bool GU, class EL>
struct MfmaTile {
  using Frag = typename EL::Frag;
  // Load slot j of wavefront wv fills LDS rows [32*j + 8*wv, +8) of a stage: slots [0, NTS) token
  // rows, then 8 slots of weight rows (gate/up: 4 of gate rows 0..127, 4 of up rows 0..127), with
  // NTS = tile height / 32.
  const char* abase;
  const char* wbase0;
  const char* wbase1;
  uint32_t off[DMA64];
  // Tiled weights: a slot is one contiguous kilobyte, half wvu & 1 of a 16-row block.  Slot i's block is
  // wblk0 + 2 i (gate/up: i mod 4, of the gate or the up rows), past N the last one: uniform, so one lane
  // offset serves every slot.  (With a lane's 16 bytes of every row in the swizzled order instead, each
  // load touched a quarter of 32 lines: the gate/up GEMM of an 8-expert prefill layer 1.12 ms against
  // 0.96.)
  int wblk0, wlast;
  uint32_t wbytes, wlane;
  int wvu;
  int bm;  // tile height: 256, 128, 64 or 32 token rows
  int arow0, brow0;  // LDS byte offsets of the wavefront's first weight and token rows
  typename EL::Acc acc[4][4];

  template <int NTS>
  __device__ __forceinline__ const char* slot_base(int j) const {
    return j < NTS ? abase : ((!GU || j < NTS + 4) ? wbase0 : wbase1);
  }

  // kt0: first K-step of the tile's K range (a piece of a split tile starts past 0).  H: the tile
  // height, or 0 for the shortest that holds the rows.
  template <int H = 0>
  __device__ __forceinline__ void setup(const Seg& sg, int m0, int rows, int n0, int kt0) {
    const int lane = tid_here() & 63;  // (lane constants stay in the claim, not held across tiles)
    wvu = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    bm = H ? H : tile_height(rows);
    const int nts = bm >> 5;
    const uint32_t rowbytes = (uint32_t)sg.K * EL::kBytes;
    abase = static_cast<const char*>(sg.a);
    wbase0 = static_cast<const char*>(sg.w0);
    wbase1 = static_cast<const char*>(GU ? sg.w1 : sg.w0);
    // Token rows of slots 0..7, fetched together whatever the tile height (slots at or past NTS
    // are weight slots and drop theirs).  Padded rows (r >= rows) all read the first row's first 16
    // bytes: one coalesced request per instruction instead of eight lines; their LDS rows are never
    // stored.
    int src[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 32 * j + 8 * wvu + (lane >> 3);
      src[j] = sg.row0 + m0 + (r < rows ? r : 0);
    }
    if (sg.tok) {
#pragma unroll
      for (int j = 0; j < 8; ++j) src[j] = gload_i32(sg.tok, src[j]);
    }
#pragma unroll
    for (int j = 0; j < DMA64; ++j) {
      const int r = 32 * j + 8 * wvu + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      // as a weight slot, LDS row r holds the tile's weight row r - bm (slots past the tile's last
      // weight slot are never issued)
      int wr = GU ? n0 + ((r - bm) & 127) : n0 + (r - bm);
      wr = wr < sg.N ? wr : sg.N - 1;
      const uint32_t woff = (uint32_t)wr * rowbytes + c * 16 + (uint32_t)kt0 * ROWB64;
      if (j < 8) {
        const int rr = 32 * j + 8 * wvu + (lane >> 3);
        const uint32_t toff =
            (uint32_t)src[j] * rowbytes + (rr < rows ? c * 16 + (uint32_t)kt0 * ROWB64 : 0);
        off[j] = j < nts ? toff : woff;
      } else {
        off[j] = woff;
      }
    }
    if (EL::kTiledW) {
      wblk0 = (n0 >> 4) + (wvu >> 1);
      wlast = (sg.N >> 4) - 1;
      wbytes = 16 * rowbytes;
      wlane = (wvu & 1) * 1024 + lane * 16 + (uint32_t)kt0 * (16 * ROWB64);
    }
    if (bm == BM) {
      const int wm = wvu & 1, wn = wvu >> 1;
      arow0 = (BM + (GU ? wn * 64 : wn * 128)) * ROWB64;
      brow0 = wm * 128 * ROWB64;
    } else {
      const int wn = wvu;
      arow0 = (bm + (GU ? wn * 32 : wn * 64)) * ROWB64;
      brow0 = 0;
    }
  }

  // A lane's offset in a weight block for k-substep kk.
  static __device__ __forceinline__ int wfrag_off(int kk) {
    return EL::kTiledW ? frag_lane_off_tiled(kk) : frag_lane_off(kk);
  }

  // Load slot j of a tile of NTS token slots at byte ko of every row, into dst.
  template <int NTS, bool NT>
  __device__ __forceinline__ void load_slot(int j, uint32_t ko, uint8_t* dst) {
    if (EL::kTiledW && j >= NTS) {
      const int i = GU ? (j - NTS) & 3 : j - NTS;
      const uint32_t blk = (uint32_t)min(wblk0 + 2 * i, wlast);
      // (16 * ko: a K-step is a 2 KB unit of every 16-row block)
      dma16<NT>(slot_base<NTS>(j) + (size_t)(blk * wbytes) + 16 * ko, wlane, (lds_void*)dst);
    } else {
      dma16<NT>(slot_base<NTS>(j) + ko, off[j], (lds_void*)dst);
    }
  }

  // ---- full tiles ----
  template <int S>
  __device__ __forceinline__ void issue_one(int j, uint32_t ko) {
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* st = stage64_ptr<S>() + wv * 8 * ROWB64;
    load_slot<8, false>(j, ko, st + j * 32 * ROWB64);
  }

  template <int S>
  __device__ __forceinline__ void issue(int kt) {
#pragma unroll
    for (int j = 0; j < DMA64; ++j) issue_one<S>(j, (uint32_t)kt * ROWB64);
  }

  // fragment i of a full tile's k-substep (0..3: weight blocks, 4..7: token blocks)
  __device__ __forceinline__ Frag frag_full(const uint8_t* st, int va, int vb, int i) const {
    const uint8_t* p = i < 4 ? st + va + full_a_blk<GU>(i) : st + vb + (i - 4) * 32 * ROWB64;
    return EL::frag(*reinterpret_cast<const uint4*>(p));
  }

  template <int S>
  __device__ __forceinline__ void read_frags(int kk, Frag (&f)[8]) const {
    const uint8_t* st = stage64_ptr<S>();
    const int va = arow0 + wfrag_off(kk), vb = brow0 + frag_lane_off(kk);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = frag_full(st, va, vb, i);
  }

  __device__ __forceinline__ void mfmas(const Frag (&f)[8]) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = EL::mfma(f[a], f[4 + b], acc[a][b]);
  }

  // 16 MFMAs with the 8 fragment reads issued behind the first 8
  template <int S>
  __device__ __forceinline__ void sub(int kk, const Frag (&cur)[8], Frag (&nxt)[8]) {
    __builtin_amdgcn_sched_barrier(0);
    read_frags<S>(kk, nxt);
    mfmas(cur);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The same with loads J0 .. J0 + N - 1 of the K-step at offset ko (into stage T), one per MFMA:
  // gate/up places them on the first N MFMAs, beside the fragment reads, down on the last N, the
  // faster placement for each (the scheduler cannot see the asm loads, so the interleave is fixed
  // by hand).
  template <int S, int T, int J0, int N>
  __device__ __forceinline__ void sub_dma(int kk, const Frag (&cur)[8], Frag (&nxt)[8], uint32_t ko) {
    const uint8_t* st = stage64_ptr<S>();
    const int va = arow0 + wfrag_off(kk), vb = brow0 + frag_lane_off(kk);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      constexpr int L0 = GU ? 0 : 16 - N;  // first MFMA with a load
      if (i >= L0 && i < L0 + N) issue_one<T>(J0 + i - L0, ko);
      if (i < 8) nxt[i] = frag_full(st, va, vb, i);
      acc[i >> 2][i & 3] = EL::mfma(cur[i >> 2], cur[4 + (i & 3)], acc[i >> 2][i & 3]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // The 16 loads of a K-step go out in two halves: kDma0 behind the MFMAs of the previous step's
  // substep 3 (right after its barrier), the rest behind substep 1 of the step before the one
  // that reads them.  Issued all at once after the barrier, the four wavefronts' 64 loads queued
  // behind each other and held up the MFMAs interleaved with them (Mixtral-shaped layer 2.68 ->
  // 2.58 ms); issuing any of them later than substep 1 left too little time for them to land.
  // (At a tile's first step the second half repeats loads of the prologue.)
  static constexpr int kDma0 = 8;

  template <int S>
  __device__ __forceinline__ void step(int kt, int nk, Frag (&f0)[8], Frag (&f1)[8]) {
    // the rest of step kt+1's loads (into stage S^1)
    const uint32_t k1 = (uint32_t)min(kt + 1, nk - 1) * ROWB64;
    sub_dma<S, S ^ 1, kDma0, DMA64 - kDma0>(1, f0, f1, k1);
    sub<S>(2, f1, f0);
    sub<S>(3, f0, f1);
    MOE_WAITCNT(0, 0);
    __builtin_amdgcn_s_barrier();
    // the first kDma0 loads for step kt+2, with substep 0 of stage S^1 read behind the first eight
    // MFMAs of substep 3
    const uint32_t ko = (uint32_t)min(kt + 2, nk - 1) * ROWB64;
    const uint8_t* rd = stage64_ptr<S ^ 1>();
    const int va = arow0 + wfrag_off(0), vb = brow0 + frag_lane_off(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i < kDma0) issue_one<S>(i, ko);
      acc[i >> 2][i & 3] = EL::mfma(f1[i >> 2], f1[4 + (i & 3)], acc[i >> 2][i & 3]);
      if (i < 8) f0[i] = frag_full(rd, va, vb, i);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void prologue_full(int nk) {
    issue<0>(0);
    issue<1>(EL::kOddSteps ? min(1, nk - 1) : 1);
  }

  // nk: K-steps of the tile's K range (even unless EL::kOddSteps)
  __device__ __forceinline__ void run_full(int nk) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[a][b][r] = 0;
    MOE_WAITCNT(DMA64, 15);  // stage 0 (the oldest loads) has landed
    __builtin_amdgcn_s_barrier();
    Frag f0[8], f1[8];
    read_frags<0>(0, f0);
    const int pairs = EL::kOddSteps ? nk & ~1 : nk;
    for (int kt = 0; kt < pairs; kt += 2) {
      step<0>(kt, nk, f0, f1);
      step<1>(kt + 1, nk, f0, f1);
    }
    if (EL::kOddSteps && (nk & 1)) step<0>(nk - 1, nk, f0, f1);
    MOE_WAITCNT(0, 0);
    __builtin_amdgcn_s_barrier();
  }

  // ---- short tiles (TB = tile height / 32 token blocks) ----
  template <int TB>
  __device__ __forceinline__ void issue_short_one(int stage, int j, uint32_t ko) {
    constexpr int kStage = (TB * 32 + BNW) * ROWB64;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* st = g_ring + stage * kStage + wv * 8 * ROWB64;
    // The gate/up weights of a short tile stream with the non-temporal policy: a light expert's
    // weight rows are read by this tile alone, and left in L2 they only push out the tiles that
    // full-height neighbours share (DeepSeek-V3-shaped decode at T = 64 and 256: gate/up -9%).
    // Not the down weights: there the mixed order keeps an expert's short last m-tile next to
    // its full-height siblings, which read the same weight rows (Kimi-K2-shaped down GEMM +7%).
    if (GU && j >= TB) load_slot<TB, true>(j, ko, st + j * 32 * ROWB64);
    else load_slot<TB, false>(j, ko, st + j * 32 * ROWB64);
  }

  template <int TB>
  __device__ __forceinline__ void issue_short(int stage, int kt) {
#pragma unroll
    for (int j = 0; j < TB + 8; ++j) issue_short_one<TB>(stage, j, (uint32_t)kt * ROWB64);
  }

  // fragment i of a short tile's k-substep (0, 1: weight blocks -- gate/up: 32 gate rows, then the
  // matching up rows 128 further; down: two consecutive blocks -- 2..: token blocks)
  template <int TB>
  __device__ __forceinline__ Frag frag_short(const uint8_t* st, int va, int vb, int i) const {
    const uint8_t* p = i < 2 ? st + va + i * (GU ? 128 : 32) * ROWB64 : st + vb + (i - 2) * 32 * ROWB64;
    return EL::frag(*reinterpret_cast<const uint4*>(p));
  }

  template <int TB>
  __device__ __forceinline__ void read_frags_short(const uint8_t* st, int kk, Frag (&f)[2 + TB]) const {
    const int va = arow0 + wfrag_off(kk), vb = brow0 + frag_lane_off(kk);
#pragma unroll
    for (int i = 0; i < 2 + TB; ++i) f[i] = frag_short<TB>(st, va, vb, i);
  }

  template <int TB>
  __device__ __forceinline__ void mfmas_short(const Frag (&f)[2 + TB]) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[a][b] = EL::mfma(f[a], f[2 + b], acc[a][b]);
  }

  template <int TB>
  __device__ __forceinline__ void sub_short(const uint8_t* st, int kk, const Frag (&cur)[2 + TB],
                                            Frag (&nxt)[2 + TB]) {
    __builtin_amdgcn_sched_barrier(0);
    read_frags_short<TB>(st, kk, nxt);
    mfmas_short<TB>(cur);
    constexpr int kPairs = 2 * TB < 2 + TB ? 2 * TB : 2 + TB;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (2 * TB > kPairs) __builtin_amdgcn_sched_group_barrier(0x008, 2 * TB - kPairs, 0);
    if constexpr (2 + TB > kPairs) __builtin_amdgcn_sched_group_barrier(0x100, 2 + TB - kPairs, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  template <int TB>
  __device__ __forceinline__ void prologue_short(int nk) {
#pragma unroll
    for (int s = 0; s < kStagesFor<TB>; ++s) issue_short<TB>(s, min(s, nk - 1));
  }

  template <int TB>
  __device__ __forceinline__ void run_short(int nk) {
    constexpr int kStage = (TB * 32 + BNW) * ROWB64;
    constexpr int D = TB + 8;  // loads per thread per stage
    constexpr int NS = kStagesFor<TB>;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[a][b][r] = 0;
    MOE_WAITCNT((NS - 1) * D, 15);  // stage 0 (the oldest loads) has landed
    __builtin_amdgcn_s_barrier();
    Frag f0[2 + TB], f1[2 + TB];
    read_frags_short<TB>(g_ring, 0, f0);
    int s = 0;
    for (int kt = 0; kt < nk; ++kt) {
      const uint8_t* st = g_ring + s * kStage;
      sub_short<TB>(st, 1, f0, f1);
      sub_short<TB>(st, 2, f1, f0);
      sub_short<TB>(st, 3, f0, f1);
      // this wavefront's reads of stage s are done and its loads for step kt+1 have landed
      MOE_WAITCNT((NS - 2) * D, 0);
      __builtin_amdgcn_s_barrier();
      // the loads for step kt+NS into stage s, interleaved with the MFMAs of substep 3 and the
      // reads of substep 0 of the next stage
      const uint32_t ko = (uint32_t)min(kt + NS, nk - 1) * ROWB64;
      const int sn = s == NS - 1 ? 0 : s + 1;
      const uint8_t* rd = g_ring + sn * kStage;
      const int va = arow0 + wfrag_off(0), vb = brow0 + frag_lane_off(0);
#pragma unroll
      for (int i = 0; i < D; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        issue_short_one<TB>(s, i, ko);
        if (i < 2 * TB) acc[i / TB][i % TB] = EL::mfma(f1[i / TB], f1[2 + i % TB], acc[i / TB][i % TB]);
        if (i < 2 + TB) f0[i] = frag_short<TB>(rd, va, vb, i);
      }
      __builtin_amdgcn_sched_barrier(0);
      s = sn;
    }
    MOE_WAITCNT(0, 0);
    __builtin_amdgcn_s_barrier();
  }

  __device__ __forceinline__ void prologue(int nk) {
    if (bm == BM) prologue_full(nk);
    else if (bm == 128) prologue_short<4>(nk);
    else if (bm == 64) prologue_short<2>(nk);
    else prologue_short<1>(nk);
  }
};

}  // namespace moe

// Plain MXFP4 GEMM on gfx950 scaled MFMA: the dense path next to the two-path
// GEMM of gemm.hip (one activation operand instead of backbone + residual):
//   Y[t][o] = sum_k deq(A)[t][k] deq(W)[o][k],
// dense or per expert segment, stored as fp32 or bf16, or, for a fused gate|up
// weight, turned into h = bf16(silu(gate) * up) and coded to MXFP4 in the
// epilogue so that neither Y nor h passes through HBM.
//
// V_MFMA_SCALE_F32_32X32X64_F8F6F4 takes the weight rows as its first operand
// and the activation rows as its second, so a lane's accumulators are 16
// output columns of ONE token: column 8 (r / 4) + 4 (lane / 32) + r % 4 of the
// 32-column tile, token lane % 32. Four neighbouring columns then leave in one
// wide LDS or global store, and the 32 entries of an MXFP4 block of h sit in
// two lanes (l and l + 32): its amax is one register maximum and one half-wave
// swap, and its codes need no LDS.
//
// Main loop: a ring of LDS stages of 128 K entries, filled by buffer loads
// that write straight into LDS. The buffer view of an operand is one stage
// (base moved by the scalar unit, rows past the end read as zero), so offsets
// stay below 2^31 for any K. The last, partial stage of a K that is no
// multiple of 128 is whole in memory (zero codes, zero scales).

#include "gemm_common.h"
#include "sharq_device.h"
#include "sharq_internal.h"
#include "silu.h"

namespace sharq {
namespace {

// Workgroup tile of NWM x NWN waves, each WM x WN MFMA tiles of 32 x 32
// (WM along the tokens), and the layout of one LDS stage: activation codes,
// weight codes, and a KB for each operand's scales. WGS workgroups share a CU
// (bounded by the LDS and by the registers).
template <int WM_, int WN_, int NWM_, int NWN_, int RING_, int WGS_>
struct MxTile {
  static constexpr int WM = WM_, WN = WN_, NWM = NWM_, NWN = NWN_;
  static constexpr int kWaves = NWM * NWN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * WM * NWM, BN = 32 * WN * NWN;
  static constexpr int kOffA = 0;
  static constexpr int kOffW = BM * kRowBytes;
  static constexpr int kOffSW = kOffW + BN * kRowBytes;
  static constexpr int kOffSA = kOffSW + 1024;
  static constexpr int kStage = kOffSA + 1024;
  static constexpr int kAChunks = BM / 16 / kWaves;
  static constexpr int kWChunks = BN / 16 / kWaves;
  static constexpr int kCodeLoads = kAChunks + kWChunks;  // of a wave in a stage
  static_assert(kAChunks * 16 * kWaves == BM && kWChunks * 16 * kWaves == BN, "whole 1 KB chunks per wave");
  static constexpr int kHalf = WM * WN;  // MFMAs of half an iteration, a slot each
  static constexpr int kRing = RING_;
  static constexpr int kWavesPerSimd = (WGS_ * kWaves + 3) / 4;
  static_assert(kRing >= 2 && WGS_ * kRing * kStage <= kLdsBytes, "ring");
};
// Large tiles load fewer operand bytes a MFMA; small ones are more, keep more
// stages in flight and finish a stage sooner, which is what few tiles need.
// (64 x 256 was between its neighbours everywhere; 32 x 128 and 32 x 64 gained
// up to 7% for a few rows.)
using Mx128x256 = MxTile<2, 4, 2, 2, 3, 2>;
using Mx128x128 = MxTile<2, 2, 2, 2, 4, 2>;
using Mx64x128 = MxTile<1, 2, 2, 2, 5, 2>;
using Mx64x64 = MxTile<1, 1, 2, 2, 6, 2>;
using Mx32x256 = MxTile<1, 4, 1, 2, 3, 2>;

struct MxOperands {
  const uint8_t* a_codes;   // [G][rows][64]
  const uint8_t* a_scales;  // [G][rows][4]
  const uint8_t* w_codes;   // [G][O][64] (grouped: already the expert's)
  const uint8_t* w_scales;  // [G][O][4]
  int64_t rows, O;
  int nsteps;
};

// A wave has one scale load in a stage (waves that share one load the same
// bytes to the same place, so that all waves count alike). Into LDS, a dword a
// lane holds the CU's load path for 32 cycles, 16 bytes a lane for 16, so that
// is the form wherever rows lie side by side: even waves load the weight's 256
// dwords, odd waves the activation's. (16 bytes partly outside the view read
// zeros per dword.) Gathered activation rows take a dword a lane: the first
// waves load a 64-row run each, the others the weight's dwords.
template <class C>
constexpr int kLoads = C::kCodeLoads + 1;

template <class C>
struct MxFrags {
  v8i a[C::WM], w[C::WN];
};
template <class C>
struct MxScales {
  uint32_t a[C::WM], w[C::WN];
};

// LDS reads in the order of their use: for sub-step 0 the stage's scale dwords
// (two rows to an item), then the fragments; for sub-step 1 the fragments. The
// scale dword of a row holds the bytes of the stage's 4 blocks; shifted right
// by 8 (lane / 32), byte 0 (sub-step 0) and byte 2 (sub-step 1) are the blocks
// of the lane's K half.
template <class C, int SUB>
constexpr int kScaleItems = SUB == 0 ? (C::WM + 1) / 2 + (C::WN + 1) / 2 : 0;
template <class C, int SUB>
constexpr int kReadItems = kScaleItems<C, SUB> + C::WM + C::WN;

// LDS reads of a slot: as many as finish the half's reads in the first 5/8 of
// its slots, so that the other MFMAs cover the latency of the last ones.
template <class C>
constexpr int kReadSlots = C::kHalf * 5 / 8 < 1 ? 1 : C::kHalf * 5 / 8;
template <class C>
constexpr int kReadsPerSlot = (kReadItems<C, 0> + kReadSlots<C> - 1) / kReadSlots<C>;

template <class C, int SUB, int R>
__device__ __forceinline__ void mx_read(const uint8_t* st, MxFrags<C>& f, MxScales<C>& c, int wm, int wn, int lr,
                                        int lh) {
  constexpr int kSA = (C::WM + 1) / 2, kS = kScaleItems<C, SUB>;
  if constexpr (R < kS && R < kSA) {
    const uint8_t* p = st + C::kOffSA + 4 * (32 * C::WM * wm + 64 * R + lr);
    c.a[2 * R] = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (2 * R + 1 < C::WM) c.a[2 * R + 1] = *reinterpret_cast<const uint32_t*>(p + 128);
  } else if constexpr (R < kS) {
    constexpr int j = 2 * (R - kSA);
    const uint8_t* p = st + C::kOffSW + 4 * (32 * C::WN * wn + 32 * j + lr);
    c.w[j] = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (j + 1 < C::WN) c.w[j + 1] = *reinterpret_cast<const uint32_t*>(p + 128);
  } else if constexpr (R < kS + C::WM) {
    constexpr int i = R - kS;
    f.a[i] = frag(st + C::kOffA + swz(32 * C::WM * wm + 32 * i + lr, 2 * SUB + lh));
  } else if constexpr (R < kS + C::WM + C::WN) {
    constexpr int j = R - kS - C::WM;
    f.w[j] = frag(st + C::kOffW + swz(32 * C::WN * wn + 32 * j + lr, 2 * SUB + lh));
  }
}

template <class C, int SUB, int R, int END>
__device__ __forceinline__ void mx_read_range(const uint8_t* st, MxFrags<C>& f, MxScales<C>& c, int wm, int wn, int lr,
                                              int lh) {
  if constexpr (R < END && R < kReadItems<C, SUB>) {
    mx_read<C, SUB, R>(st, f, c, wm, wn, lr, lh);
    mx_read_range<C, SUB, R + 1, END>(st, f, c, wm, wn, lr, lh);
  }
}

// The shift of the scale dwords, kept where it stands (as an ordinary shift the
// compiler moves it behind the loop's edge, where it waits for every LDS read).
template <class C>
__device__ __forceinline__ void mx_shift_scales(MxScales<C>& c, uint32_t bits) {
#pragma unroll
  for (int i = 0; i < C::WM; ++i) asm volatile("v_lshrrev_b32 %0, %1, %0" : "+v"(c.a[i]) : "v"(bits));
#pragma unroll
  for (int j = 0; j < C::WN; ++j) asm volatile("v_lshrrev_b32 %0, %1, %0" : "+v"(c.w[j]) : "v"(bits));
}

// MFMA number M of a sub-step. (Skipping the row blocks of a partial expert
// tile that hold no valid row puts a branch at every MFMA: the grouped gate|up
// of the Qwen3-30B-A3B layer 92.8 us with it, 89.4 without.)
template <class C, int SUB, int M>
__device__ __forceinline__ void mx_mfma(const MxFrags<C>& f, const MxScales<C>& c, v16f (&acc)[C::WM][C::WN]) {
  constexpr int i = M / C::WN, j = M % C::WN;
  acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.w[j], f.a[i], acc[i][j], 4, 4, 2 * SUB,
                                                              (int)c.w[j], 2 * SUB, (int)c.a[i]);
}

// Buffer loads into LDS as in gemm_common.h, the LDS address a sum formed in
// M0 itself: base + the bytes that the template names.
template <int BYTES>
__device__ __forceinline__ void load_lds16(i32x4 rsrc, uint32_t voff, uint32_t base) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(base), "n"(BYTES) : "memory", "m0", "scc");
}
__device__ __forceinline__ void load_lds4(i32x4 rsrc, uint32_t voff, uint32_t base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(base) : "memory", "m0");
}

// One operand array: the buffer view of the stage to load next.
struct MxView {
  i32x4 r;
  uint32_t stage_bytes;
  __device__ __forceinline__ void start(const uint8_t* base, int64_t bytes, int stage) {
    stage_bytes = (uint32_t)bytes;
    r = make_rsrc(base + (int64_t)stage * bytes, bytes);
  }
  // On to the next stage; without one, to a view of nothing.
  __device__ __forceinline__ void advance(bool live) {
    const uint64_t at = ((uint64_t)(uint32_t)r[1] << 32 | (uint32_t)r[0]) + stage_bytes;
    r[0] = (int)(uint32_t)at;
    r[1] = (int)(uint32_t)(at >> 32);
    r[2] = live ? (int)stage_bytes : 0;
  }
};

// The loads of a wave; kDword: its scale load is a dword a lane. Every array's view moves on right behind its last load
// of a stage, so that the scalar work is spread between the MFMAs too.
template <class C, bool kDword>
struct MxLoader {
  MxView a, w, s;               // codes; the scales that the wave loads
  uint32_t a_off[C::kAChunks];  // byte offset of this lane's A code chunk inside a stage, kOOB if absent
  uint32_t w_off[C::kWChunks];
  uint32_t s_off;               // this lane's scale dwords
  uint32_t wave_base;           // 1024 * wave: the wave's chunk inside a stage
  uint32_t s_lds;               // where its scales go inside a stage
  uint32_t ring, at;            // LDS address of the ring; offset of the slot to fill
  int left;                     // stages not yet issued; batches past the last one read nothing

  template <int J>
  __device__ __forceinline__ void issue() {
    if constexpr (J < C::kAChunks) {
      load_lds16<C::kOffA + 1024 * C::kWaves * J>(a.r, a_off[J], ring + at + wave_base);
      if constexpr (J == C::kAChunks - 1) a.advance(--left > 0);
    } else if constexpr (J < C::kCodeLoads) {
      constexpr int j = J - C::kAChunks;
      load_lds16<C::kOffW + 1024 * C::kWaves * j>(w.r, w_off[j], ring + at + wave_base);
      if constexpr (J == C::kCodeLoads - 1) w.advance(left > 0);
    } else {
      if constexpr (kDword)
        load_lds4(s.r, s_off, ring + at + s_lds);
      else
        load_lds16<0>(s.r, s_off, ring + at + s_lds);
      s.advance(left > 0);
      at = at + C::kStage == C::kRing * C::kStage ? 0 : at + C::kStage;
    }
  }
  template <int J, int END>
  __device__ __forceinline__ void issue_range() {
    if constexpr (J < END) {
      issue<J>();
      issue_range<J + 1, END>();
    }
  }
  // Loads of slots [0, SLOT) of the 2 kHalf slots over which a stage's are spread.
  template <int SLOT>
  static constexpr int kBefore = (SLOT * kLoads<C> + 2 * C::kHalf - 1) / (2 * C::kHalf);
  template <int FROM, int TO>
  __device__ __forceinline__ void issue_slots() {
    issue_range<kBefore<FROM>, kBefore<TO>>();
  }
};

// An iteration is two halves of one MFMA a slot, the other work threaded
// between the MFMAs:
//   first half: the sub-step 0 MFMAs of stage s, the fragment reads of its
//     sub-step 1;
//   wait for stage s + 1 and barrier: stage s is in registers in every wave,
//     so its LDS slot is free;
//   second half: the sub-step 1 MFMAs, the scale and fragment reads of stage
//     s + 1.
// The loads of stage s + ring go into the freed slot, spread evenly over the
// second half and the first half of the next iteration: the waves of a barrier
// that issue theirs in a burst queue up at the CU's one load path (16 cycles a
// KB), and an MFMA behind a queued load waits with it.
template <class C, int M, bool kDword>
__device__ __forceinline__ void mx_first_half(const MxFrags<C>& f0, const MxScales<C>& c, v16f (&acc)[C::WM][C::WN],
                                              MxLoader<C, kDword>& ld, const uint8_t* cur,
                                              MxFrags<C>& f1, MxScales<C>& unused, int wm, int wn, int lr, int lh) {
  if constexpr (M < C::kHalf) {
    mx_mfma<C, 0, M>(f0, c, acc);
    mx_read_range<C, 1, M * kReadsPerSlot<C>, (M + 1) * kReadsPerSlot<C>>(cur, f1, unused, wm, wn, lr, lh);
    ld.template issue_slots<C::kHalf + M, C::kHalf + M + 1>();
    __builtin_amdgcn_sched_barrier(0);
    mx_first_half<C, M + 1, kDword>(f0, c, acc, ld, cur, f1, unused, wm, wn, lr, lh);
  }
}

template <class C, int M, bool kDword>
__device__ __forceinline__ void mx_second_half(const MxFrags<C>& f1, const MxScales<C>& c, v16f (&acc)[C::WM][C::WN],
                                               MxLoader<C, kDword>& ld, const uint8_t* next,
                                               MxFrags<C>& f0, MxScales<C>& cn, int wm, int wn, int lr, int lh) {
  if constexpr (M < C::kHalf) {
    mx_mfma<C, 1, M>(f1, c, acc);
    mx_read_range<C, 0, M * kReadsPerSlot<C>, (M + 1) * kReadsPerSlot<C>>(next, f0, cn, wm, wn, lr, lh);
    if constexpr (M == C::kHalf - 1) mx_shift_scales<C>(cn, 8 * lh);
    ld.template issue_slots<M, M + 1>();
    __builtin_amdgcn_sched_barrier(0);
    mx_second_half<C, M + 1, kDword>(f1, c, acc, ld, next, f0, cn, wm, wn, lr, lh);
  }
}

template <class C, bool kDword>
__device__ __forceinline__ void mx_loop(const MxOperands& op, const TileRows& tr, const TileCols& tc,
                                        uint8_t* ring, v16f (&acc)[C::WM][C::WN], int s_begin, int s_end, int wave,
                                        bool act_scales) {
  const int lane = threadIdx.x & 63;
  const int wm = wave % C::NWM, wn = wave / C::NWM;
  const int lr = lane & 31, lh = lane >> 5;
  MxLoader<C, kDword> ld;
  ld.left = s_end - s_begin;
  ld.a.start(op.a_codes, op.rows * kRowBytes, s_begin);
  ld.w.start(op.w_codes, op.O * kRowBytes, s_begin);
  ld.s.start(act_scales ? op.a_scales : op.w_scales, (act_scales ? op.rows : op.O) * 4, s_begin);
  ld.wave_base = 1024 * wave;
  ld.s_lds = kDword ? C::kOffSA + 256 * wave : act_scales ? C::kOffSA : C::kOffSW;
  ld.ring = lds_offset(ring);
  ld.at = 0;
  // A lane fills a fixed LDS chunk; it reads the global chunk that belongs there after the swizzle.
#pragma unroll
  for (int j = 0; j < C::kAChunks; ++j) {
    const int row = 16 * (wave + C::kWaves * j) + (lane >> 2);
    const int64_t src = tr.src(row);
    ld.a_off[j] = src >= 0 ? (uint32_t)(src * kRowBytes + ((lane & 3) ^ swz_part(row)) * 16) : kOOB;
  }
#pragma unroll
  for (int j = 0; j < C::kWChunks; ++j) {
    const int row = 16 * (wave + C::kWaves * j) + (lane >> 2);
    const int64_t o = tc.w_row(row);
    ld.w_off[j] = o < op.O ? (uint32_t)(o * kRowBytes + ((lane & 3) ^ swz_part(row)) * 16) : kOOB;
  }
  ld.s_off = kOOB;
  if (kDword) {
    const int64_t src = tr.src(64 * wave + lane);
    if (src >= 0) ld.s_off = (uint32_t)(src * 4);
  } else if (!act_scales) {
    const int64_t o = tc.w_row(4 * lane);  // four rows of one 64-row block
    if (4 * lane < C::BN && o < op.O) ld.s_off = (uint32_t)(o * 4);
  } else if (4 * lane < C::BM && tr.m0 + 4 * lane < op.rows) {
    ld.s_off = (uint32_t)((tr.m0 + 4 * lane) * 4);
  }

  // The first ring of stages; the last one's first-half loads follow in the loop.
  constexpr int kN = kLoads<C>;
#pragma unroll
  for (int b = 0; b + 1 < C::kRing; ++b) ld.template issue_range<0, kN>();
  ld.template issue_slots<0, C::kHalf>();
  wait_vmcnt<(C::kRing - 2) * kN + MxLoader<C, kDword>::template kBefore<C::kHalf>>();  // the first batch landed
  ring_barrier();
  MxFrags<C> f0, f1;
  MxScales<C> c, cn;
  mx_read_range<C, 0, 0, kReadItems<C, 0>>(ring, f0, c, wm, wn, lr, lh);
  mx_shift_scales<C>(c, 8 * lh);
  const uint8_t* cur = ring;
#pragma unroll 1
  for (int s = s_begin; s < s_end; ++s) {
    const uint8_t* next = cur == ring + (C::kRing - 1) * C::kStage ? ring : cur + C::kStage;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    mx_first_half<C, 0, kDword>(f0, c, acc, ld, cur, f1, cn, wm, wn, lr, lh);
    __builtin_amdgcn_s_setprio(0);
    wait_vmcnt<(C::kRing - 2) * kN>();  // the next stage landed; later batches may be in flight
    ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    mx_second_half<C, 0, kDword>(f1, c, acc, ld, next, f0, cn, wm, wn, lr, lh);
    __builtin_amdgcn_s_setprio(0);
    c = cn;
    cur = next;
  }
  wait_vmcnt<0>();  // the trailing batches, before the LDS is used again
}

// acc += the product over stages [s_begin, s_end) (s_begin < s_end). The two
// kinds of scale load are loops of their own, between which the waves of a
// gathered tile part: a choice inside the loop would put branches between its
// MFMAs, and with both loads in every wave two workgroups hold the CU's load
// path for 1152 cycles a stage, longer than their MFMAs run (1024); this way
// it is 960. Grouped gate|up, 4096 tokens x 8 of 128 experts, 2048 -> 2 x 768,
// means of four runs in turn: 99 us with both, 94 so.
template <class C, bool kGather>
__device__ __forceinline__ void mx_mainloop(const MxOperands& op, const TileRows& tr, const TileCols& tc,
                                            uint8_t* ring, v16f (&acc)[C::WM][C::WN], int s_begin, int s_end) {
  constexpr int kARuns = (C::BM + 63) / 64;
  static_assert(kARuns < C::kWaves, "a wave is left for the weight's scales");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool gathered = kGather && tr.gather != nullptr;
  if (kGather && gathered && wave < kARuns)
    mx_loop<C, true>(op, tr, tc, ring, acc, s_begin, s_end, wave, true);
  else
    mx_loop<C, false>(op, tr, tc, ring, acc, s_begin, s_end, wave, !gathered && (wave & 1));
}

template <class C>
__device__ __forceinline__ void mx_zero(v16f (&acc)[C::WM][C::WN]) {
#pragma unroll
  for (int i = 0; i < C::WM; ++i)
#pragma unroll
    for (int j = 0; j < C::WN; ++j) acc[i][j] = v16f{};
}

// ---------------------------------------------------------------------------
// Epilogues
// ---------------------------------------------------------------------------

// Store the tile to y (fp32, or bf16 rounded to nearest even). A wave turns
// slabs of 32 tokens x 256 bytes (64 fp32 or 128 bf16 columns; fewer where the
// wave has fewer) through LDS of its own, so that every global store is 16 bytes
// a lane in row runs of that length.
// wide: y rows are 16-byte aligned (leading dimension included).
template <class C, class Out>
__device__ __forceinline__ void mx_store(const v16f (&acc)[C::WM][C::WN], uint8_t* lds, Out* __restrict__ y,
                                         int64_t ldy, const TileRows& tr, int64_t n0, int64_t O, bool wide) {
  constexpr bool kBf16 = sizeof(Out) == 2;
  constexpr int kMost = kBf16 ? 4 : 2;
  constexpr int kJ = C::WN < kMost ? C::WN : kMost;  // MFMA column tiles of a slab
  constexpr int kPer = 16 / sizeof(Out);             // columns of a 16-byte piece
  constexpr int kPieces = 32 * kJ / kPer;            // of a row
  constexpr int kSlabStride = 16 * kPieces + 16;     // 16 more, so that rows start on distinct banks
  static_assert(C::kRing * C::kStage >= C::kWaves * 32 * kSlabStride, "the slabs fit in the ring's LDS");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % C::NWM, wn = wave / C::NWM;
  const int lr = lane & 31, lh = lane >> 5;
  ring_barrier();  // every wave is done with the ring
  uint8_t* slab = lds + wave * 32 * kSlabStride;
#pragma unroll
  for (int i = 0; i < C::WM; ++i) {
    const int row0 = 32 * C::WM * wm + 32 * i;
    if (row0 >= tr.rows_valid) break;  // wave-uniform
#pragma unroll
    for (int j0 = 0; j0 < C::WN; j0 += kJ) {
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const v16f& a = acc[i][j0 + j];
          const int col = 32 * j + 8 * g + 4 * lh;
          if constexpr (kBf16) {
            *reinterpret_cast<uint2*>(slab + lr * kSlabStride + 2 * col) =
                make_uint2(bf16x2_rne(a[4 * g], a[4 * g + 1]), bf16x2_rne(a[4 * g + 2], a[4 * g + 3]));
          } else {
            *reinterpret_cast<float4*>(slab + lr * kSlabStride + 4 * col) =
                make_float4(a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]);
          }
        }
#pragma unroll
      for (int q = 0; q < kPieces / 2; ++q) {
        const int r = 64 / kPieces * q + lane / kPieces, piece = lane % kPieces;
        const uint4 v = *reinterpret_cast<const uint4*>(slab + r * kSlabStride + 16 * piece);
        const int64_t o = n0 + 32 * (C::WN * wn + j0) + kPer * piece;
        if (row0 + r < tr.rows_valid) {
          Out* dst = y + (tr.m0 + row0 + r) * ldy + o;
          if (wide && o + kPer <= O) {
            *reinterpret_cast<uint4*>(dst) = v;
          } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              if (o + e < O) {
                if constexpr (kBf16)
                  dst[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
                else
                  dst[e] = __uint_as_float(w[e]);
              }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

struct MxH {
  uint8_t* codes;   // [ceil(I / 128)][T][64]
  uint8_t* scales;  // [ceil(I / 128)][T][4]
  int64_t T, I;
};

// 16 values of a block in the accumulator order of one lane (four runs of four
// neighbouring columns) -> 8 bytes of E2M1 codes, a run of four per 16 bits.
__device__ __forceinline__ void quantize16(const float (&v)[16], float scale, uint32_t (&w)[2]) {
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * d + 0], v[8 * d + 1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * d + 2], v[8 * d + 3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * d + 4], v[8 * d + 5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * d + 6], v[8 * d + 7], scale, 3);
    w[d] = r;
  }
}

typedef unsigned int v2u __attribute__((ext_vector_type(2)));

// The pair (x of lane l % 32, y of lane l % 32 + 32) of two registers: lanes
// below 32 get x's two halves, lanes from 32 on y's.
__device__ __forceinline__ v2u half_swap(uint32_t x, uint32_t y) {
  return __builtin_amdgcn_permlane32_swap(x, y, false, false);
}

// h columns of a gate|up tile, and the row blocks that alternate in its weight rows.
template <class C>
constexpr int kHCols = C::BN / 2;
template <class C>
constexpr int kHShift = C::WN == 4 ? 6 : 5;

// h = bf16(silu(gate) * up) of the tile, coded to MXFP4: the first half of a
// wave's MFMA column tiles is gate, the second up, of one block of its tokens
// each. Lane l holds half of a block of token l % 32. Two blocks are coded
// together (two of a token, or with one a token those of two row tiles): after
// the half-wave swap lane l holds all of block l / 32 and writes its 16 bytes.
template <class C>
__device__ __forceinline__ void mx_silu_store(const v16f (&acc)[C::WM][C::WN], const TileRows& tr, int64_t h0,
                                              const MxH& out) {
  static_assert(C::WN == 4 || C::WN == 2, "gate, gate, up, up or gate, up");
  constexpr int kJ = C::WN / 2;                        // blocks of a token in this wave
  constexpr int kRows = kJ == 2 || C::WM == 1 ? 1 : 2;  // row tiles coded together
  static_assert(C::WM % kRows == 0, "row tiles in pairs");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % C::NWM, wn = wave / C::NWM;
  const int lr = lane & 31, lh = lane >> 5;
  const int64_t block = (h0 >> 5) + kJ * wn + (kJ == 2 ? lh : 0);  // the block this lane writes
  const int64_t blocks = out.I >> 5, padded = (blocks + 3) & ~(int64_t)3;
  const bool writes = kJ * kRows == 2 || lh == 0;
#pragma unroll
  for (int i = 0; i < C::WM; i += kRows) {
    const int row = 32 * C::WM * wm + 32 * (kRows == 2 ? i + lh : i) + lr;
    uint32_t code[2][2], byte[2];
#pragma unroll
    for (int q = 0; q < kJ * kRows; ++q) {
      const v16f &gate = acc[kRows == 2 ? i + q : i][kRows == 2 ? 0 : q],
                 &up = acc[kRows == 2 ? i + q : i][kJ + (kRows == 2 ? 0 : q)];
      float h[16], m = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const uint32_t b = bf16x2_rne(silu_times(gate[r], up[r]), silu_times(gate[r + 1], up[r + 1]));
        h[r] = bf16_lo(b);
        h[r + 1] = bf16_hi(b);
        m = fmaxf(m, fmaxf(fabsf(h[r]), fabsf(h[r + 1])));
      }
      const v2u both = half_swap(__float_as_uint(m), __float_as_uint(m));
      byte[q] = e8m0_from_amax_bits(max(both[0], both[1]));  // non-negative floats order as their bits
      quantize16(h, scale_from_e8m0(byte[q]), code[q]);
    }
    if constexpr (kJ * kRows == 1) code[1][0] = code[0][0], code[1][1] = code[0][1], byte[1] = byte[0];
    const v2u lo = half_swap(code[0][0], code[1][0]);  // [0]: columns 0-3, 8-11; [1]: columns 4-7, 12-15
    const v2u hi = half_swap(code[0][1], code[1][1]);  // the same from column 16 on
    if (writes && row < tr.rows_valid && block < padded) {
      const int64_t t = tr.m0 + row;
      const bool real = block < blocks;
      const uint4 c = make_uint4((lo[0] & 0xFFFFu) | (lo[1] << 16), (lo[0] >> 16) | (lo[1] & 0xFFFF0000u),
                                 (hi[0] & 0xFFFFu) | (hi[1] << 16), (hi[0] >> 16) | (hi[1] & 0xFFFF0000u));
      *reinterpret_cast<uint4*>(out.codes + code_offset(t, (uint32_t)block, out.T)) =
          real ? c : make_uint4(0, 0, 0, 0);
      out.scales[scale_index(t, (uint32_t)block, out.T)] = (uint8_t)(real ? (lh ? byte[1] : byte[0]) : 0u);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---------------------------------------------------------------------------
// Kernels
// ---------------------------------------------------------------------------

#define SHARQ_MX_LDS(C) __shared__ __attribute__((aligned(16))) uint8_t lds[C::kRing * C::kStage];

__device__ __forceinline__ TileRows dense_rows(int64_t m0, int64_t T, int bm) {
  TileRows tr;
  tr.m0 = m0;
  tr.rows_valid = T - m0 < bm ? T - m0 : bm;
  tr.gather = nullptr;
  tr.src_rows = T;
  return tr;
}

// Many tokens, as 2048 x 14336 x 4096 (65 us with fp32 out, 61 with bf16, 3.7-4.0
// PFLOP/s): 256 tiles, so a CU has one workgroup of four waves, whose stage takes
// 812 cycles where its MFMAs take 512, and the stores at the end overlap nothing
// (11.9k of 103.6k cycles, 4.8k of 96.7k with bf16). The matrix cores are busy for
// 54-58% of the cycles, at the 1.5-1.7 GHz that the chip holds then; a loop of MFMAs
// on registers reaches 6.2-6.6 PFLOP/s at 1.55 GHz. Few tokens: by the weight's
// bytes (57344 x 8192: 42 us, 6 TB/s), or by a workgroup's own chain of stages
// (333 x 4128 x 1000: 9.4 us for 33 stages, 4 of them launch, first loads and
// stores).
template <class C, class Out>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void mx_linear_kernel(MxOperands op, Out* __restrict__ y,
                                                                               int64_t ldy, bool wide, int tiles_m,
                                                                               int tiles_total) {
  SHARQ_MX_LDS(C)
  const TileIndex ti = tile_index(blockIdx.x, tiles_m, tiles_total);
  const TileRows tr = dense_rows((int64_t)ti.tm * C::BM, op.rows, C::BM);
  const int64_t n0 = (int64_t)ti.tn * C::BN;
  v16f acc[C::WM][C::WN];
  mx_zero<C>(acc);
  mx_mainloop<C, false>(op, tr, TileCols{n0, 0}, lds, acc, 0, op.nsteps);
  mx_store<C, Out>(acc, lds, y, ldy, tr, n0, op.O, wide);
}

// 2048 x 4096 -> 2 x 14336 118 us (4.1 PFLOP/s): two workgroups a CU, whose stages
// take 1058 cycles together where their MFMAs take 1024; with the SiLU and coding
// (8.1k of a workgroup's 42.6k cycles) and 1792 tiles on 512 places (3.5 rounds) the
// matrix cores are busy for 66% of the cycles, at 1.47 GHz. 8 x 8192 -> 2 x 28672 41
// us (6 TB/s of weights).
template <class C>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void mx_linear_silu_kernel(MxOperands op, MxH out,
                                                                                    int tiles_m, int tiles_total) {
  SHARQ_MX_LDS(C)
  const TileIndex ti = tile_index(blockIdx.x, tiles_m, tiles_total);
  const TileRows tr = dense_rows((int64_t)ti.tm * C::BM, op.rows, C::BM);
  const int64_t h0 = (int64_t)ti.tn * kHCols<C>;
  v16f acc[C::WM][C::WN];
  mx_zero<C>(acc);
  mx_mainloop<C, false>(op, tr, TileCols{h0, out.I, kHShift<C>}, lds, acc, 0, op.nsteps);
  mx_silu_store<C>(acc, tr, h0, out);
}

// Split-K: item q of the S * tiles work items computes split q / tiles (stages
// [split * nsteps / S, (split + 1) * nsteps / S)) of tile q % tiles and stores
// its fp32 partial in partials[split] ([S][T][O]). The reduce kernels add the
// partials in split order, so results do not depend on timing; the kernel
// boundary makes them visible to every XCD. 1 x 28672 x 8192: 22.5 us (5.5 TB/s)
// and 4 us for the sum.
template <class C>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void mx_split_kernel(MxOperands op, int tiles_m,
                                                                              int tiles_total, int S, bool wide,
                                                                              float* __restrict__ partials) {
  SHARQ_MX_LDS(C)
  const int item = xcd_item(blockIdx.x, tiles_total * S);
  const int split = item / tiles_total;
  const TileIndex ti = tile_order(item - split * tiles_total, tiles_m, tiles_total);
  const TileRows tr = dense_rows((int64_t)ti.tm * C::BM, op.rows, C::BM);
  const int64_t n0 = (int64_t)ti.tn * C::BN;
  v16f acc[C::WM][C::WN];
  mx_zero<C>(acc);
  const int s0 = (int)((int64_t)split * op.nsteps / S), s1 = (int)((int64_t)(split + 1) * op.nsteps / S);
  mx_mainloop<C, false>(op, tr, TileCols{n0, 0}, lds, acc, s0, s1);
  mx_store<C, float>(acc, lds, partials + (int64_t)split * op.rows * op.O, op.O, tr, n0, op.O, wide);
}

constexpr int kMxMaxSplits = 16;

__device__ __forceinline__ void store_out(float* y, float v) { *y = v; }
__device__ __forceinline__ void store_out(uint16_t* y, float v) { *y = (uint16_t)bf16_rne_bits(v); }

template <class Out>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ partials, int S, int64_t T,
                                                        int64_t O, Out* __restrict__ y, int64_t ldy) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= T * O) return;
  const int64_t t = e / O, o = e - t * O;
  float part[kMxMaxSplits];
#pragma unroll
  for (int q = 0; q < kMxMaxSplits; ++q) part[q] = q < S ? partials[(int64_t)q * T * O + e] : 0.0f;
  float v = part[0];
#pragma unroll
  for (int q = 1; q < kMxMaxSplits; ++q)
    if (q < S) v += part[q];
  store_out(y + t * ldy + o, v);
}

// The reduce of a split gate|up product with the SiLU and the coding of h:
// half-wave lane l of a row's block owns column l, so a block's gate and up
// runs are 128 contiguous bytes a partial. Blocks of a partial last stage are
// written as zeros.
__global__ __launch_bounds__(256) void mx_reduce_silu_kernel(const float* __restrict__ partials, int S, MxH out) {
  const int64_t blocks = out.I >> 5, padded = (blocks + 3) & ~(int64_t)3;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int col = threadIdx.x & 31;
  const int64_t t = unit / padded, b = unit - t * padded;
  if (t >= out.T) return;  // whole half-waves
  float h = 0.0f;
  if (b < blocks) {
    const int64_t plane = out.T * 2 * out.I;
    const float* src = partials + t * 2 * out.I + 32 * b + col;
    float g[kMxMaxSplits], u[kMxMaxSplits];
#pragma unroll
    for (int q = 0; q < kMxMaxSplits; ++q) {
      g[q] = q < S ? src[q * plane] : 0.0f;
      u[q] = q < S ? src[q * plane + out.I] : 0.0f;
    }
    float gs = g[0], us = u[0];
#pragma unroll
    for (int q = 1; q < kMxMaxSplits; ++q)
      if (q < S) gs += g[q], us += u[q];
    h = __uint_as_float(bf16_rne_bits(silu_times(gs, us)) << 16);
  }
  float m = fmaxf(0.0f, fabsf(h));  // 0 for NaN
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 32));
  const uint32_t byte = b < blocks ? e8m0_from_amax_bits(__float_as_uint(m)) : 0u;
  const float other = __shfl_xor(h, 1, 32);
  uint32_t code = 0;
  code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, h, other, scale_from_e8m0(byte), 0);  // even columns
  if ((col & 1) == 0) out.codes[code_offset(t, (uint32_t)b, out.T) + (col >> 1)] = (uint8_t)code;
  if (col == 0) out.scales[scale_index(t, (uint32_t)b, out.T)] = (uint8_t)byte;
}

__device__ __forceinline__ void mx_select_expert(MxOperands& op, int e) {
  op.w_codes += (int64_t)e * op.O * kRowBytes * op.nsteps;
  op.w_scales += (int64_t)e * op.O * 4 * op.nsteps;
}

// Per expert. Bound by the weights' bytes at few tokens. At many a workgroup's ends
// weigh, for K is short: Qwen3-30B-A3B layer (128 experts, top 8, 2048 -> 2 x 768 ->
// 2048) with 4096 tokens, cycles of a workgroup (two a CU): gate|up 3.4k until the
// tile is found, 24.8k for 16 stages with the ring's first fill (1551 a stage), 5.5k
// for SiLU and coding; down 2.8k, 11.8k for 6 stages (1966 each), 4.8k for the
// stores of bf16 rows (134 MB in all, 28 us at the rate of a copy). The row tiles
// hold 1.26 times the pairs. The matrix cores are busy for 40% and 24% of the
// cycles. 4 tokens gate|up 13.5 us, down 7-8; 512 tokens 42 and 28; 4096 tokens
// 80-105 and 62-78 with weights from the last-level cache or from memory.
template <class C, class Out>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void mx_grouped_kernel(
    MxOperands op, const int32_t* __restrict__ a_rows, const int32_t* __restrict__ seg, int E, Out* __restrict__ y,
    int64_t P, bool wide, int tiles_n) {
  SHARQ_MX_LDS(C)
  // Without the XCD ranges: with 8 column tiles each XCD keeps a column slice of every weight (the same time).
  const GroupedTile g = grouped_tile<C, false>(seg, E, P, a_rows, op.rows, tiles_n);
  if (g.e < 0) return;  // uniform across the workgroup
  mx_select_expert(op, g.e);
  const int64_t n0 = (int64_t)g.col * C::BN;
  v16f acc[C::WM][C::WN];
  mx_zero<C>(acc);
  mx_mainloop<C, true>(op, g.tr, TileCols{n0, 0}, lds, acc, 0, op.nsteps);
  mx_store<C, Out>(acc, lds, y, op.O, g.tr, n0, op.O, wide);
}

template <class C>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void mx_grouped_silu_kernel(
    MxOperands op, const int32_t* __restrict__ a_rows, const int32_t* __restrict__ seg, int E, MxH out, int tiles_n) {
  SHARQ_MX_LDS(C)
  // With them: an expert's row tiles share its weight in one L2 (95 us, 117 without).
  const GroupedTile g = grouped_tile<C, true>(seg, E, out.T, a_rows, op.rows, tiles_n);
  if (g.e < 0) return;
  mx_select_expert(op, g.e);
  const int64_t h0 = (int64_t)g.col * kHCols<C>;
  v16f acc[C::WM][C::WN];
  mx_zero<C>(acc);
  mx_mainloop<C, true>(op, g.tr, TileCols{h0, out.I, kHShift<C>}, lds, acc, 0, op.nsteps);
  mx_silu_store<C>(acc, g.tr, h0, out);
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------

MxOperands mx_operands(const MxProduct& p) {
  return MxOperands{p.a_codes, p.a_scales, p.w_codes, p.w_scales, p.rows, p.O, (int)((p.K + 127) / 128)};
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Times of the K loop in microseconds a stage, for the choice of tiles alone:
// of a workgroup on a CU of its own, and of each of several.
struct MxTileCost {
  int64_t rows, cols;
  double alone, each;
};
constexpr int kMxTiles = 5;
constexpr MxTileCost kTiles[kMxTiles] = {
    {128, 256, 0.48, 0.47}, {128, 128, 0.22, 0.29}, {64, 128, 0.175, 0.205}, {64, 64, 0.135, 0.15}, {32, 256, 0.40, 0.30}};
constexpr int kMx64x64 = 3;  // too narrow for gate and up columns in one wave

// Calls f with the tile type of kTiles[tile].
template <class F>
void mx_with_tile(int tile, F f) {
  switch (tile) {
    case 0: f(Mx128x256{}); break;
    case 1: f(Mx128x128{}); break;
    case 2: f(Mx64x128{}); break;
    case kMx64x64: f(Mx64x64{}); break;
    default: f(Mx32x256{}); break;
  }
}

// The K loops of a launch: `share` workgroups on the busiest CU, and no less
// than the operands' bytes at the rate of memory.
double mx_loop_cost(int tile, double share, int64_t steps, double operand_bytes) {
  const MxTileCost& c = kTiles[tile];
  const double each = c.each * share;
  const double loop = (double)steps * (c.alone > each ? c.alone : each), stream = operand_bytes / 5.8e6;
  return loop > stream ? loop + 0.1 * stream : stream + 0.1 * loop;
}

double mx_operand_bytes(double rows, double K) { return rows * K * 17.0 / 32.0; }

struct MxPlan {
  int tile, S;
  int tiles_m, tiles_total;
};

// Tile and K split of a dense product: the cheapest of all tiles and S in [1,
// 16] (each split over at least 4 stages, the partials at most 256 MB) by the
// loops above and, for S > 1, a second launch and the partials' traffic. The
// constants are fitted to timed launches of all of them on 11 layer shapes from
// 2048 x 768 to 57344 x 8192 (O x K), T = 1 .. 1024, whose best they pick but
// for 1% on average and 13% at most. With 256 columns a tile alone the best was
// 22% slower on average: 4096 x 4096 at T = 128 15.9 us, 64 x 64 tiles 8.9;
// 4096 x 14336 at T = 1024 49.9 us, 128 x 128 tiles 37.9; 28672 x 4096 at T = 1
// 16.3 us, 64 x 128 tiles 12.8; and the other way round 57344 x 8192 at T = 1
// 42 us, 45 to 50 with narrower tiles, 28672 x 4096 at T = 1024 72 us, 128 x 128
// tiles 81. Split: 8192 x 28672 at T = 1 47 us whole, 24.5 us with S = 4.
MxPlan mx_plan(int64_t T, int64_t O, int64_t K, bool may_split) {
  const int64_t nsteps = ceil_div(K, 128);
  const int64_t s_max = !may_split || nsteps < 8 ? 1 : nsteps / 4 < kMxMaxSplits ? nsteps / 4 : kMxMaxSplits;
  const double bytes = mx_operand_bytes((double)O + (double)T, (double)K), out = (double)T * (double)O * 4.0;
  MxPlan p{0, 1, 0, 0};
  double best = 0;
  for (int t = 0; t < kMxTiles; ++t) {
    const int64_t tiles = ceil_div(T, kTiles[t].rows) * ceil_div(O, kTiles[t].cols);
    for (int64_t s = 1; s <= s_max && (s == 1 || s * T * O * 4 <= ((int64_t)256 << 20)); ++s) {
      if (s * tiles >= kMxMaxWorkgroups) break;
      double us = mx_loop_cost(t, (double)ceil_div(s * tiles, 256), ceil_div(nsteps, s), bytes);
      if (s > 1) us += 2.5 + 0.1 * (double)s + (double)(2 * s + 1) * out / 4.7e6;
      if ((t == 0 && s == 1) || us < best) best = us, p.tile = t, p.S = (int)s;
    }
  }
  p.tiles_m = (int)ceil_div(T, kTiles[p.tile].rows);
  p.tiles_total = p.tiles_m * (int)ceil_div(O, kTiles[p.tile].cols);
  return p;
}

// Column tiles of a gate|up product: they cover whole stages of h, 128 columns.
int64_t mx_silu_cols(int64_t I, int tile) { return ceil_div(I, 128) * (256 / kTiles[tile].cols); }

// Tile of a gate|up product whose K is not split, by the same costs: 2 x 14336 x
// 4096 at T = 1 19 us with 128 x 256, 13 with 64 x 128; 2 x 28672 x 8192 at T = 8
// 43 us with 32 x 256, 47 with the others; 2 x 4096 x 2048 at T = 512 12.6 us
// with 128 x 256, 9.9 with 128 x 128.
MxPlan mx_silu_plan(int64_t T, int64_t I, int64_t K) {
  MxPlan p{0, 1, 0, 0};
  double best = 0;
  for (int t = 0; t < kMxTiles; ++t) {
    const int64_t tiles = ceil_div(T, kTiles[t].rows) * mx_silu_cols(I, t);
    if (t == kMx64x64 || (t > 0 && tiles >= kMxMaxWorkgroups)) continue;
    const double us = mx_loop_cost(t, (double)ceil_div(tiles, 256), ceil_div(K, 128),
                                   mx_operand_bytes(2.0 * (double)I + (double)T, (double)K));
    if (t == 0 || us < best) best = us, p.tile = t;
  }
  p.tiles_m = (int)ceil_div(T, kTiles[p.tile].rows);
  p.tiles_total = p.tiles_m * (int)mx_silu_cols(I, p.tile);
  return p;
}

// Row slots of a grouped launch: no sorted segments of P rows fill more tiles.
int64_t mx_row_slots(int64_t P, int64_t E, int tile) {
  const int64_t filled = P < E ? P : E;
  return filled + (P - filled) / kTiles[tile].rows;
}

// Tile of a grouped product of `cols` columns (or h columns) of O weight rows,
// by the same costs for segments of about P / E rows, half a row tile more each
// for what does not fill one, and 1 us for every 512 workgroups' lookup of their
// tile. Fitted to timed launches of 18 expert layers (8 to 128 experts, 8 to
// 32768 pairs; within 1% of the best on average, 7% at most): the gate|up of 4096
// tokens x 8 of 128 experts (2048 -> 2 x 768) 93 us with 128 x 256, 117 and
// more with the others; of 4 tokens 14.4 us with 64 x 128, 16.1 with 128 x 256;
// the down product of 500 tokens x 3 of 16 experts (1024 -> 2080) 13.5 us with
// 128 x 256, 11.2 with 128 x 128.
int mx_grouped_tile(int64_t P, int64_t E, int64_t O, int64_t K, bool silu) {
  const double filled = (double)(P < E ? P : E), mean = (double)P / filled;
  const double bytes = mx_operand_bytes(filled * (double)O + (double)P, (double)K);
  int pick = 0;
  double best = 0;
  for (int t = 0; t < kMxTiles; ++t) {
    const int64_t cols = silu ? mx_silu_cols(O / 2, t) : ceil_div(O, kTiles[t].cols);
    if ((silu && t == kMx64x64) || (t > 0 && mx_row_slots(P, E, t) * cols + 8 > kMxMaxWorkgroups)) continue;
    const double rows = mean / (double)kTiles[t].rows + 0.5;
    const double tiles = filled * (rows > 1 ? rows : 1) * (double)cols;
    const double us = mx_loop_cost(t, tiles > 256 ? tiles / 256 : 1, ceil_div(K, 128), bytes) + ceil(tiles / 512);
    if (t == 0 || us < best) best = us, pick = t;
  }
  return pick;
}

// A multiple of 8, of which the XCDs take equal shares.
dim3 mx_grouped_grid(int64_t P, int64_t E, int tile, int64_t cols) {
  return dim3((unsigned)((mx_row_slots(P, E, tile) * cols + 7) / 8 * 8));
}

bool mx_wide(const void* y, int64_t ldy, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(y) & 15) == 0 && ldy * bytes % 16 == 0;
}

template <class Out>
void launch_mx_store(const MxPlan& p, const MxOperands& op, Out* y, int64_t ldy, hipStream_t stream) {
  const bool wide = mx_wide(y, ldy, sizeof(Out));
  mx_with_tile(p.tile, [&](auto c) {
    using C = decltype(c);
    hipLaunchKernelGGL((mx_linear_kernel<C, Out>), dim3(p.tiles_total), dim3(C::kThreads), 0, stream, op, y, ldy, wide,
                       p.tiles_m, p.tiles_total);
  });
}

void launch_mx_split(const MxPlan& p, const MxOperands& op, float* partials, hipStream_t stream) {
  const bool wide = op.O % 4 == 0;
  mx_with_tile(p.tile, [&](auto c) {
    using C = decltype(c);
    hipLaunchKernelGGL(mx_split_kernel<C>, dim3(p.tiles_total * p.S), dim3(C::kThreads), 0, stream, op, p.tiles_m,
                       p.tiles_total, p.S, wide, partials);
  });
}

}  // namespace

namespace {

int64_t mx_workspace(const MxPlan& p, int64_t T, int64_t O) { return p.S > 1 ? (int64_t)p.S * T * O * 4 : 0; }

// The plan of a product with a workspace of so many bytes.
MxPlan mx_plan_with(const MxProduct& m, const void* workspace, int64_t workspace_bytes) {
  const MxPlan p = mx_plan(m.rows, m.O, m.K, workspace != nullptr);
  return mx_workspace(p, m.rows, m.O) <= workspace_bytes ? p : mx_plan(m.rows, m.O, m.K, false);
}

}  // namespace

int64_t mx_linear_workspace_bytes(int64_t T, int64_t O, int64_t K) {
  return T <= 0 || O <= 0 ? 0 : mx_workspace(mx_plan(T, O, K, true), T, O);
}

hipError_t launch_mx_linear(const MxProduct& m, void* y, int64_t ldy, bool bf16, void* workspace,
                            int64_t workspace_bytes, hipStream_t stream) {
  const MxOperands op = mx_operands(m);
  const MxPlan p = mx_plan_with(m, workspace, workspace_bytes);
  if (p.S == 1) {
    if (bf16) launch_mx_store(p, op, static_cast<uint16_t*>(y), ldy, stream);
    else launch_mx_store(p, op, static_cast<float*>(y), ldy, stream);
    return hipGetLastError();
  }
  float* partials = static_cast<float*>(workspace);
  launch_mx_split(p, op, partials, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((m.rows * m.O + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(mx_reduce_kernel<uint16_t>, grid, dim3(256), 0, stream, partials, p.S, m.rows, m.O,
                       static_cast<uint16_t*>(y), ldy);
  else
    hipLaunchKernelGGL(mx_reduce_kernel<float>, grid, dim3(256), 0, stream, partials, p.S, m.rows, m.O,
                       static_cast<float*>(y), ldy);
  return hipGetLastError();
}

hipError_t launch_mx_linear_silu(const MxProduct& m, uint8_t* h_codes, uint8_t* h_scales, void* workspace,
                                 int64_t workspace_bytes, hipStream_t stream) {
  const MxOperands op = mx_operands(m);
  const MxH out{h_codes, h_scales, m.rows, m.O / 2};
  MxPlan p = mx_plan_with(m, workspace, workspace_bytes);
  if (p.S > 1) {
    float* partials = static_cast<float*>(workspace);
    launch_mx_split(p, op, partials, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t units = m.rows * ((out.I / 32 + 3) & ~(int64_t)3);
    hipLaunchKernelGGL(mx_reduce_silu_kernel, dim3((unsigned)((units + 7) / 8)), dim3(256), 0, stream, partials, p.S,
                       out);
    return hipGetLastError();
  }
  p = mx_silu_plan(m.rows, out.I, m.K);
  mx_with_tile(p.tile, [&](auto c) {
    using C = decltype(c);
    if constexpr (C::WN > 1)
      hipLaunchKernelGGL(mx_linear_silu_kernel<C>, dim3(p.tiles_total), dim3(C::kThreads), 0, stream, op, out,
                         p.tiles_m, p.tiles_total);
  });
  return hipGetLastError();
}

bool mx_grouped_fits(int64_t P, int32_t E, int64_t O) {
  return mx_row_slots(P, E, 0) * ceil_div(O, 256) + 8 <= kMxMaxWorkgroups;
}

hipError_t launch_mx_grouped(const MxProduct& m, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                             void* y, bool bf16, hipStream_t stream) {
  const MxOperands op = mx_operands(m);
  const int tile = mx_grouped_tile(P, E, m.O, m.K, false);
  const int tiles_n = (int)ceil_div(m.O, kTiles[tile].cols);
  const dim3 grid = mx_grouped_grid(P, E, tile, tiles_n);
  const bool wide = mx_wide(y, m.O, bf16 ? 2 : 4);
  mx_with_tile(tile, [&](auto c) {
    using C = decltype(c);
    if (bf16)
      hipLaunchKernelGGL((mx_grouped_kernel<C, uint16_t>), grid, dim3(C::kThreads), 0, stream, op, a_rows, seg, E,
                         static_cast<uint16_t*>(y), P, wide, tiles_n);
    else
      hipLaunchKernelGGL((mx_grouped_kernel<C, float>), grid, dim3(C::kThreads), 0, stream, op, a_rows, seg, E,
                         static_cast<float*>(y), P, wide, tiles_n);
  });
  return hipGetLastError();
}

hipError_t launch_mx_grouped_silu(const MxProduct& m, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                                  uint8_t* h_codes, uint8_t* h_scales, hipStream_t stream) {
  const MxOperands op = mx_operands(m);
  const MxH out{h_codes, h_scales, P, m.O / 2};
  const int tile = mx_grouped_tile(P, E, m.O, m.K, true);
  const int tiles_n = (int)mx_silu_cols(out.I, tile);
  const dim3 grid = mx_grouped_grid(P, E, tile, tiles_n);
  mx_with_tile(tile, [&](auto c) {
    using C = decltype(c);
    if constexpr (C::WN > 1)
      hipLaunchKernelGGL(mx_grouped_silu_kernel<C>, grid, dim3(C::kThreads), 0, stream, op, a_rows, seg, E, out,
                         tiles_n);
  });
  return hipGetLastError();
}

}  // namespace sharq

// Products of 8-bit integer codes with a scale for each token and each output
// channel on gfx950 MFMA, dense or per expert segment:
//   Y[t][o] = (sum_k qa[t][k] qw[o][k]) sa[t] sw[o] (+ bias[o]),
// stored as fp32 or bf16, or, for a fused gate|up weight, turned into
// h = bf16(silu(gate) * up). The sum is exact in int32 (K < 2^17), so no choice
// of tile or of how K is divided changes a result.
//
// V_MFMA_I32_16X16X64_I8 takes 16 weight rows as its first operand and 16
// activation rows as its second: lane l gives 16 bytes (K entries 16 (l / 16)
// on) of row l % 16 of each, and its four accumulators are weight rows
// 4 (l / 16) .. + 3 of token l % 16. On register operands it runs at 3.6-3.8
// POP/s where V_MFMA_I32_32X32X32_I8 runs at 3.0-3.4: the chip's power sets the
// clock, and this form draws less.

#pragma once

#include <type_traits>
#include <utility>

#include "gemm_common.h"
#include "sharq_device.h"
#include "sharq_internal.h"
#include "silu.h"

namespace sharq {
namespace {

#define SHARQ_INLINE __attribute__((always_inline))

// f(0), ..., f(N - 1) with the number as a compile-time constant.
template <class F, int... I>
__device__ __forceinline__ void static_for_each(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_each(f, std::make_integer_sequence<int, N>{});
}
template <int I>
using int_c = std::integral_constant<int, I>;

struct I8Operands {
  const int8_t* a_codes;  // [G][rows][64]
  const float* a_scales;  // [rows]
  const int8_t* w_codes;  // [G][O][64] (grouped: already the expert's)
  const float* w_scales;  // [O]
  const float* bias;      // [O] or null
  int64_t rows, O;
  int nsteps;  // G
};

struct I8Out {
  void* y;
  int64_t ld;
  bool wide;   // rows of y are 16-byte aligned
  int64_t I;   // h columns of a gate|up product
};

// What a kernel makes of a tile's sums.
enum I8Kind { kI8F32, kI8Bf16, kI8Silu };

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------

// A workgroup tile of BM tokens x BN weight rows. Its waves stand in KS groups,
// which divide K; the NWM x NWN waves of a group have WM x WN MFMA tiles of 16 x
// 16 each. A group has a ring of RING LDS stages (64 K entries of the tile's rows);
// WGS workgroups share a CU.
template <int WM_, int WN_, int NWM_, int NWN_, int KS_, int RING_, int WGS_>
struct I8Tile {
  static constexpr int WM = WM_, WN = WN_, NWM = NWM_, NWN = NWN_, KS = KS_;
  static constexpr int kGroup = NWM * NWN, kWaves = kGroup * KS, kThreads = 64 * kWaves;
  static constexpr int BM = 16 * WM * NWM, BN = 16 * WN * NWN;
  static constexpr int kOffW = BM * kRowBytes, kStage = (BM + BN) * kRowBytes;
  // 1 KB chunks of a stage; waves past the activation's last load the same bytes to the same place as an earlier one,
  // so that all count their loads alike
  static constexpr int kAChunks = BM / 16;
  static constexpr int kALoads = kAChunks < kGroup ? 1 : kAChunks / kGroup, kWLoads = BN / 16 / kGroup;
  static constexpr int kLoads = kALoads + kWLoads;
  static_assert((kAChunks < kGroup || kAChunks % kGroup == 0) && BN / 16 % kGroup == 0, "whole chunks per wave");
  static constexpr int kRing = RING_;
  static constexpr int kRingBytes = KS * kRing * kStage;
  static constexpr int kReduceBytes = (KS - 1) * BM * BN * 4;
  static constexpr int kMain = kRingBytes > kReduceBytes ? kRingBytes : kReduceBytes;
  // behind the ring: the tokens' scales, the weight rows' scales and biases
  static constexpr int kScaleA = kMain, kScaleW = kScaleA + 4 * (BM < 64 ? 64 : BM), kBias = kScaleW + 4 * BN;
  static constexpr int kLds = kBias + 4 * BN;
  static constexpr int kWavesPerSimd = (WGS_ * kWaves + 3) / 4;
  static_assert(BN % 64 == 0 && WN % 2 == 0, "whole scale loads, columns in pairs");
  static_assert(kRing >= 3 && WGS_ * (kLds + 64) <= kLdsBytes, "ring");
  // The same workgroup for half the rows: an expert's last row tile.
  using Half = I8Tile<(WM + 1) / 2, WN, NWM, NWN, KS, RING_, WGS_>;
};
// Named by rows x columns; kN: N groups divide K, where there are few tiles for the
// chip; wide ones load fewer operand bytes a MFMA, narrow ones are more and finish
// a stage sooner.
using I8x64x64k2 = I8Tile<2, 2, 2, 2, 2, 4, 2>;
using I8x64x128 = I8Tile<2, 4, 2, 2, 1, 4, 3>;
using I8x64x128k2 = I8Tile<2, 4, 2, 2, 2, 6, 1>;
using I8x128x128 = I8Tile<4, 4, 2, 2, 1, 3, 3>;
using I8x128x128k2 = I8Tile<4, 4, 2, 2, 2, 4, 1>;
using I8x128x256 = I8Tile<4, 8, 2, 2, 1, 3, 2>;
using I8x256x128 = I8Tile<8, 4, 2, 2, 1, 3, 2>;
using I8x256x128k2 = I8Tile<8, 4, 2, 2, 2, 3, 1>;
using I8x256x256 = I8Tile<8, 4, 2, 4, 1, 4, 1>;

// LDS chunk swizzle for the 16-row fragments: a ds_read_b128 serves lanes 0-3,
// 12-15, 20-23 and 24-27 (then 4-11, 16-19, 28-31, and the same from 32 on)
// together. Those are, for each residue of the row by 4 (a quarter of the 64
// banks), rows 4 q + r with q = 0, 3 of chunk c and q = 1, 2 of chunk c ^ 1; XOR
// of the chunk with -q puts the four on different banks (no conflicts measured;
// with +q, right for 32-row fragments, every read takes twice as long).
__device__ __forceinline__ int i8_swz_part(int row) { return (-(row >> 2)) & 3; }
__device__ __forceinline__ int i8_swz(int row, int part) {
  return row * kRowBytes + ((part ^ i8_swz_part(row)) << 4);
}

// Weight rows behind the LDS rows of a tile. A lane's accumulators of an MFMA tile
// are four columns side by side, 16 bytes of fp32: LDS rows in order. For 16 bytes
// of bf16 those of two (gate|up: four) neighbouring MFMA tiles are eight columns:
// 32 LDS rows are 32 output columns, row 16 j + r column 8 (r / 4) + 4 j + r % 4;
// gate|up: 64 rows are gate (j even) and up (j odd) of 32 h columns, row
// 16 j + r h column 8 (r / 4) + 4 (j / 2) + r % 4 (with two MFMA tiles a wave 32
// rows are gate and up of 16 h columns, in order).
template <class C, int K>
struct I8Cols {
  int64_t n0;  // first output (or h) column of the tile
  int64_t n;   // output (or h) columns
  static constexpr bool kEight = C::WN % 4 == 0;
  __device__ __forceinline__ int64_t w_row(int x) const {  // -1 past the last column
    const int j = x >> 4, r = x & 15;
    if constexpr (K == kI8F32) {
      return n0 + x < n ? n0 + x : -1;
    } else if constexpr (K == kI8Bf16) {
      const int64_t o = n0 + 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
      return o < n ? o : -1;
    } else {
      const int64_t h = n0 + (kEight ? 32 * (j >> 2) + 8 * (r >> 2) + 4 * ((j >> 1) & 1) + (r & 3) : 16 * (j >> 1) + r);
      return h < n ? h + ((j & 1) ? n : 0) : -1;
    }
  }
};

template <class C, int K>
constexpr int kI8Cols = K == kI8Silu ? C::BN / 2 : C::BN;  // output (or h) columns of a tile

// acc = the tile's sums; with KS groups, group q holds those of the WM rows i with
// i % KS == q when it returns.
//
// An iteration multiplies the fragments of one stage, read in the one before,
// and threads between its MFMAs the reads of the next stage's and the loads of
// stage s + ring into the slot that stage s left: at its barrier every wave has
// stage s in registers, and stage s + 1 has landed.
template <class C, int K>
__device__ __forceinline__ void i8_mainloop(const I8Operands& op, const TileRows& tr, const I8Cols<C, K>& tc,
                                            uint8_t* lds, v4i (&acc)[C::WM][C::WN]) {
  const int lane = threadIdx.x & 63, all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = all / C::kGroup, wave = all % C::kGroup;
  const int wm = wave % C::NWM, wn = wave / C::NWM, lr = lane & 15, lc = lane >> 4;
#pragma unroll
  for (int i = 0; i < C::WM; ++i)
#pragma unroll
    for (int j = 0; j < C::WN; ++j) acc[i][j] = v4i{};

  // Scales and biases, 64 at a load: older than any stage's loads, so there before the first is read.
  {
    const i32x4 ra = make_rsrc(op.a_scales, op.rows * 4), rw = make_rsrc(op.w_scales, op.O * 4);
    const i32x4 rb = make_rsrc(op.bias, op.bias ? op.O * 4 : 0);
    constexpr int kA = (C::BM + 63) / 64, kW = C::BN / 64;
    const uint32_t base = lds_offset(lds + C::kScaleA);
    for (int q = all; q < kA + 2 * kW; q += C::kWaves) {
      const int x = 64 * (q < kA ? q : (q - kA) % kW) + lane;
      const int64_t src = q < kA ? tr.src(x) : tc.w_row(x);
      buffer_to_lds4(q < kA ? ra : q < kA + kW ? rw : rb, src >= 0 ? (uint32_t)(src * 4) : kOOB, base + 256 * q);
    }
  }

  const int steps = (op.nsteps + C::KS - 1) / C::KS, first = kg * steps;
  int left = op.nsteps - first < steps ? op.nsteps - first : steps;  // stages not yet issued
  uint8_t* ring = lds + kg * C::kRing * C::kStage;
  StageView va, vw;
  va.start(reinterpret_cast<const uint8_t*>(op.a_codes), op.rows * kRowBytes, first);
  vw.start(reinterpret_cast<const uint8_t*>(op.w_codes), op.O * kRowBytes, first);
  if (left <= 0) va.r[2] = vw.r[2] = 0;
  // A lane fills a fixed LDS chunk; it reads the global chunk that belongs there after the swizzle.
  uint32_t a_off[C::kALoads], w_off[C::kWLoads];
#pragma unroll
  for (int j = 0; j < C::kALoads; ++j) {
    const int row = 16 * ((wave + C::kGroup * j) % C::kAChunks) + (lane >> 2);
    const int64_t src = tr.src(row);
    a_off[j] = src >= 0 ? (uint32_t)(src * kRowBytes + ((lane & 3) ^ i8_swz_part(row)) * 16) : kOOB;
  }
#pragma unroll
  for (int j = 0; j < C::kWLoads; ++j) {
    const int row = 16 * (wave + C::kGroup * j) + (lane >> 2);
    const int64_t src = tc.w_row(row);
    w_off[j] = src >= 0 ? (uint32_t)(src * kRowBytes + ((lane & 3) ^ i8_swz_part(row)) * 16) : kOOB;
  }
  const uint32_t base = lds_offset(ring) + 1024 * wave, a_back = 1024 * (wave - wave % C::kAChunks);
  uint32_t at = 0;
  auto issue = [&](auto J) SHARQ_INLINE {
    constexpr int j = decltype(J)::value;
    const uint32_t to = __builtin_amdgcn_readfirstlane(base + at);
    if constexpr (j < C::kALoads) {
      load_lds16<1024 * C::kGroup * j>(va.r, a_off[j], C::kAChunks < C::kGroup ? to - a_back : to);
      if constexpr (j == C::kALoads - 1) va.advance(--left > 0);
    } else {
      load_lds16<C::kOffW + 1024 * C::kGroup * (j - C::kALoads)>(vw.r, w_off[j - C::kALoads], to);
      if constexpr (j == C::kLoads - 1) {
        vw.advance(left > 0);
        at = at + C::kStage == C::kRing * C::kStage ? 0 : at + C::kStage;
      }
    }
  };
#pragma unroll
  for (int b = 0; b < C::kRing; ++b) static_for<C::kLoads>(issue);

  v4i fa[2][C::WM], fw[2][C::WN];
  constexpr int kReads = C::WM + C::WN, kMfmas = C::WM * C::WN;
  auto read = [&](auto R, auto SET, const uint8_t* st) SHARQ_INLINE {
    constexpr int r = decltype(R)::value, set = decltype(SET)::value;
    if constexpr (r < C::WM)
      fa[set][r] = *reinterpret_cast<const v4i*>(st + i8_swz(16 * (C::WM * wm + r) + lr, lc));
    else if constexpr (r < kReads)
      fw[set][r - C::WM] = *reinterpret_cast<const v4i*>(st + C::kOffW + i8_swz(16 * (C::WN * wn + r - C::WM) + lr, lc));
  };
  wait_vmcnt<(C::kRing - 1) * C::kLoads>();
  ring_barrier();
  static_for<kReads>([&](auto R) SHARQ_INLINE { read(R, int_c<0>{}, ring); });
  const uint8_t* cur = ring;
  // Reads go into the first 5/8 of the slots, so that the other MFMAs cover the latency of the last.
  constexpr int kReadSlots = kMfmas * 5 / 8 < 1 ? 1 : kMfmas * 5 / 8, kPerSlot = (kReads + kReadSlots - 1) / kReadSlots;
  auto body = [&](auto SET) SHARQ_INLINE {
    constexpr int set = decltype(SET)::value;
    const uint8_t* next = cur == ring + (C::kRing - 1) * C::kStage ? ring : cur + C::kStage;
    wait_vmcnt<(C::kRing - 2) * C::kLoads>();  // the next stage landed; later ones may be in flight
    ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    static_for<kMfmas>([&](auto M) SHARQ_INLINE {
      constexpr int m = decltype(M)::value, i = m / C::WN, j = m % C::WN;
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[set][j], fa[set][i], acc[i][j], 0, 0, 0);
      static_for<kPerSlot>([&](auto Q) SHARQ_INLINE { read(int_c<m * kPerSlot + decltype(Q)::value>{}, int_c<set ^ 1>{}, next); });
      constexpr int lo = (m * C::kLoads + kMfmas - 1) / kMfmas, hi = ((m + 1) * C::kLoads + kMfmas - 1) / kMfmas;
      static_for<hi - lo>([&](auto Q) SHARQ_INLINE { issue(int_c<lo + decltype(Q)::value>{}); });
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
    cur = next;
  };
  int s = 0;
#pragma unroll 1
  for (; s + 2 <= steps; s += 2) {
    body(int_c<0>{});
    body(int_c<1>{});
  }
  if (s < steps) body(int_c<0>{});
  wait_vmcnt<0>();  // the trailing batches, before the LDS is used again

  if constexpr (C::KS > 1) {
    ring_barrier();
    v4i* red = reinterpret_cast<v4i*>(lds);
    auto place = [&](int i, int q, int j) { return (((wave * C::WM + i) * (C::KS - 1) + q) * C::WN + j) * 64 + lane; };
#pragma unroll
    for (int i = 0; i < C::WM; ++i) {
      const int q = (kg - i % C::KS + C::KS) % C::KS;  // 0: this group finishes row i
      if (q > 0)
#pragma unroll
        for (int j = 0; j < C::WN; ++j) red[place(i, q - 1, j)] = acc[i][j];
    }
    ring_barrier();
#pragma unroll
    for (int i = 0; i < C::WM; ++i)
      if (i % C::KS == kg)
#pragma unroll
        for (int q = 0; q < C::KS - 1; ++q)
#pragma unroll
          for (int j = 0; j < C::WN; ++j) acc[i][j] += red[place(i, q, j)];
  }
}

// Eight (kN = 4: four) neighbouring columns to a row of y.
template <int kN, class Out>
__device__ __forceinline__ void i8_store(Out* __restrict__ y, const float (&v)[kN], int64_t o, int64_t n, bool wide) {
  if (wide && o + kN <= n) {
    if constexpr (sizeof(Out) == 4) {
#pragma unroll
      for (int e = 0; e < kN; e += 4)
        *reinterpret_cast<float4*>(y + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else if constexpr (kN == 8) {
      *reinterpret_cast<uint4*>(y) =
          make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
    } else {
      *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (o + e < n) {
        if constexpr (sizeof(Out) == 4) y[e] = v[e];
        else y[e] = (uint16_t)bf16_rne_bits(v[e]);
      }
  }
}

// The sum of a product's codes to its value: the int32 sum rounded once to fp32, a
// product and a fused one. (The gate and up values of a gate|up product are the same
// without the bias's addition.)
__device__ __forceinline__ float i8_value(int sum, float sa, float sw, float bias) {
  return fmaf((float)sum * sa, sw, bias);
}

template <class C, int K>
__device__ __forceinline__ void i8_epilogue(const v4i (&acc)[C::WM][C::WN], const uint8_t* lds, const TileRows& tr,
                                            int64_t n0, int64_t n, const I8Out& out) {
  using Out = std::conditional_t<K == kI8F32, float, uint16_t>;
  const int lane = threadIdx.x & 63, all = threadIdx.x >> 6;
  const int kg = all / C::kGroup, wave = all % C::kGroup;
  const int wm = wave % C::NWM, wn = wave / C::NWM, lr = lane & 15, lc = lane >> 4;
  const float* sa = reinterpret_cast<const float*>(lds + C::kScaleA);
  // scales (and biases) of the lane's four weight rows of MFMA tile j
  auto four = [&](int at, int j) {
    return *reinterpret_cast<const float4*>(lds + at + 4 * (16 * (C::WN * wn + j) + 4 * lc));
  };
#pragma unroll
  for (int i = 0; i < C::WM; ++i) {
    if (C::KS > 1 && i % C::KS != kg) continue;  // wave-uniform
    const int row = 16 * (C::WM * wm + i) + lr;
    if (row >= tr.rows_valid) continue;
    const float a = sa[row];
    Out* y = static_cast<Out*>(out.y) + (tr.m0 + row) * out.ld;
    if constexpr (K != kI8Silu) {
      constexpr int kTiles = K == kI8F32 ? 1 : 2;
#pragma unroll
      for (int j = 0; j < C::WN; j += kTiles) {
        float v[4 * kTiles];
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
          const float4 w = four(C::kScaleW, j + h), b = four(C::kBias, j + h);
          v[4 * h] = i8_value(acc[i][j + h][0], a, w.x, b.x);
          v[4 * h + 1] = i8_value(acc[i][j + h][1], a, w.y, b.y);
          v[4 * h + 2] = i8_value(acc[i][j + h][2], a, w.z, b.z);
          v[4 * h + 3] = i8_value(acc[i][j + h][3], a, w.w, b.w);
        }
        const int64_t o = n0 + 16 * (C::WN * wn + j) + 4 * kTiles * lc;
        i8_store(y + o, v, o, n, out.wide);
      }
    } else {
      constexpr int kPairs = C::WN % 4 == 0 ? 2 : 1;  // gate and up tiles behind a lane's columns
#pragma unroll
      for (int j = 0; j < C::WN; j += 2 * kPairs) {
        float v[4 * kPairs];
#pragma unroll
        for (int h = 0; h < kPairs; ++h) {
          const float4 g = four(C::kScaleW, j + 2 * h), u = four(C::kScaleW, j + 2 * h + 1);
          const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[4 * h + r] = silu_times((float)acc[i][j + 2 * h][r] * a * gs[r], (float)acc[i][j + 2 * h + 1][r] * a * us[r]);
        }
        const int64_t o = n0 + 8 * (C::WN * wn + j) + 4 * kPairs * lc;
        i8_store(y + o, v, o, n, out.wide);
      }
    }
  }
}

__device__ __forceinline__ TileRows i8_dense_rows(int64_t m0, int64_t T, int bm) {
  TileRows tr;
  tr.m0 = m0;
  tr.rows_valid = T - m0 < bm ? T - m0 : bm;
  tr.gather = nullptr;
  tr.src_rows = T;
  return tr;
}

template <class C, int K>
__device__ __forceinline__ void i8_tile(const I8Operands& op, const TileRows& tr, int64_t n0, const I8Out& out,
                                        uint8_t* lds) {
  const int64_t n = K == kI8Silu ? out.I : op.O;
  v4i acc[C::WM][C::WN];
  i8_mainloop<C, K>(op, tr, I8Cols<C, K>{n0, n}, lds, acc);
  i8_epilogue<C, K>(acc, lds, tr, n0, n, out);
}

// ---------------------------------------------------------------------------
// Few rows: operands straight into registers
// ---------------------------------------------------------------------------

// BM = 16 WM tokens x BN = 16 WN weight rows; the KW waves of a workgroup divide
// K, stage s to wave s % KW, and add their sums through LDS at the end. No
// operand passes through LDS and no barrier stands in the loop: a wave keeps the
// loads of PF stages in flight, which is what streaming a weight at the rate of
// memory takes.
template <int WM_, int WN_, int KW_, int PF_>
struct I8Thin {
  static constexpr int WM = WM_, WN = WN_, KW = KW_, PF = PF_;
  static constexpr int BM = 16 * WM, BN = 16 * WN, kThreads = 64 * KW;
  static constexpr int kLds = KW * WM * WN * 1024;
  static_assert(kLds <= kLdsBytes - 64, "the waves' sums");
};
using I8Thin16 = I8Thin<1, 2, 4, 4>;
using I8Thin16x64 = I8Thin<1, 4, 4, 4>;
using I8Thin32 = I8Thin<2, 2, 4, 4>;
using I8Thin64 = I8Thin<4, 2, 8, 2>;

template <class C, int K>
__device__ __forceinline__ void i8_thin_tile(const I8Operands& op, const TileRows& tr, int64_t n0, const I8Out& out,
                                             uint8_t* lds) {
  constexpr bool kSilu = K == kI8Silu;
  using Out = std::conditional_t<K == kI8F32, float, uint16_t>;
  const int64_t n = kSilu ? out.I : op.O;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lc = lane >> 4;
  // MFMA tile j has columns n0 + 16 j on; gate|up: gate (j even) or up (j odd) of h columns n0 + 16 (j / 2) on
  auto w_row = [&](int j, int r) -> int64_t {
    const int64_t o = n0 + 16 * (kSilu ? j / 2 : j) + r;
    return o < n ? o + (kSilu && (j & 1) ? n : 0) : -1;
  };
  uint32_t a_off[C::WM], w_off[C::WN];
#pragma unroll
  for (int i = 0; i < C::WM; ++i) {
    const int64_t src = tr.src(16 * i + lr);
    a_off[i] = src >= 0 ? (uint32_t)(src * kRowBytes + 16 * lc) : kOOB;
  }
#pragma unroll
  for (int j = 0; j < C::WN; ++j) {
    const int64_t src = w_row(j, lr);
    w_off[j] = src >= 0 ? (uint32_t)(src * kRowBytes + 16 * lc) : kOOB;
  }
  const int64_t a_stage = op.rows * kRowBytes, w_stage = op.O * kRowBytes;
  const int8_t *a = op.a_codes + wave * a_stage, *w = op.w_codes + wave * w_stage;
  int left = (op.nsteps - wave + C::KW - 1) / C::KW;  // stages of this wave not yet asked for
  const int trips = left;
  v4i fa[C::PF][C::WM], fw[C::PF][C::WN];
  auto load = [&](auto U) SHARQ_INLINE {  // past the last stage: views of nothing
    constexpr int u = decltype(U)::value;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)a, 0, left > 0 ? (int)a_stage : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)w, 0, left > 0 ? (int)w_stage : 0, 0x00020000);
#pragma unroll
    for (int j = 0; j < C::WN; ++j) fw[u][j] = __builtin_amdgcn_raw_buffer_load_b128(rw, w_off[j], 0, 0);
#pragma unroll
    for (int i = 0; i < C::WM; ++i) fa[u][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, a_off[i], 0, 0);
    a += C::KW * a_stage;
    w += C::KW * w_stage;
    --left;
  };
  static_for<C::PF>(load);
  // the scales of the columns that the thread finishes, four at a time
  constexpr int kCols = kSilu ? C::WN / 2 : C::WN, kUnits = 64 * C::WM * kCols;
  constexpr int kEach = kUnits < C::kThreads ? 1 : kUnits / C::kThreads;
  static_assert(kUnits < C::kThreads || kUnits % C::kThreads == 0, "threads finish columns alike");
  float sa[kEach], sw[kEach][4], su[kEach][4], bias[kEach][4];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int unit = threadIdx.x + e * C::kThreads, i = (unit >> 6) / kCols, j = (unit >> 6) % kCols;
    sa[e] = 0.0f;
    if (unit < kUnits) {
      const int64_t src = tr.src(16 * i + lr);
      if (src >= 0) sa[e] = op.a_scales[src];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t o = w_row(kSilu ? 2 * j : j, 4 * lc + r);
        sw[e][r] = o >= 0 ? op.w_scales[o] : 0.0f;
        bias[e][r] = !kSilu && o >= 0 && op.bias ? op.bias[o] : 0.0f;
        su[e][r] = kSilu && o >= 0 ? op.w_scales[o + n] : 0.0f;
      }
    }
  }
  v4i acc[C::WM][C::WN];
#pragma unroll
  for (int i = 0; i < C::WM; ++i)
#pragma unroll
    for (int j = 0; j < C::WN; ++j) acc[i][j] = v4i{};
#pragma unroll 1
  for (int s = 0; s < trips; s += C::PF)
    static_for<C::PF>([&](auto U) SHARQ_INLINE {
      constexpr int u = decltype(U)::value;
#pragma unroll
      for (int i = 0; i < C::WM; ++i)
#pragma unroll
        for (int j = 0; j < C::WN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][j], fa[u][i], acc[i][j], 0, 0, 0);
      load(U);
    });

  v4i* red = reinterpret_cast<v4i*>(lds);
#pragma unroll
  for (int i = 0; i < C::WM; ++i)
#pragma unroll
    for (int j = 0; j < C::WN; ++j) red[((wave * C::WM + i) * C::WN + j) * 64 + lane] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int unit = threadIdx.x + e * C::kThreads, i = (unit >> 6) / kCols, j = (unit >> 6) % kCols, row = 16 * i + lr;
    if (unit >= kUnits || row >= tr.rows_valid) continue;
    auto sum = [&](int tile) {
      v4i v = v4i{};
#pragma unroll
      for (int q = 0; q < C::KW; ++q) v += red[((q * C::WM + i) * C::WN + tile) * 64 + lane];
      return v;
    };
    float v[4];
    if constexpr (kSilu) {
      const v4i g = sum(2 * j), u = sum(2 * j + 1);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = silu_times((float)g[r] * sa[e] * sw[e][r], (float)u[r] * sa[e] * su[e][r]);
    } else {
      const v4i q = sum(j);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = i8_value(q[r], sa[e], sw[e][r], bias[e][r]);
    }
    const int64_t o = n0 + 16 * j + 4 * lc;
    i8_store(static_cast<Out*>(out.y) + (tr.m0 + row) * out.ld + o, v, o, n, out.wide);
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------

inline I8Operands i8_operands(const I8Product& p) {
  return I8Operands{p.a_codes, p.a_scales, p.w_codes, p.w_scales, p.bias, p.rows, p.O, (int)((p.K + 63) / 64)};
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// For the choice of a tile alone, in microseconds: of a stage on a CU, by a
// workgroup's own chain and by each workgroup's share of the CU; of the ends of each
// workgroup there; and of the launch.
struct I8TileCost {
  int64_t rows, cols;
  double chain, each, ends, launch;
  int per_cu = 1;  // workgroups that share a CU
};

// The loops of a launch, and no less than its bytes at the rate of memory.
inline double i8_cost(double launch, double loops, double bytes) {
  const double stream = bytes / 5.6e6;
  return launch + (loops > stream ? loops + 0.1 * stream : stream + 0.1 * loops);
}

// Column tiles of a product of O weight rows (gate|up: of O / 2 h columns).
inline int64_t i8_cols(int64_t O, bool silu, const I8TileCost& c) {
  return silu ? ceil_div(O / 2, c.cols / 2) : ceil_div(O, c.cols);
}

inline double i8_out_bytes(int64_t rows, int64_t O, I8Kind kind) {
  return (double)rows * (double)O * (kind == kI8F32 ? 4.0 : kind == kI8Bf16 ? 2.0 : 1.0);
}

inline bool i8_wide(const void* y, int64_t ld, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(y) & 15) == 0 && ld * bytes % 16 == 0;
}

inline int64_t i8_h_ld(int64_t I) { return (I + 7) & ~(int64_t)7; }

}  // namespace
}  // namespace sharq

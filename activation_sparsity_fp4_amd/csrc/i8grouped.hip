// Products of 8-bit codes per expert segment: kernels and the choice of a tile
// (i8gemm.h has the products themselves).

#include "i8gemm.h"

namespace sharq {
namespace {

__device__ __forceinline__ void i8_select_expert(I8Operands& op, int e) {
  op.w_codes += (int64_t)e * op.O * kRowBytes * op.nsteps;
  op.w_scales += (int64_t)e * op.O;
}

// Per expert. Many tokens: bound by the ends of the workgroups' short loops and by cold
// weights. 4096 tokens x 8 of 128 experts, 2048 -> 2 x 768 151-155 us (160-170 in the first
// passes on new inputs), 768 -> 2048 98-105 us; the same products dense 90 and 62, with
// segments of 256 rows each 141 and 90, with 64 experts of 512 rows 111 and 78. 1024 tokens
// x 2 of 8, 4096 -> 14336, ragged: 157-160 us where the least is 103 (the 470 MB of weights
// 91 of it), with tiles that fill 75% of their rows. (The experts' full row tiles first and
// the short ones last: 171 us for 164 then; three quarters of the height as a fourth loop:
// no gain.)
template <class C, int K>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void i8_grouped_kernel(
    I8Operands op, const int32_t* __restrict__ a_rows, const int32_t* __restrict__ seg, int E, int64_t P, I8Out out,
    int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  // With column tiles in eights each XCD keeps a column slice of every weight, and all have the same work (1024 tokens x
  // 2 of 8 experts, 4096 -> 2 x 14336: 280 us, 375 with ranges); otherwise an XCD takes a range of tiles, so that an
  // expert's row tiles share its weight in one L2. Column by column those widths take longer: there, of skewed segments,
  // 10.4 us per 1000 weight rows at 14336 (112 column tiles), 12.9 at 11008 (86), 12.6 at 13824 (108); without SiLU
  // 4096 -> 14336 11.1 (56), 11008 13.4 (43), 13824 12.1 (54).
  const GroupedTile g = (tiles_n & 7) == 0 ? grouped_tile<C, false>(seg, E, P, a_rows, op.rows, tiles_n)
                                           : grouped_tile<C, true>(seg, E, P, a_rows, op.rows, tiles_n);
  if (g.e < 0) return;  // uniform across the workgroup
  i8_select_expert(op, g.e);
  // A tile with few rows (an expert's last) runs the loop of one of half or a quarter of the height: fewer MFMAs and
  // loads for the same weight tile.
  const int64_t n0 = (int64_t)g.col * kI8Cols<C, K>;
  using Half = typename C::Half;
  using Quarter = typename Half::Half;
  static_assert(Half::kLds <= C::kLds && Quarter::kLds <= C::kLds, "in the same LDS");
  if (g.tr.rows_valid > Half::BM) i8_tile<C, K>(op, g.tr, n0, out, lds);
  else if (g.tr.rows_valid > Quarter::BM) i8_tile<Half, K>(op, g.tr, n0, out, lds);
  else i8_tile<Quarter, K>(op, g.tr, n0, out, lds);
}

// Few tokens: the weights' bytes and the lookup of the tile. 4 tokens x 8 of 128 experts
// gate|up 20-22 us (91 MB, 4.2-4.6 TB/s); 1 token x 2 of 8, 4096 -> 2 x 14336 43 us (235 MB),
// 14336 -> 4096 20 us.
template <class C, int K>
__global__ __launch_bounds__(C::kThreads) void i8_thin_grouped_kernel(I8Operands op, const int32_t* __restrict__ a_rows,
                                                                      const int32_t* __restrict__ seg, int E,
                                                                      int64_t P, I8Out out, int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const GroupedTile g = grouped_tile<C, false>(seg, E, P, a_rows, op.rows, tiles_n);
  if (g.e < 0) return;  // uniform across the workgroup
  i8_select_expert(op, g.e);
  i8_thin_tile<C, K>(op, g.tr, (int64_t)g.col * kI8Cols<C, K>, out, lds);
}

constexpr int kI8Tiles = 7;
constexpr I8TileCost kI8Costs[kI8Tiles] = {
    {16, 32, 0.094, 0.009, 1.16, 2.0},  {16, 64, 0.119, 0.028, 1.39, 2.4},  {64, 128, 0.012, 0.190, 0.61, 2.6},
    {128, 128, 0.214, 0.286, 2.98, 2.1}, {128, 256, 0.603, 0.499, 2.18, 2.2}, {256, 128, 0.032, 0.338, 8.61, 3.5},
    {256, 256, 0.554, 0.537, 9.11, 3.5}};

// Calls f with the tile type of kI8Costs[tile] and whether it is a thin one.
template <class F>
void i8_with_tile(int tile, F f) {
  switch (tile) {
    case 0: f(I8Thin16{}, std::true_type{}); break;
    case 1: f(I8Thin16x64{}, std::true_type{}); break;
    case 2: f(I8x64x128{}, std::false_type{}); break;
    case 3: f(I8x128x128{}, std::false_type{}); break;
    case 4: f(I8x128x256{}, std::false_type{}); break;
    case 5: f(I8x256x128k2{}, std::false_type{}); break;
    default: f(I8x256x256{}, std::false_type{}); break;
  }
}

// Row slots of a grouped launch: no sorted segments of P rows fill more tiles.
int64_t i8_row_slots(int64_t P, int64_t E, int64_t rows) {
  const int64_t filled = P < E ? P : E;
  return filled + (P - filled) / rows;
}

int64_t i8_grid(int64_t P, int64_t E, int64_t O, bool silu, const I8TileCost& c) {
  return (i8_row_slots(P, E, c.rows) * i8_cols(O, silu, c) + 7) / 8 * 8;  // XCDs take equal shares
}

// The cheapest tile by the costs, for segments of about P / min(P, E) rows, 0.58 row
// tiles more each for what does not fill one, and 0.42 us for every 512 workgroups'
// lookup of their tile. Fitted to timed launches on 88 expert layers (8 to 128
// experts, 2 to 32768 pairs, even segments); up to 4 rows an expert the fit took the
// other tiles' times 6% longer than they were, for thin tiles keep more of a cold
// weight in flight: that preference is in the constants. In graphs on cold weights
// the pick is 2.5% over the best on average there and 3.9% at 40 layers held out, with
// skewed segments (24% at most). Farthest off: 16 to 32 rows each of 8 experts, 14336 ->
// 4096, thin tiles where 64 x 128 is faster (128 x 2: 120 us for 79). The costs do not
// know in which order of the column tiles a tile runs.
int i8_grouped_tile(int64_t P, int64_t E, int64_t O, int64_t K, I8Kind kind) {
  const double filled = (double)(P < E ? P : E), mean = (double)P / filled;
  const double bytes = (filled * (double)O + (double)P) * (double)K + i8_out_bytes(P, O, kind);
  int pick = kI8Tiles - 1;
  double best = 0;
  for (int t = kI8Tiles - 1; t >= 0; --t) {
    if (i8_grid(P, E, O, kind == kI8Silu, kI8Costs[t]) >= kI8MaxWorkgroups) break;  // narrower ones are more
    const double rows = mean / (double)kI8Costs[t].rows + 0.58;
    const double tiles = filled * (rows > 1 ? rows : 1) * (double)i8_cols(O, kind == kI8Silu, kI8Costs[t]);
    const I8TileCost& c = kI8Costs[t];
    const double share = tiles > 256 ? tiles / 256 : 1, each = c.each * share;
    const double loops = (double)ceil_div(K, 64) * (c.chain > each ? c.chain : each) + c.ends * share;
    const double us = i8_cost(c.launch, loops, bytes) + 0.42 * tiles / 512;
    if (t == kI8Tiles - 1 || us < best) best = us, pick = t;
  }
  return pick;
}

template <I8Kind K>
hipError_t i8_launch_grouped(const I8Operands& op, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                             const I8Out& out, int64_t K_, hipStream_t stream) {
  const int tile = i8_grouped_tile(P, E, op.O, K_, K);
  const int64_t tiles_n = i8_cols(op.O, K == kI8Silu, kI8Costs[tile]);
  const dim3 grid((unsigned)i8_grid(P, E, op.O, K == kI8Silu, kI8Costs[tile]));
  i8_with_tile(tile, [&](auto c, auto thin) {
    using C = decltype(c);
    if constexpr (decltype(thin)::value)
      hipLaunchKernelGGL((i8_thin_grouped_kernel<C, K>), grid, dim3(C::kThreads), 0, stream, op, a_rows, seg, E, P, out,
                         (int)tiles_n);
    else
      hipLaunchKernelGGL((i8_grouped_kernel<C, K>), grid, dim3(C::kThreads), 0, stream, op, a_rows, seg, E, P, out,
                         (int)tiles_n);
  });
  return hipGetLastError();
}

}  // namespace

I8TileChoice i8_grouped_choice(int64_t P, int32_t E, int64_t O, int64_t K, int kind) {
  const int tile = i8_grouped_tile(P, E, O, K, (I8Kind)kind);
  return I8TileChoice{tile, kI8Tiles, (int)kI8Costs[tile].rows, (int)kI8Costs[tile].cols};
}

bool i8_grouped_fits(int64_t P, int32_t E, int64_t O) {
  return (i8_row_slots(P, E, 256) + 1) * (ceil_div(O, 256) + 1) < kI8MaxWorkgroups;
}

hipError_t launch_i8_grouped(const I8Product& p, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                             void* y, bool bf16, hipStream_t stream) {
  const I8Operands op = i8_operands(p);
  const I8Out out{y, p.O, i8_wide(y, p.O, bf16 ? 2 : 4), 0};
  return bf16 ? i8_launch_grouped<kI8Bf16>(op, a_rows, seg, E, P, out, p.K, stream)
              : i8_launch_grouped<kI8F32>(op, a_rows, seg, E, P, out, p.K, stream);
}

hipError_t launch_i8_grouped_silu(const I8Product& p, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                                  int8_t* h_codes, float* h_scales, void* workspace, hipStream_t stream) {
  const int64_t I = p.O / 2, ld = i8_h_ld(I);
  const I8Out out{workspace, ld, true, I};
  const hipError_t e = i8_launch_grouped<kI8Silu>(i8_operands(p), a_rows, seg, E, P, out, p.K, stream);
  if (e != hipSuccess) return e;
  return launch_quantize_int8(workspace, 1, 1, P, I, ld, h_codes, h_scales, seg, E, stream);
}

}  // namespace sharq

// Dense products of 8-bit codes: kernels and the choice of a tile (i8gemm.h has
// the products themselves).

#include "i8gemm.h"

namespace sharq {
namespace {

// Many tokens: bound by the matrix cores at the clock that their power leaves, and by
// the loads' way from L2. 8192 x 8192 x 8192 (bf16 out, 256 x 256 tiles) 400-408 us, 2.75
// POP/s: the matrix cores are busy 71% at 1.81 GHz. 2048 x 14336 x 4096 95 us with bf16
// out, 100 with fp32 (60% at 1.94 GHz): one workgroup a CU, whose first loads, sum over
// its K groups and stores overlap nothing. 2048 x 4096 -> 2 x 14336 with SiLU 190 us (67%
// at 1.74 GHz); a 256 x 256 tile's SiLU takes 6 us of vector instructions, which with two
// workgroups of 256 x 128 a CU run beside the other's MFMAs.
template <class C, int K>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void i8_linear_kernel(I8Operands op, I8Out out,
                                                                                  int tiles_m, int tiles_total) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const TileIndex ti = tile_index(blockIdx.x, tiles_m, tiles_total);
  i8_tile<C, K>(op, i8_dense_rows((int64_t)ti.tm * C::BM, op.rows, C::BM), (int64_t)ti.tn * kI8Cols<C, K>, out, lds);
}

// Few tokens: bound by the weight's bytes (1 x 28672 x 8192 38 us, 6.2 TB/s; 8 x 8192 ->
// 2 x 28672 83 us, 5.7 TB/s, where tiles through LDS take 82) or by the round trips of one
// (1 x 4096 x 4096 5.2-5.6 us, 6.4 where the weight is in no cache).
template <class C, int K>
__global__ __launch_bounds__(C::kThreads) void i8_thin_kernel(I8Operands op, I8Out out, int tiles_m) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
  i8_thin_tile<C, K>(op, i8_dense_rows((int64_t)tm * C::BM, op.rows, C::BM), (int64_t)tn * kI8Cols<C, K>, out, lds);
}

constexpr int kI8Tiles = 12;
constexpr I8TileCost kI8Costs[kI8Tiles] = {
    {16, 32, 0.014, 0.032, 1.96, 2.8, 4},   {32, 32, 0.007, 0.039, 1.28, 2.7, 4}, {64, 32, 0.001, 0.075, 2.74, 2.4, 2},
    {64, 64, 0.045, 0.082, 1.31, 2.4, 2},   {64, 128, 0.042, 0.184, 1.57, 2.0, 3}, {64, 128, 0.152, 0.0, 1.82, 2.8},
    {128, 128, 0.309, 0.197, 1.80, 2.1, 3}, {128, 128, 0.0, 0.197, 3.46, 2.2},     {128, 256, 0.278, 0.355, 4.9, 2.0, 2},
    {256, 128, 0.464, 0.326, 3.26, 2.6, 2}, {256, 128, 0.0, 0.341, 5.46, 2.0},     {256, 256, 0.601, 0.0, 9.6, 2.8}};

// n workgroups on the busiest CU: per_cu at a time, then the rest.
double i8_loops(const I8TileCost& c, int64_t n, int64_t steps) {
  auto stage = [&](int64_t together) { return c.each * (double)together > c.chain ? c.each * (double)together : c.chain; };
  const int64_t rounds = n / c.per_cu, rest = n % c.per_cu;
  return (double)steps * ((double)rounds * stage(c.per_cu) + (rest ? stage(rest) : 0.0)) + c.ends * (double)n;
}

// Calls f with the tile type of kI8Costs[tile] and whether it is a thin one.
template <class F>
void i8_with_tile(int tile, F f) {
  switch (tile) {
    case 0: f(I8Thin16{}, std::true_type{}); break;
    case 1: f(I8Thin32{}, std::true_type{}); break;
    case 2: f(I8Thin64{}, std::true_type{}); break;
    case 3: f(I8x64x64k2{}, std::false_type{}); break;
    case 4: f(I8x64x128{}, std::false_type{}); break;
    case 5: f(I8x64x128k2{}, std::false_type{}); break;
    case 6: f(I8x128x128{}, std::false_type{}); break;
    case 7: f(I8x128x128k2{}, std::false_type{}); break;
    case 8: f(I8x128x256{}, std::false_type{}); break;
    case 9: f(I8x256x128{}, std::false_type{}); break;
    case 10: f(I8x256x128k2{}, std::false_type{}); break;
    default: f(I8x256x256{}, std::false_type{}); break;
  }
}

// The cheapest tile by the costs. They were fitted to launches of all tiles on 10 layer
// shapes from 512 x 4096 to 4096 x 28672 (K x O), T = 1 .. 4096, and on larger ones at
// few tokens; up to 16 tokens the fit took the other tiles' times 6% longer than they
// were, for thin tiles keep more of a cold weight in flight: that preference is in the
// constants. In graphs on cold weights the pick is 4% over the best on average at those
// sizes, 11% at 64 held out (45% at most): the fit saw no launch below the 4.8 us that
// the host takes for one, and products of less take 64 x 64 with K in two where 16 x 32
// is shorter (1 x 768 x 2048 4.2 and 3.0 us). There also: 1 x 28672 x 8192 38-40 us in thin
// tiles, 55 to 237 in the others; 2048 x 4096 -> 2 x 14336 192 us in 256 x 128, 198 in
// 128 x 256, 216 in 256 x 256; 256 x 4096 x 4096 12.0 us in 64 x 64 with K in two, 17 in
// 64 x 128, 18 in 64 x 32; 2048 x 14336 x 4096 96 us in 256 x 128 with K in two, 107
// without.
int i8_dense_tile(int64_t T, int64_t O, int64_t K, I8Kind kind) {
  const double bytes = ((double)O + (double)T) * (double)K + i8_out_bytes(T, O, kind);
  int pick = kI8Tiles - 1;
  double best = 0;
  for (int t = kI8Tiles - 1; t >= 0; --t) {
    const int64_t tiles = ceil_div(T, kI8Costs[t].rows) * i8_cols(O, kind == kI8Silu, kI8Costs[t]);
    if (tiles >= kI8MaxWorkgroups) break;  // narrower ones are more
    if ((t == 1 || t == 2) && T <= kI8Costs[t - 1].rows) continue;  // the thin tile of half the rows has them all
    const double us = i8_cost(kI8Costs[t].launch, i8_loops(kI8Costs[t], ceil_div(tiles, 256), ceil_div(K, 64)), bytes);
    if (t == kI8Tiles - 1 || us < best) best = us, pick = t;
  }
  return pick;
}

template <I8Kind K>
hipError_t i8_launch_dense(const I8Operands& op, const I8Out& out, int64_t K_, hipStream_t stream) {
  const int tile = i8_dense_tile(op.rows, op.O, K_, K);
  const int64_t tiles_m = ceil_div(op.rows, kI8Costs[tile].rows),
                tiles = tiles_m * i8_cols(op.O, K == kI8Silu, kI8Costs[tile]);
  i8_with_tile(tile, [&](auto c, auto thin) {
    using C = decltype(c);
    if constexpr (decltype(thin)::value)
      hipLaunchKernelGGL((i8_thin_kernel<C, K>), dim3((unsigned)tiles), dim3(C::kThreads), 0, stream, op, out,
                         (int)tiles_m);
    else
      hipLaunchKernelGGL((i8_linear_kernel<C, K>), dim3((unsigned)tiles), dim3(C::kThreads), 0, stream, op, out,
                         (int)tiles_m, (int)tiles);
  });
  return hipGetLastError();
}

}  // namespace

I8TileChoice i8_linear_choice(int64_t T, int64_t O, int64_t K, int kind) {
  const int tile = i8_dense_tile(T, O, K, (I8Kind)kind);
  return I8TileChoice{tile, kI8Tiles, (int)kI8Costs[tile].rows, (int)kI8Costs[tile].cols};
}

bool i8_linear_fits(int64_t T, int64_t O) { return ceil_div(T, 256) * ceil_div(O, 256) < kI8MaxWorkgroups; }

hipError_t launch_i8_linear(const I8Product& p, void* y, int64_t ldy, bool bf16, hipStream_t stream) {
  const I8Operands op = i8_operands(p);
  const I8Out out{y, ldy, i8_wide(y, ldy, bf16 ? 2 : 4), 0};
  return bf16 ? i8_launch_dense<kI8Bf16>(op, out, p.K, stream) : i8_launch_dense<kI8F32>(op, out, p.K, stream);
}

int64_t i8_silu_workspace_bytes(int64_t T, int64_t I) { return T * i8_h_ld(I) * 2; }

hipError_t launch_i8_linear_silu(const I8Product& p, int8_t* h_codes, float* h_scales, void* workspace,
                                 hipStream_t stream) {
  const int64_t I = p.O / 2, ld = i8_h_ld(I);
  const I8Out out{workspace, ld, true, I};
  const hipError_t e = i8_launch_dense<kI8Silu>(i8_operands(p), out, p.K, stream);
  if (e != hipSuccess) return e;
  return launch_quantize_int8(workspace, 1, 1, p.rows, I, ld, h_codes, h_scales, nullptr, 0, stream);
}

}  // namespace sharq

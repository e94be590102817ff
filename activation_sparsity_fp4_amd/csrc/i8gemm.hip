// Dense products of 8-bit codes: kernels and the choice of a tile (i8gemm.h has
// the products themselves).

#include "i8gemm.h"

namespace sharq {
namespace {

template <class C, int K>
__global__ __launch_bounds__(C::kThreads, C::kWavesPerSimd) void i8_linear_kernel(I8Operands op, I8Out out,
                                                                                  int tiles_m, int tiles_total) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const TileIndex ti = tile_index(blockIdx.x, tiles_m, tiles_total);
  i8_tile<C, K>(op, i8_dense_rows((int64_t)ti.tm * C::BM, op.rows, C::BM), (int64_t)ti.tn * kI8Cols<C, K>, out, lds);
}

template <class C, int K>
__global__ __launch_bounds__(C::kThreads) void i8_thin_kernel(I8Operands op, I8Out out, int tiles_m) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
  i8_thin_tile<C, K>(op, i8_dense_rows((int64_t)tm * C::BM, op.rows, C::BM), (int64_t)tn * kI8Cols<C, K>, out, lds);
}

constexpr int kI8Tiles = 12;
constexpr I8TileCost kI8Costs[kI8Tiles] = {
    {16, 32, 0.012, 0.040, 0.68, 2.6},   {32, 32, 0.051, 0.070, 0.57, 2.5},   {64, 32, 0.101, 0.067, 1.22, 3.2},
    {64, 64, 0.056, 0.104, 1.18, 2.6},   {64, 128, 0.045, 0.180, 0.43, 2.2},  {64, 128, 0.055, 0.152, 0.98, 2.6},
    {128, 128, 0.139, 0.230, 1.6, 3.0},  {128, 128, 0.125, 0.218, 1.18, 3.8}, {128, 256, 0.092, 0.477, 1.32, 2.75},
    {256, 128, 0.106, 0.387, 1.16, 3.6}, {256, 128, 0.087, 0.325, 10.0, 0.0}, {256, 256, 0.110, 0.670, 2.7, 3.6}};

// Calls f with the tile type of kI8Costs[tile] and whether it is a thin one.
template <class F>
void i8_with_tile(int tile, F f) {
  switch (tile) {
    case 0: f(I8Thin16{}, std::true_type{}); break;
    case 1: f(I8Thin32{}, std::true_type{}); break;
    case 2: f(I8Thin64{}, std::true_type{}); break;
    case 3: f(I8x64x64k4{}, std::false_type{}); break;
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

// The cheapest tile by the costs, which are fitted to timed launches of all of them
// on 10 layer shapes from 512 x 4096 to 4096 x 28672 (K x O), T = 1 .. 4096, and
// the 8192 x 57344 pair: within 1.3% of the best on average, 15% at most.
int i8_dense_tile(int64_t T, int64_t O, int64_t K, I8Kind kind) {
  const double bytes = ((double)O + (double)T) * (double)K + i8_out_bytes(T, O, kind);
  int pick = kI8Tiles - 1;
  double best = 0;
  for (int t = kI8Tiles - 1; t >= 0; --t) {
    const int64_t tiles = ceil_div(T, kI8Costs[t].rows) * i8_cols(O, kind == kI8Silu, kI8Costs[t]);
    if (tiles >= kI8MaxWorkgroups) break;  // narrower ones are more
    const double us = i8_cost(kI8Costs[t], (double)ceil_div(tiles, 256), ceil_div(K, 64), bytes);
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

// Launchers behind the C ABI. Arguments reaching these have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sharq {

// rms_scale == nullptr: no RMSNorm; otherwise r per row is written there and
// absorbed (rms_eps > 0).
hipError_t launch_prepare(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma,
                          float rms_eps, float* rms_scale, int n, int m, uint8_t* bb_codes, uint8_t* bb_scales,
                          uint8_t* res_codes, uint8_t* res_scales, uint8_t* mask, hipStream_t stream);

hipError_t launch_quantize(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, uint8_t* codes,
                           uint8_t* scales, hipStream_t stream);

hipError_t launch_linear(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                         const uint8_t* res_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                         int64_t T, int64_t O, int64_t K, float* y, int64_t ldy, hipStream_t stream);

int64_t linear_workspace_bytes(int64_t T, int64_t O, int64_t K);
int64_t linear_silu_prepare_workspace_bytes(int64_t T, int64_t I, int64_t K);

hipError_t launch_linear_ws(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                            const uint8_t* res_scales, const uint8_t* w_codes, const uint8_t* w_scales, int64_t T,
                            int64_t O, int64_t K, float* y, int64_t ldy, void* workspace, int64_t workspace_bytes,
                            hipStream_t stream);

// The scratch-free split-K GEMM (scratchfree.hip): whether the split plan's
// partials fit its static array, and the launch.
bool linear_scratchfree_fits(int64_t T, int64_t O, int64_t K);
hipError_t launch_linear_scratchfree(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                                     const uint8_t* res_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                     int64_t T, int64_t O, int64_t K, float* y, int64_t ldy, hipStream_t stream);

hipError_t launch_linear_grouped(const uint8_t* bb_codes, const uint8_t* bb_scales,
                                 const uint8_t* res_codes, const uint8_t* res_scales,
                                 const int32_t* a_rows, const int32_t* seg_offsets, int32_t E,
                                 const uint8_t* w_codes, const uint8_t* w_scales, int64_t P, int64_t O,
                                 int64_t K, float* y, int64_t a_rows_total, hipStream_t stream);

hipError_t launch_linear_silu_prepare(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                                      const uint8_t* res_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                      int64_t T, int64_t I, int64_t K, int n, int m, uint16_t* h,
                                      uint8_t* h_bb_codes, uint8_t* h_bb_scales, uint8_t* h_res_codes,
                                      uint8_t* h_res_scales, uint8_t* h_mask, hipStream_t stream);

hipError_t launch_linear_silu_prepare_ws(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                                         const uint8_t* res_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                                         int64_t T, int64_t I, int64_t K, int n, int m, uint16_t* h,
                                         uint8_t* h_bb_codes, uint8_t* h_bb_scales, uint8_t* h_res_codes,
                                         uint8_t* h_res_scales, uint8_t* h_mask, void* workspace,
                                         int64_t workspace_bytes, hipStream_t stream);

hipError_t launch_linear_grouped_silu_prepare(const uint8_t* bb_codes, const uint8_t* bb_scales,
                                              const uint8_t* res_codes, const uint8_t* res_scales,
                                              const int32_t* a_rows, const int32_t* seg_offsets, int32_t E,
                                              const uint8_t* w_codes, const uint8_t* w_scales, int64_t P, int64_t I,
                                              int64_t K, int64_t a_rows_total, int n, int m, uint16_t* h,
                                              uint8_t* h_bb_codes, uint8_t* h_bb_scales, uint8_t* h_res_codes,
                                              uint8_t* h_res_scales, uint8_t* h_mask, hipStream_t stream);

int64_t backbone_meta_row_bytes(int64_t K, int m);

hipError_t launch_compress_backbone(const uint8_t* bb_codes, const uint8_t* mask, int64_t T, int64_t K, int n, int m,
                                    uint8_t* codes, uint8_t* meta, hipStream_t stream);

hipError_t launch_expand_backbone(const uint8_t* codes, const uint8_t* meta, int64_t T, int64_t K, int n, int m,
                                  uint8_t* bb_codes, uint8_t* mask, hipStream_t stream);

hipError_t launch_moe_combine(const float* y, int64_t P, int64_t H, const int32_t* pair_index, const float* weights,
                              int64_t T, int k, float* out, uint16_t* out_bf16, hipStream_t stream);

hipError_t launch_prepare_nvfp4(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma, int n,
                                int m, float s_t, uint8_t* bb_codes, uint8_t* bb_scales, uint8_t* res_codes,
                                uint8_t* res_scales, uint8_t* mask, hipStream_t stream);

hipError_t launch_quantize_nvfp4(const uint16_t* w, int64_t O, int64_t K, int64_t ldw, float s_t, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream);

hipError_t launch_linear_nvfp4(const uint8_t* bb_codes, const uint8_t* bb_scales, const uint8_t* res_codes,
                               const uint8_t* res_scales, float s_a, const uint8_t* w_codes, const uint8_t* w_scales,
                               float s_w, int64_t T, int64_t O, int64_t K, float* y, int64_t ldy,
                               hipStream_t stream);

hipError_t launch_pack(const uint8_t* codes_rm, const uint8_t* scales_rm, int64_t R, int64_t K, int block,
                       uint8_t* codes, uint8_t* scales, hipStream_t stream);

hipError_t launch_unpack(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t K, int block,
                         uint8_t* codes_rm, uint8_t* scales_rm, hipStream_t stream);

// Plain MXFP4 products (mxgemm.hip): activation [ceil(K/128)][rows][64] against
// weight [ceil(K/128)][O][64] (grouped: one such tensor per expert).
struct MxProduct {
  const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
  int64_t rows, O, K;
};
int64_t mx_linear_workspace_bytes(int64_t T, int64_t O, int64_t K);
hipError_t launch_mx_linear(const MxProduct& m, void* y, int64_t ldy, bool bf16, void* workspace,
                            int64_t workspace_bytes, hipStream_t stream);
// O = 2 I: gate rows, then up rows
hipError_t launch_mx_linear_silu(const MxProduct& m, uint8_t* h_codes, uint8_t* h_scales, void* workspace,
                                 int64_t workspace_bytes, hipStream_t stream);
constexpr int64_t kMxMaxWorkgroups = (int64_t)1 << 24;  // fewer than 2^32 threads
bool mx_grouped_fits(int64_t P, int32_t E, int64_t O);  // O: weight rows of an expert
hipError_t launch_mx_grouped(const MxProduct& m, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                             void* y, bool bf16, hipStream_t stream);
hipError_t launch_mx_grouped_silu(const MxProduct& m, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                                  uint8_t* h_codes, uint8_t* h_scales, hipStream_t stream);

// Plain MXFP4 coding of the RMS-normed rows (prepare.hip); rms_scale may be null.
hipError_t launch_quantize_rms(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma, float eps,
                               float* rms_scale, uint8_t* codes, uint8_t* scales, hipStream_t stream);

// Routing (moe_route.hip).
struct RouteArgs {
  const void* logits;
  int dtype;  // 0 fp32, 1 bf16, 2 fp16
  int64_t T, ld;
  int32_t E, k;
  const float* bias;  // or null
  int32_t groups, top_groups;
  int sum2, sigmoid, renormalize;
  double scale;
  const int32_t* num_tokens;  // or null
  int32_t* expert;
  float* weight;
  int32_t *seg_offsets, *a_rows, *pair_index;
  int32_t* counts;  // workspace: [chunks][E]
  int32_t group_values = 0;  // set by the launch
};
int64_t moe_route_workspace_bytes(int64_t T, int32_t E);
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);

// 8-bit integer coding (int8.hip). dtype as in the ABI (0 fp32, 1 bf16, 2 fp16);
// seg (or null) bounds the rows that are written: [seg[0], seg[segments]).
hipError_t launch_quantize_int8(const void* x, int dtype, int64_t E, int64_t R, int64_t K, int64_t ldx, int8_t* codes,
                                float* scales, const int32_t* seg, int32_t segments, hipStream_t stream);
hipError_t launch_quantize_int8_rms(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma,
                                    float eps, float* rms_scale, int8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_pack_int8(const int8_t* codes_rm, int64_t E, int64_t R, int64_t K, int8_t* codes, bool unpack,
                            int8_t* out_rm, hipStream_t stream);

// Products of 8-bit codes (i8gemm.hip, i8grouped.hip): activation [ceil(K/64)][rows][64] against
// weight [ceil(K/64)][O][64] (grouped: one such tensor per expert).
struct I8Product {
  const int8_t* a_codes;
  const float* a_scales;
  const int8_t* w_codes;
  const float* w_scales;
  const float* bias;  // or null
  int64_t rows, O, K;
};
constexpr int64_t kI8MaxWorkgroups = (int64_t)1 << 22;  // fewer than 2^32 threads
bool i8_linear_fits(int64_t T, int64_t O);
hipError_t launch_i8_linear(const I8Product& p, void* y, int64_t ldy, bool bf16, hipStream_t stream);
// O = 2 I: gate rows, then up rows; the workspace holds h
int64_t i8_silu_workspace_bytes(int64_t T, int64_t I);
hipError_t launch_i8_linear_silu(const I8Product& p, int8_t* h_codes, float* h_scales, void* workspace,
                                 hipStream_t stream);
bool i8_grouped_fits(int64_t P, int32_t E, int64_t O);  // O: weight rows of an expert
hipError_t launch_i8_grouped(const I8Product& p, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                             void* y, bool bf16, hipStream_t stream);
hipError_t launch_i8_grouped_silu(const I8Product& p, const int32_t* a_rows, const int32_t* seg, int32_t E, int64_t P,
                                  int8_t* h_codes, float* h_scales, void* workspace, hipStream_t stream);

// The tile that a product runs on (kind: 0 fp32, 1 bf16, 2 gate|up; O: weight rows).
struct I8TileChoice {
  int number, count;  // of how many
  int rows, cols;     // tokens, weight rows
};
I8TileChoice i8_linear_choice(int64_t T, int64_t O, int64_t K, int kind);
I8TileChoice i8_grouped_choice(int64_t P, int32_t E, int64_t O, int64_t K, int kind);

hipError_t launch_moe_combine_bf16(const uint16_t* y, int64_t P, int64_t H, const int32_t* pair_index,
                                   const float* weights, int64_t T, int k, float* out, uint16_t* out_bf16,
                                   hipStream_t stream);

hipError_t launch_silu_mul(const float* gu, int64_t T, int64_t I, uint16_t* h, hipStream_t stream);

}  // namespace sharq

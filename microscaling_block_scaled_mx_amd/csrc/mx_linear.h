// Internal launch interface of the linear operators: the GEMM with an
// activation epilogue (mx_gemm_act.hip) and the 8-bit activation checkpoints
// with the packs that read them (mx_saved.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_kernels.h"

namespace mx {

// Dense GEMM epilogue of mx_gemm_act (beside those of mx_kernels.h).
constexpr int kEpiAct = 5;
// ... and one that the kernel's parameter type brings along.
constexpr int kEpiOwn = 6;

// C = act(A . B^T + bias) + residual for any M, N a multiple of 32 and K a
// multiple of 32 (operands padded to whole K groups); c may be null when the
// pre-activation's checkpoint is written.
struct GemmActParams : GemmParams {
  const void* residual;   // [M][ldr] of C's type, or nullptr
  int64_t ldr;
  int act;                // Act
  uint8_t* saved_codes;   // E4M3 checkpoint of the pre-activation, [M] x K=N, or nullptr
  uint8_t* saved_scales;
};
hipError_t launch_gemm_act(const GemmActParams& p, int fmt, hipStream_t stream);

// Column sums to finish: out[c] = partials [rows][cols] of column c in
// increasing order, from +0 (out nullptr: none).
struct ColumnSums {
  const float* partials;
  int64_t rows, cols;
  float* out;
};
__device__ __forceinline__ void finish_column_sum(const ColumnSums& s, int64_t c) {
  if (c >= s.cols) return;
  const float* src = s.partials + c;
  float sum = 0.0f;
#pragma unroll 32
  for (int64_t b = 0; b < s.rows; ++b) sum = sum + src[b * s.cols];
  s.out[c] = sum;
}

// Two independent products of one format and column sums to finish, in one
// launch where one kernel variant serves both products.
hipError_t launch_gemm_act_pair(const GemmActParams& p, const GemmActParams& q, const ColumnSums& sums, int fmt,
                                hipStream_t stream);

// x [R][ldx] (bf16 or binary32) -> E4M3 operand [R] x K=C, RCEIL scales.
hipError_t launch_checkpoint_save(const void* x, int x_f32, int64_t R, int64_t C, int64_t ldx, uint8_t* codes,
                                  uint8_t* scales, hipStream_t stream);
// The reverse, into y [R][ldy] (bf16 or binary32).
hipError_t launch_checkpoint_load(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t C, void* y,
                                  int y_f32, int64_t ldy, hipStream_t stream);

// v = act(saved), or x * act'(saved) where x is given (x itself without a
// checkpoint), rounded to bf16 and packed.
struct SavedPackParams {
  const uint16_t* x;            // bf16 [R][ldx] or nullptr
  int64_t ldx;
  const uint8_t* saved_codes;   // E4M3 [R] x K=C or nullptr
  const uint8_t* saved_scales;
  int64_t R, C;                 // any R, C a multiple of 32
  uint8_t* row_codes;           // [R] x K=C, or nullptr
  uint8_t* row_scales;
  uint8_t* col_codes;           // [C] x K=R (rounded up to 32), or nullptr
  uint8_t* col_scales;
  float* partials;              // [ceil(R/128)][C] or nullptr
  int act;                      // Act
};
// One pack, or two in a launch (q may be nullptr), of one format, scale mode
// and rotation.
hipError_t launch_quantize_saved(const SavedPackParams& p, const SavedPackParams* q, int fmt, int mode, int had,
                                 hipStream_t stream);

}  // namespace mx

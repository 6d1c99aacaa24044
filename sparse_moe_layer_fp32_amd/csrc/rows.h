// Host-side launchers of the steps between the permutation and the experts'
// products: rows out to the experts, rows back with weights, their gradients,
// and block quantisation (internal to libmoe.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct RowsArgs {
  int64_t tokens, rows;
  int top_k, hidden;
  const int32_t* pos;  // [tokens][top_k]; outside [0, rows): no row
  const float* w;      // [tokens][top_k], or null for ones
  const void* tok;     // [tokens][hidden]: x or dy
  const void* base;    // [tokens][hidden] or null
  void* tok_out;       // [tokens][hidden]
  const void* row;     // [rows][hidden]
  void* row_out;       // [rows][hidden]
  float* dw;           // [tokens][top_k]
  int tok_f32, row_f32;
};
// Whether the rows that a call's pairs can name go past the last-level cache.
bool rows_past_cache(int64_t tokens, int64_t rows, int top_k, int64_t row_bytes);

// row_out[pos] = tok
hipError_t launch_dispatch(const RowsArgs& p, hipStream_t stream);
// tok_out = base + sum_j w row[pos]
hipError_t launch_combine_rows(const RowsArgs& p, hipStream_t stream);
// row_out[pos] = w tok;  dw = <tok, row[pos]>  (either may be null)
hipError_t launch_combine_grad(const RowsArgs& p, hipStream_t stream);

// Codes and scales of the rows of x in blocks of 1 x 128; with pos, to the rows
// that it names.
hipError_t launch_quantize_rows(const uint16_t* x, const int32_t* pos, int64_t tokens,
                                int64_t rows, int top_k, int cols, uint8_t* codes, float* scales,
                                hipStream_t stream);
// Codes and scales of w [groups][F][K] in blocks of 128 x 128.
hipError_t launch_quantize_weight(const uint16_t* w, int groups, int F, int K, uint8_t* codes,
                                  float* scales, hipStream_t stream);

}  // namespace moe

// Host-side launchers of the linear and grouped products, their gradients and
// the SwiGLU activation (internal to libmoe.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Which of the three products of a (grouped) linear map a launch forms.  With
// F out features, K in features, W [F][K] (one per group):
enum ProductOp : int {
  kForward = 0,    // y[r][f]  = sum_k x[src(r)][k] W[f][k]
  kInputGrad = 1,  // dx[r][k] = sum_f dy[r][f] W[f][k]
  kWeightGrad = 2  // dW[f][k] = sum_r dy[r][f] x[src(r)][k],  db[f] = sum_r dy[r][f]
};

// Arguments of one product.  Rows [offsets[g], offsets[g+1]) belong to group
// g; a null `offsets` means one group of all P rows.  Offsets are clamped to
// [0, P] on the device.
struct ProductArgs {
  const uint16_t* a;       // x (forward) or dy (gradients)
  const uint16_t* b;       // W (forward, input gradient) or x (weight gradient)
  const int32_t* offsets;  // [G+1] or null
  const int32_t* src;      // x's row of each row, times row_div; null: the row itself
  int row_div;
  int64_t x_rows;          // rows of x behind `src`; a row outside [0, x_rows) reads as zeros
  int64_t P;
  int G, K, F;
  // epilogue: v = sum + bias; z = v; y = act(v) + residual, or y += v
  const float* bias;         // [G][F] or null (forward)
  const uint16_t* residual;  // [P][F] or null (forward)
  uint16_t* z;               // [P][F] or null (forward)
  void* y;                   // bf16, or fp32 when y_f32 (weight gradient: null for db alone)
  int y_f32;
  int act;                   // MOE_ACT_*
  int accumulate;            // weight gradient: add to y and db
  int stream;                // weight gradient: y is larger than the last-level cache
  float* db;                 // [G][F] or null (weight gradient)
  // Contraction cut into `splits` ranges whose fp32 sums meet in `part`
  // (kForward, kInputGrad: [splits][P][columns]; kWeightGrad: [splits][G F][K],
  // and part_db [splits][G F]).
  int splits;
  float* part;
  float* part_db;
  // set by the launcher
  int cus;
  int whole, slices;  // Big tiles left whole (-1: all), slices of the rows of the others
};

// A row tile of a ragged product of codes.
struct RowTile {
  int32_t row0, rows, g;
  int32_t first, tiles;  // of its group: the first tile's index, and their number
  int32_t pad[3];
};

// Arguments of one product of e4m3 codes: a and b as rows of K 16-bit pairs of
// codes, and their scales: a's of a step and row at [row of x][step] (codes_run:
// a_scale[step a_scale_step + row of y]), b's at [G][F / 128][step], rounded up.
struct CodesArgs : ProductArgs {
  const float* a_scale;
  const float* b_scale;
  int64_t a_scale_step;
  const RowTile* tiles;  // codes_run with groups: row tiles, and their number
  const int32_t* num_tiles;
  const uint32_t* sources;  // codes_run with src: byte offsets of the rows of y in x
};

// How a product is run: the tile shape and the number of contraction ranges.
struct ProductPlan {
  int shape;
  int splits;
  int cus;     // compute units of the device
  int slices;  // Big: slices of rows that the last round's tiles are cut into
  float us;    // its estimated time (0 for a forward product of few rows)
};
ProductPlan product_plan(int op, int64_t P, int G, int K, int F, int cus);
// Plans of kInputGrad and kWeightGrad in one launch; false when two launches,
// each by its own plan, are expected to be faster.
bool pair_plan(int64_t P, int G, int K, int F, int cus, ProductPlan* x, ProductPlan* w);
// The forward product of codes, with K in pairs of them; exact: fp32 results.
ProductPlan product_fp8_plan(int64_t P, int G, int K, int F, int cus, bool exact);
// What a plan's launch needs in the workspace before its partial sums: for large
// tiles the row tiles and x's scales by step.
size_t codes_prepare_bytes(int64_t P, int G, int K, bool grouped, const ProductPlan& plan);
// `area`: that many bytes.
hipError_t launch_product_fp8(const CodesArgs& p, const ProductPlan& plan, bool exact, void* area,
                              hipStream_t stream);
// Bytes of `part` (with part_db behind it) for that plan; 0 when splits == 1.
size_t product_part_bytes(int op, int64_t P, int G, int K, int F, const ProductPlan& plan);
hipError_t launch_product(int op, const ProductArgs& p, const ProductPlan& plan, hipStream_t stream);
// kInputGrad of x and kWeightGrad of w in one launch, by the plans of pair_plan.
hipError_t launch_pair(const ProductArgs& x, const ProductPlan& px, const ProductArgs& w,
                       const ProductPlan& pw, hipStream_t stream);

// src[r] = row_ids[r] / row_div, or -1 where that is outside [0, x_rows); and
// kSourcePad further entries of -1.
constexpr int kSourcePad = 64;
hipError_t launch_source_rows(const int32_t* row_ids, int row_div, int64_t x_rows, int64_t P,
                              int32_t* src, hipStream_t stream);

// dz = dy act'(z) in bf16, and db = sum over rows of the unrounded dz (db may
// be null).  part: act_grad_part_bytes().
size_t act_grad_part_bytes(int64_t T, int F);
hipError_t launch_act_grad(const uint16_t* dy, const uint16_t* z, int act, int64_t T, int F,
                           uint16_t* dz, float* db, int accumulate, float* part,
                           hipStream_t stream);

// SwiGLU (swiglu.hip); ld is the row stride of gate, up, dgate and dup.
hipError_t launch_swiglu(const uint16_t* gate, const uint16_t* up, uint16_t* h, int64_t rows,
                         int inter, int64_t ld, float limit, hipStream_t stream);
hipError_t launch_swiglu_grad(const uint16_t* dh, const uint16_t* gate, const uint16_t* up,
                              uint16_t* dgate, uint16_t* dup, uint16_t* h, int64_t rows, int inter,
                              int64_t ld, float limit, hipStream_t stream);

}  // namespace moe

// The forward product of e4m3 codes with an fp32 scale for each block, of 1 x 128
// in x and of 128 x 128 in W:
//
//   y[r][f] = sum_b xs[r][b] ws[f / 128][b] sum_{k in block b} x[r][k] W[f][k]
//
// on the tiles of the bf16 products (product_tile.h), whose steps of 128 bytes
// are one block of codes each.  For bf16 results the tiles multiply codes as they
// are, for fp32 results codes widened to bf16 (codes_tile.h).

#include "codes_tile.h"
#include "product_blocks.h"

namespace moe {

namespace {

// Few rows: as product_thin (products.hip), W streamed straight into the
// fragments, its codes and x's widened to bf16 on the way: the stream bounds it,
// not the products, and their sums are exact for both types of y.  A wave takes
// blocks of 128 codes in turn, 32 of each W row a lane; the four products of a
// block start from zero and are added times its scales.
constexpr int kThinWaves = 8;
constexpr int kThinAhead = 4;  // blocks that a wave requests before it multiplies

template <int COLS>
__global__ __launch_bounds__(64 * kThinWaves) void product_thin_fp8(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[kThinWaves * 256];
  Unit un;
  if (!find_unit<kForward, kThinRows, COLS, 64 * kThinWaves>(p, blockIdx.x,
                                                             reinterpret_cast<int*>(sums), &un))
    return;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int K = p.K, blocks = (K + 63) / 64;  // pairs of codes
  const int col = un.col0 + r;
  const bool live_col = r < COLS && col < p.F;
  const uint16_t* w = p.b + (static_cast<int64_t>(un.g) * p.F + min(col, p.F - 1)) * K;
  const int64_t s = r < un.rows ? source_row(p, un.row0 + r) : -1;
  const uint16_t* x = p.a + max(s, int64_t(0)) * K;
  const int fblocks = (p.F + 127) / 128;
  const float* ws = p.b_scale + (static_cast<int64_t>(un.g) * fblocks + un.col0 / 128) * blocks;
  const float* xs = p.a_scale + max(s, int64_t(0)) * p.a_scale_row;
  f32x4 acc{};
  for (int c0 = wid; c0 < blocks; c0 += kThinWaves * kThinAhead) {
    u32x4 wf[kThinAhead][2], xf[kThinAhead][2];
    float scale[kThinAhead];
#pragma unroll
    for (int i = 0; i < kThinAhead; ++i) {
      const int b = c0 + kThinWaves * i;
      scale[i] = 0.0f;
      if (b < blocks && s >= 0) scale[i] = ws[b] * xs[b];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 64 * b + 16 * q + 8 * h;
        wf[i][h] = xf[i][h] = u32x4{};
        if (k < K && live_col) wf[i][h] = *reinterpret_cast<const u32x4*>(w + k);
        if (k < K && s >= 0) xf[i][h] = *reinterpret_cast<const u32x4*>(x + k);
      }
    }
#pragma unroll
    for (int i = 0; i < kThinAhead; ++i) {
      f32x4 t{};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 2; ++d)
          t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              e4m3x8_to_bf16(wf[i][h][2 * d], wf[i][h][2 * d + 1]),
              e4m3x8_to_bf16(xf[i][h][2 * d], xf[i][h][2 * d + 1]), t, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(scale[i], t[j], acc[j]);
    }
  }
  // lane: row lane % 16, columns 4 (lane / 16) .. + 3
  *reinterpret_cast<f32x4*>(sums + wid * 256 + r * 16 + 4 * q) = acc;
  __syncthreads();
  const int row = threadIdx.x / 2, c = threadIdx.x % 2 * 8;
  if (row >= un.rows || c >= COLS || un.col0 + c >= p.F) return;
  F8 v = load8(sums + row * 16 + c);
#pragma unroll
  for (int i = 1; i < kThinWaves; ++i) {
    const F8 o = load8(sums + i * 256 + row * 16 + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) v.v[j] += o.v[j];
  }
  finish_one(p, v, p.bias ? p.bias + static_cast<int64_t>(un.g) * p.F : nullptr, un.row0 + row,
             un.col0 + c, p.F);
}

// A block takes 64 rows and 32 steps through LDS, reading rows and writing steps.
constexpr int kTurnRows = 64, kTurnSteps = 32;

__global__ __launch_bounds__(256) void scales_by_step_kernel(
    const float* __restrict__ scales, const int32_t* __restrict__ row_ids, int row_div,
    int64_t x_rows, int64_t P, int steps, int64_t pitch, float* __restrict__ by_step) {
  __shared__ float tile[kTurnSteps][kTurnRows + 1];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kTurnRows;
  const int s0 = blockIdx.y * kTurnSteps;
  const int s = threadIdx.x % kTurnSteps;
#pragma unroll
  for (int i = threadIdx.x / kTurnSteps; i < kTurnRows; i += 256 / kTurnSteps) {
    int64_t src = r0 + i < P ? r0 + i : -1;
    if (src >= 0 && row_ids) {
      const int id = row_ids[src];
      src = id >= 0 && id / row_div < x_rows ? id / row_div : -1;
    }
    tile[s][i] = src >= 0 && s0 + s < steps ? scales[src * steps + s0 + s] : 0.0f;
  }
  __syncthreads();
  const int r = threadIdx.x % kTurnRows;
#pragma unroll
  for (int i = threadIdx.x / kTurnRows; i < kTurnSteps; i += 256 / kTurnRows)
    if (s0 + i < steps) by_step[(s0 + i) * pitch + r0 + r] = tile[i][r];
}

template <int COLS>
hipError_t launch_thin_fp8(const ProductArgs& p, hipStream_t stream) {
  const int64_t units =
      tile_count(kForward, p.P, p.G, p.K, p.F, p.offsets != nullptr, {kThinRows, COLS});
  if (units <= 0) return hipSuccess;
  product_thin_fp8<COLS><<<block_count(units, 1), 64 * kThinWaves, 0, stream>>>(p);
  return hipGetLastError();
}

template <class T>
__global__ __launch_bounds__(T::THREADS, 2) void codes_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
  Unit un;
  if (!find_unit<kForward, T::BM, T::BN, T::THREADS>(p, blockIdx.x, reinterpret_cast<int*>(smem),
                                                     &un))
    return;
  if constexpr (T::BM == 256) {
    // fewer rows, the remainder of a group or a cut tile: the same columns with
    // less of x to load and to multiply
    using Three = CodesThree<T::KIND>;
    using Half = CodesHalf<T::KIND>;
    using Flat = CodesFlat<T::KIND>;
    static_assert(Flat::LDS <= T::LDS && Half::LDS <= T::LDS && Three::LDS <= T::LDS &&
                      Flat::THREADS == T::THREADS && Half::THREADS == T::THREADS &&
                      Three::THREADS == T::THREADS,
                  "the same LDS and waves");
    if (un.rows <= 64) return codes_tile<Flat>(p, smem, un);
    if (un.rows <= 128) return codes_tile<Half>(p, smem, un);
    if (un.rows <= 192) return codes_tile<Three>(p, smem, un);
  }
  codes_tile<T>(p, smem, un);
}

template <class T>
hipError_t launch_codes(ProductArgs p, hipStream_t stream) {
  const unsigned grid = grid_of<kForward, T>(&p);
  if (grid == 0) return hipSuccess;
  codes_kernel<T><<<grid, T::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

template <int Q>
hipError_t launch_shape(const ProductArgs& p, int shape, hipStream_t stream) {
  switch (shape) {
    case kShapeBig:
      if constexpr (Q == kNative) return launch_codes<CodesBig<Q>>(p, stream);
      return hipErrorInvalidValue;
    case kShapeHalf: return launch_codes<CodesHalf<Q>>(p, stream);
    default: return launch_codes<CodesSmall<Q>>(p, stream);
  }
}

}  // namespace

bool wants_scales_by_step(const ProductPlan& plan) { return plan.shape == kShapeBig; }

hipError_t launch_scales_by_step(const float* scales, const int32_t* row_ids, int row_div,
                                 int64_t x_rows, int64_t P, int steps, float* by_step,
                                 hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((P + kTurnRows - 1) / kTurnRows),
                  static_cast<unsigned>((steps + kTurnSteps - 1) / kTurnSteps));
  scales_by_step_kernel<<<grid, 256, 0, stream>>>(scales, row_ids, row_div, x_rows, P, steps,
                                                  scale_pitch(P), by_step);
  return hipGetLastError();
}

hipError_t launch_product_fp8(const ProductArgs& p, const ProductPlan& plan, bool exact,
                              hipStream_t stream) {
  ProductArgs q = p;
  q.splits = plan.splits;
  q.cus = plan.cus;
  q.slices = plan.slices;
  if (plan.shape == kShapeThin8) return launch_thin_fp8<8>(q, stream);
  if (plan.shape == kShapeThin16) return launch_thin_fp8<16>(q, stream);
  const hipError_t e = exact ? launch_shape<kExact>(q, plan.shape, stream)
                             : launch_shape<kNative>(q, plan.shape, stream);
  return e != hipSuccess || q.splits == 1 ? e : launch_join<kForward>(q, stream);
}

}  // namespace moe

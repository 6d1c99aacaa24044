// The forward product of e4m3 codes with an fp32 scale for each block, of 1 x 128
// in x and of 128 x 128 in W:
//
//   y[r][f] = sum_b xs[r][b] ws[f / 128][b] sum_{k in block b} x[r][k] W[f][k]
//
// on the tiles of the bf16 products (product_tile.h), whose steps of 128 bytes
// are one block of codes each.  For bf16 results the tiles multiply codes as they
// are, for fp32 results codes widened to bf16 (codes_tile.h).

#include "product_blocks.h"

#include "codes_run.h"

namespace moe {

namespace {

// Few rows: as product_thin (products.hip), W streamed straight into the
// fragments, its codes and x's widened to bf16 on the way: the stream bounds it,
// not the products, and their sums are exact for both types of y.  A wave takes
// blocks of 128 codes in turn, 32 of each W row a lane; the four products of a
// block start from zero and are added times its scales.  One row, 4096 -> 1280: 5.8
// us (latency: 80 blocks, one turn of loads), 11264 -> 4096: 10.2, 4.5 TB/s.
constexpr int kThinWaves = 8;
constexpr int kThinAhead = 4;  // blocks that a wave requests before it multiplies

template <int COLS>
__global__ __launch_bounds__(64 * kThinWaves) void product_thin_fp8(CodesArgs p) {
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
  const float* xs = p.a_scale + max(s, int64_t(0)) * blocks;
  int none = 0;
  asm volatile("" : "+v"(none));
  f32x4 acc{};
  for (int c0 = wid; c0 < blocks; c0 += kThinWaves * kThinAhead) {
    u32x4 wf[kThinAhead][2], xf[kThinAhead][2];
    float wscale[kThinAhead], xscale[kThinAhead];
#pragma unroll
    for (int i = 0; i < kThinAhead; ++i) {
      const int b = c0 + kThinWaves * i;
      // (by each lane: a scalar load would be waited for before the next loads)
      wscale[i] = ws[min(b, blocks - 1) + none];
      xscale[i] = 0.0f;
      if (s >= 0) xscale[i] = xs[min(b, blocks - 1)];
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
      // (0 for a row without a source, times W's scale: NaN where that is not finite)
      const float scale = c0 + kThinWaves * i < blocks ? wscale[i] * xscale[i] : 0.0f;
      f32x4 t{};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 2; ++d)
          t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              e4m3x8_to_bf16(wf[i][h][2 * d], wf[i][h][2 * d + 1]),
              e4m3x8_to_bf16(xf[i][h][2 * d], xf[i][h][2 * d + 1]), t, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(scale, t[j], acc[j]);
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

// What the large tiles need: x's scales by steps of the rows of y (0 where x has
// no such row), a block turning 64 rows and 32 steps through LDS; the rows'
// sources in x; and, of ragged groups, the row tiles, in one block more.
constexpr int kTurnRows = 64, kTurnSteps = 32, kPrepareThreads = 256;

int64_t scale_pitch(int64_t P) { return (P + kTurnRows - 1) / kTurnRows * kTurnRows; }

__device__ void list_row_tiles(const int32_t* __restrict__ offsets, int64_t P, int G,
                               RowTile* __restrict__ tiles, int most,
                               int32_t* __restrict__ num_tiles, int* sh) {
  constexpr int BM = CodesRun::BM;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int c = (G + kPrepareThreads - 1) / kPrepareThreads;
  auto rows_of = [&](int g, int* begin) {
    *begin = clamp_row(offsets[g], P);
    return max(0, clamp_row(offsets[g + 1], P) - *begin);
  };
  int mine = 0, b;
  for (int g = tid * c; g < min(tid * c + c, G); ++g) mine += (rows_of(g, &b) + BM - 1) / BM;
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 63) sh[wid] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kPrepareThreads / 64; ++w) {
    if (w < wid) at += sh[w];
    total += sh[w];
  }
  if (tid == 0) *num_tiles = min(total, most);
  for (int g = tid * c; g < min(tid * c + c, G); ++g) {
    const int rows = rows_of(g, &b);
    // (offsets that do not ascend could make more tiles than there is room for)
    const int n = min((rows + BM - 1) / BM, max(0, most - at));
    for (int i = 0; i < n; ++i)
      tiles[at + i] = {b + i * BM, min(BM, rows - i * BM), g, at, n, {}};
    at += n;
  }
}

template <bool GATHER>
__global__ __launch_bounds__(kPrepareThreads) void codes_prepare_kernel(
    const float* __restrict__ scales, const int32_t* __restrict__ row_ids, int row_div,
    int64_t x_rows, int64_t P, int steps, int64_t pitch, float* __restrict__ by_step,
    const int32_t* __restrict__ offsets, int G, RowTile* __restrict__ tiles, int most_tiles,
    int32_t* __restrict__ num_tiles, uint32_t* __restrict__ sources, uint32_t x_pitch) {
  __shared__ float tile[kTurnSteps][kTurnRows + 1];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kTurnRows;
  if (r0 >= P) {  // the block more
    if (blockIdx.y == 0)
      list_row_tiles(offsets, P, G, tiles, most_tiles, num_tiles, reinterpret_cast<int*>(tile));
    return;
  }
  const int s0 = blockIdx.y * kTurnSteps;
  const int s = threadIdx.x % kTurnSteps;
  // (loads without branches between them, so that they are under way together)
  constexpr int STEP = kPrepareThreads / kTurnSteps, N = kTurnRows / STEP;
  const int i0 = threadIdx.x / kTurnSteps;
  int64_t src[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int64_t r = r0 + i0 + n * STEP;
    src[n] = GATHER ? row_ids[min(r, P - 1)] : r;
    if (r >= P) src[n] = -1;
  }
  if (GATHER)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int id = static_cast<int>(src[n]);
      src[n] = id >= 0 && id / row_div < x_rows ? id / row_div : -1;
      if (s == 0 && blockIdx.y == 0)
        sources[r0 + i0 + n * STEP] = src[n] >= 0 ? static_cast<uint32_t>(src[n]) * x_pitch : kFar;
    }
  float v[N] = {};
  if (!GATHER || x_rows > 0)
#pragma unroll
    for (int n = 0; n < N; ++n)
      v[n] = scales[max(src[n], int64_t(0)) * steps + min(s0 + s, steps - 1)];
#pragma unroll
  for (int n = 0; n < N; ++n)
    tile[s][i0 + n * STEP] = src[n] >= 0 && s0 + s < steps ? v[n] : 0.0f;
  __syncthreads();
  const int r = threadIdx.x % kTurnRows;
#pragma unroll
  for (int i = threadIdx.x / kTurnRows; i < kTurnSteps; i += kPrepareThreads / kTurnRows)
    if (s0 + i < steps) by_step[(s0 + i) * pitch + r0 + r] = tile[i][r];
}

// The area: the number of row tiles, the tiles, the rows' sources (a tile's more
// than there are rows), the scales.
struct CodesArea {
  size_t tiles, sources, scales, total;
  int most_tiles;
};
CodesArea codes_area(int64_t P, int G, int K, bool grouped) {
  const int64_t tiles = grouped ? P / CodesRun::BM + std::min<int64_t>(G, P) : 0;
  CodesArea a;
  a.tiles = 64;
  a.most_tiles = static_cast<int>(tiles);
  a.sources = (a.tiles + tiles * sizeof(RowTile) + 255) / 256 * 256;
  a.scales = a.sources + (grouped ? (scale_pitch(P) + CodesRun::BM) * 4 : 0);
  a.total = a.scales + static_cast<size_t>(scale_pitch(P)) * ((K + 63) / 64) * 4;
  return a;
}

hipError_t launch_run(CodesArgs p, char* area, hipStream_t stream) {
  const CodesArea a = codes_area(p.P, p.G, p.K, p.offsets != nullptr);
  const int steps = (p.K + 63) / 64;
  const int64_t pitch = scale_pitch(p.P);
  float* const by_step = reinterpret_cast<float*>(area + a.scales);
  RowTile* const tiles = p.offsets ? reinterpret_cast<RowTile*>(area + a.tiles) : nullptr;
  int32_t* const num_tiles = reinterpret_cast<int32_t*>(area);
  uint32_t* const sources = reinterpret_cast<uint32_t*>(area + a.sources);
  const dim3 grid(static_cast<unsigned>(pitch / kTurnRows + (tiles ? 1 : 0)),
                  static_cast<unsigned>((steps + kTurnSteps - 1) / kTurnSteps));
  const auto prepare = p.src ? codes_prepare_kernel<true> : codes_prepare_kernel<false>;
  prepare<<<grid, kPrepareThreads, 0, stream>>>(
      p.a_scale, p.src, p.row_div, p.x_rows, p.P, steps, pitch, by_step, p.offsets, p.G, tiles,
      a.most_tiles, num_tiles, sources, static_cast<uint32_t>(p.K) * 2);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  p.a_scale = by_step;
  p.a_scale_step = pitch;
  p.tiles = tiles;
  p.num_tiles = num_tiles;
  p.sources = sources;
  // a block of each CU, as many on every XCD, walks the grid of one block per tile
  const unsigned all = grid_of<kForward, CodesRun>(&p);
  const unsigned cus = static_cast<unsigned>(std::max(p.cus / kNumXcd * kNumXcd, kNumXcd));
  const unsigned blocks = std::min(all, cus);
  const bool act = p.act != MOE_ACT_NONE;
  if (p.src)  // (a gathered product has no activation)
    codes_run_kernel<true, false><<<blocks, CodesRun::THREADS, 0, stream>>>(p);
  else if (act)
    codes_run_kernel<false, true><<<blocks, CodesRun::THREADS, 0, stream>>>(p);
  else
    codes_run_kernel<false, false><<<blocks, CodesRun::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

template <int COLS>
hipError_t launch_thin_fp8(const CodesArgs& p, hipStream_t stream) {
  const int64_t units =
      tile_count(kForward, p.P, p.G, p.K, p.F, p.offsets != nullptr, {kThinRows, COLS});
  if (units <= 0) return hipSuccess;
  product_thin_fp8<COLS><<<block_count(units, 1), 64 * kThinWaves, 0, stream>>>(p);
  return hipGetLastError();
}

template <class T>
__global__ __launch_bounds__(T::THREADS, 2) void codes_kernel(CodesArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
  Unit un;
  if (find_unit<kForward, T::BM, T::BN, T::THREADS>(p, blockIdx.x, reinterpret_cast<int*>(smem),
                                                    &un))
    codes_tile<T>(p, smem, un);
}

template <class T>
hipError_t launch_codes(CodesArgs p, hipStream_t stream) {
  const unsigned grid = grid_of<kForward, T>(&p);
  if (grid == 0) return hipSuccess;
  codes_kernel<T><<<grid, T::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

template <int Q>
hipError_t launch_shape(const CodesArgs& p, int shape, hipStream_t stream) {
  return shape == kShapeHalf ? launch_codes<CodesHalf<Q>>(p, stream)
                             : launch_codes<CodesSmall<Q>>(p, stream);
}

}  // namespace

size_t codes_prepare_bytes(int64_t P, int G, int K, bool grouped, const ProductPlan& plan) {
  return plan.shape == kShapeBig ? codes_area(P, G, K, grouped).total : 0;
}

hipError_t launch_product_fp8(const CodesArgs& p, const ProductPlan& plan, bool exact, void* area,
                              hipStream_t stream) {
  CodesArgs q = p;
  q.splits = plan.splits;
  q.cus = plan.cus;
  q.slices = plan.slices;
  if (plan.shape == kShapeThin8) return launch_thin_fp8<8>(q, stream);
  if (plan.shape == kShapeThin16) return launch_thin_fp8<16>(q, stream);
  if (plan.shape == kShapeBig) return launch_run(q, static_cast<char*>(area), stream);
  const hipError_t e = exact ? launch_shape<kExact>(q, plan.shape, stream)
                             : launch_shape<kNative>(q, plan.shape, stream);
  return e != hipSuccess || q.splits == 1 ? e : launch_join<kForward>(q, stream);
}

}  // namespace moe

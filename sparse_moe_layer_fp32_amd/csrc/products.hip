// Linear and grouped products on gfx950 matrix cores: y = x W^T with bias,
// activation and residual, and the gradients dx = dy W and dW = dy^T x, for
// one group of rows or for one group per expert with ragged sizes.  The tile
// itself (mainloop and epilogue) is in product_tile.h, each block's share of
// the work in product_blocks.h, the gradients' launches in product_grads.hip
// and product_pairs.hip; this file holds the forward product, the choice of
// tile shapes and the elementwise kernels.

#include "product_blocks.h"

namespace moe {

namespace {

// Few rows (a token, or some): the product streams W once and is bound by
// that stream and by latency, so nothing goes through LDS on the way.  A block
// takes COLS W rows; its eight waves take 64 contraction values in turn (a
// 128-byte line of each W row, two fragments of v_mfma_f32_16x16x32_bf16 at 16
// and 8 values a lane), straight from memory into the fragments; the waves'
// sums meet in LDS in wave order.  One launch, no split and join.
//
// A CU draws about 25 GB/s, so a narrow output needs more blocks than it has
// 16-row pieces: with 8 rows a block half the lanes idle but 1 x 4096 -> 1280
// takes 6.3 us instead of 7.6, while 1 x 4096 -> 4096, whose 256 pieces of 16
// fill the GPU, takes 9.6 instead of 8.0.  64-byte pieces of W, or the
// non-temporal hint, cost 8% more (lines fetched twice).
constexpr int kThinWaves = 8;
constexpr int kThinAhead = 4;  // lines of each row that a wave requests before it multiplies

template <int COLS>
__global__ __launch_bounds__(64 * kThinWaves) void product_thin(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[kThinWaves * 256];
  Unit un;
  if (!find_unit<kForward, kThinRows, COLS, 64 * kThinWaves>(p, blockIdx.x, reinterpret_cast<int*>(sums),
                                                       &un))
    return;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int K = p.K, chunks = (K + 63) / 64;
  const int col = un.col0 + r;
  const bool live_col = r < COLS && col < p.F;
  const uint16_t* w = p.b + (static_cast<int64_t>(un.g) * p.F + min(col, p.F - 1)) * K;
  const int64_t s = r < un.rows ? source_row(p, un.row0 + r) : -1;
  const uint16_t* x = p.a + max(s, int64_t(0)) * K;
  f32x4 acc{};
  for (int c0 = wid; c0 < chunks; c0 += kThinWaves * kThinAhead) {
    u32x4 wf[kThinAhead][2], xf[kThinAhead][2];
#pragma unroll
    for (int i = 0; i < kThinAhead; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 64 * (c0 + kThinWaves * i) + 16 * q + 8 * h;
        wf[i][h] = xf[i][h] = u32x4{};
        if (k < K && live_col) wf[i][h] = *reinterpret_cast<const u32x4*>(w + k);
        if (k < K && s >= 0) xf[i][h] = *reinterpret_cast<const u32x4*>(x + k);
      }
#pragma unroll
    for (int i = 0; i < kThinAhead; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[i][h]),
                                                      __builtin_bit_cast(bf16x8, xf[i][h]), acc, 0,
                                                      0, 0);
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

__global__ __launch_bounds__(256) void source_rows_kernel(const int32_t* __restrict__ row_ids,
                                                          int row_div, int64_t x_rows, int64_t P,
                                                          int32_t* __restrict__ src) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= P + kSourcePad) return;
  int s = -1;
  if (i < P) {
    const int id = row_ids[i];
    if (id >= 0 && id / row_div < x_rows) s = id / row_div;
  }
  src[i] = s;
}

// dz = dy act'(z) and the column sums of each strip of rows: a block takes a
// strip of 64 x 8 columns, its waves rows in turn, a thread eight columns of
// kStripAhead rows at a time, whose loads are under way together; the waves'
// sums meet in LDS.  A single strip's sums are db itself.
//
// Bound: HBM, 6 bytes an element, and latency below some hundred blocks, where
// more waves with fewer rows each help (GELU and db, both kernels, with 4, 8 and
// 16 waves a block: 64 x 512 15.4, 9.1, 7.8 us; 1024 x 1024 20.6, 13.0, 11.4;
// 4096 x 2048, 256 blocks, 25.6, 20.2, 18.5; 4096 x 4096, 512 blocks, 29.9, 27.9,
// 29.9; 8192 x 4096 51.9, 48.9, 53.2; 4096 x 11264 63.5, 59.6, 68.3; 65536 x 1280
// 114, 108, 120).  Of four waves with one row each under way, 8192 x 4096 takes
// 45.6, but 16384 x 4096 90.1 (here 85.4) and 4096 x 11264 62.4 (60.2).
constexpr int kStripAhead = 4, kStripCols = 64 * 8, kStripMany = 512;
int strip_rows(int64_t T) { return 64 * static_cast<int>((T + 65535) / 65536); }

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void act_grad_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, int act, int64_t T, int F,
    uint16_t* __restrict__ dz, float* __restrict__ part, int strip, int accumulate) {
  __shared__ __attribute__((aligned(16))) float sums[WAVES - 1][kStripCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * kStripCols + lane * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * strip;
  const int64_t r1 = min<int64_t>(T, r0 + strip);
  F8 sum{};
  if (c < F) {
    for (int64_t r = r0 + wave; r < r1; r += WAVES * kStripAhead) {
      u32x4 d4[kStripAhead], z4[kStripAhead];
#pragma unroll
      for (int i = 0; i < kStripAhead; ++i) {
        const int64_t at = min(r + i * WAVES, r1 - 1) * F + c;
        d4[i] = *reinterpret_cast<const u32x4*>(dy + at);
        z4[i] = *reinterpret_cast<const u32x4*>(z + at);
      }
#pragma unroll
      for (int i = 0; i < kStripAhead; ++i) {
        if (r + i * WAVES >= r1) break;
        F8 d = unpack8(d4[i]);
        const F8 v = unpack8(z4[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          d.v[q] *= act_slope(v.v[q], act);
          sum.v[q] += d.v[q];
        }
        store8(dz + (r + i * WAVES) * F + c, d);
      }
    }
  }
  if (!part) return;
  if (wave > 0) store8(&sums[wave - 1][lane * 8], sum);
  __syncthreads();
  if (wave > 0 || c >= F) return;
#pragma unroll
  for (int w = 0; w < WAVES - 1; ++w) {
    const F8 o = load8(&sums[w][lane * 8]);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum.v[q] += o.v[q];
  }
  put_grad8<false>(part + static_cast<int64_t>(blockIdx.y) * F + c, sum, accumulate);
}

// The strips' sums, in order: a block takes 64 columns, wave w every fourth strip.
__global__ __launch_bounds__(256) void strip_sum_kernel(const float* __restrict__ part, int strips,
                                                        int F, float* __restrict__ db,
                                                        int accumulate) {
  __shared__ float sums[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (c < F) {
#pragma unroll 16
    for (int s = wave; s < strips; s += 4) v += part[static_cast<int64_t>(s) * F + c];
  }
  sums[wave][lane] = v;
  __syncthreads();
  if (wave > 0 || c >= F) return;
  v = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
  db[c] = accumulate ? db[c] + v : v;
}

template <int COLS>
hipError_t launch_thin(const ProductArgs& p, hipStream_t stream) {
  const int64_t units =
      tile_count(kForward, p.P, p.G, p.K, p.F, p.offsets != nullptr, {kThinRows, COLS});
  if (units <= 0) return hipSuccess;
  const unsigned grid = block_count(units, 1);
  product_thin<COLS><<<grid, 64 * kThinWaves, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_forward(const ProductArgs& p, int shape, hipStream_t stream) {
  if (shape == kShapeThin8) return launch_thin<8>(p, stream);
  if (shape == kShapeThin16) return launch_thin<16>(p, stream);
  return launch_op<kForward>(p, shape, stream);
}

// Estimated microseconds of each shape: rounds of the GPU's tile slots times
// contraction steps of 64.  A round whose tiles leave the second slot of the
// CUs empty takes `partly` per step, more as more CUs work, else `full`.  A
// split adds the join and its traffic.  Fitted to the times of 648 products
// (1 to 32768 rows, 64 to 11264 features, all three kinds), each measured in
// every shape and split: the choice made by these figures is 2% slower than
// the best measured, on the mean, and 46% at worst.
struct ShapeCost {
  int per_cu;  // tiles resident on a CU
  float full, partly, fixed;
};
constexpr ShapeCost kCosts[] = {{1, 1.66f, 0.83f, 9.5f},   // Big
                                {1, 0.98f, 0.49f, 6.2f},   // Half
                                {2, 2.09f, 0.58f, 5.9f},   // Duo
                                {2, 0.46f, 0.14f, 2.1f}};  // Small
constexpr ShapeCost kFlatCost = {1, 0.62f, 0.42f, 5.0f};
constexpr float kFilling = 0.93f;  // partly grows by this share up to one tile on every CU
// Both gradients in one launch (383 backward passes, 64 to 16384 rows, 2e9 to
// 6e11 operations, in each of ten pairs of shapes and apart: 2% slower than
// the best measured on the mean; always apart would be 14% slower).  kShared
// came later, from about 150 passes of up to 113000 rows.
constexpr float kSecondLaunch = 6.0f, kMixed = 1.08f, kLeftOver = 0.6f, kLongest = 0.85f,
                kShared = 0.3f;
constexpr float kJoin = 2.4f, kJoinBytesPerUs = 7.65e6f;
constexpr int kRangeSteps = 16;
constexpr float kManyJoin = 2.0f;    // more in product_join_many
constexpr float kRaggedJoin = 2.5f;  // more where each thread looks its group up

namespace {

// A product's sizes as the estimates see them.
struct Sizes {
  int64_t rows, cols, steps;  // of the output, and contraction steps of 64
  bool ragged;
};

Sizes sizes_of(int op, int64_t P, int G, int K, int F) {
  const int64_t L = op == kForward ? K : op == kInputGrad ? F : (P + G - 1) / G;
  return {op == kWeightGrad ? static_cast<int64_t>(G) * F : P, op == kForward ? F : K,
          std::max<int64_t>(1, (L + 63) / 64), G > 1};
}

// Tiles as they will be, about: a group with rows has half a tile more (Big,
// whose launches give remainders smaller tiles: a quarter).
int64_t tiles_about(int op, int64_t P, int G, int K, int F, int shape) {
  const ShapeSize s = kShapeSizes[shape];
  int64_t n = tile_count(op, P, G, K, F, false, s);
  if (op != kWeightGrad && G > 1)
    n += (std::min<int64_t>(G, P) + 1) / (shape == kShapeBig ? 4 : 2) *
         (((op == kForward ? F : K) + s.bn - 1) / s.bn);
  return n;
}

float partly_us(const ShapeCost& c, float steps, float taken) {
  return steps * c.partly * (1.0f + kFilling * std::min(taken, 1.0f)) + c.fixed;
}

// Slices of rows that the tiles of a Big launch's last round are cut into:
// tiles that would leave half of the GPU idle are halved or quartered (8192 x
// 4096 -> 11264, 5.5 rounds: 606 us instead of 622).
int last_round_slices(int64_t units, int cus) {
  const int64_t last = units % cus;
  return last == 0 || last * 2 > cus ? 1 : last * 4 > cus ? 2 : 4;
}

const ShapeCost& cost_of(int shape, int slices) {
  return slices == 4 ? kFlatCost : kCosts[slices == 2 ? kShapeHalf : shape];
}

}  // namespace

namespace {

// The estimate for `tiles` tiles of a shape in `splits` contraction ranges.
float product_us(const Sizes& z, int64_t tiles, int shape, int splits, int slices, int cus) {
  const ShapeCost& c = kCosts[shape];
  const int64_t slots = static_cast<int64_t>(cus) * c.per_cu;
  const int64_t units = tiles * splits, rest = units % slots;
  const float n = static_cast<float>((z.steps + splits - 1) / splits);
  const float whole = n * c.full + c.fixed;
  float us = static_cast<float>(units / slots) * whole;
  if (z.ragged && units > slots)  // tiles of different lengths end at different times
    us = static_cast<float>(units) / slots * whole;
  else if (rest > cus)
    us += whole;
  else if (rest)
    us += partly_us(cost_of(shape, slices), n, static_cast<float>(rest * slices) / cus);
  if (splits > 1)
    us += kJoin + static_cast<float>(z.rows) * z.cols * (8.0f * splits + 4.0f) / kJoinBytesPerUs;
  return us;
}

// Contraction ranges to consider.  A weight gradient's contraction, the rows,
// may be much longer than its output has tiles: more than eight ranges where
// eight leave a fifth of the CUs without work, while each has kRangeSteps
// steps and a slot of the GPU (65536 x 64 -> 64, one tile: 64 ranges 11 us,
// eight 35; 2^22 x 8 -> 8: 512 ranges 56 us, eight 1803; 76483 x 336 -> 264,
// 30 tiles: 16 ranges 43 us, eight 40).
int64_t most_splits(int op, const Sizes& z, int64_t tiles, int shape, int cus) {
  const int64_t few = std::min<int64_t>(kFewSplits, z.steps);
  if (op != kWeightGrad || tiles * kFewSplits * 5 > cus * 4) return few;
  return std::max(few, std::min(z.steps / kRangeSteps, cus * kCosts[shape].per_cu / tiles));
}

}  // namespace

ProductPlan product_plan(int op, int64_t P, int G, int K, int F, int cus) {
  const Sizes z = sizes_of(op, P, G, K, F);
  // Few rows: the thin kernel, while the rows of x, which every block reads,
  // weigh little (16 x 4096 -> 4096: 11.4 us against 13.8 for the best tile
  // and split; 16 x 11264 -> 4096: 27.6 against 23.8).  No estimate: only the
  // gradients' are compared.
  if (op == kForward && P <= kThinRows && P * K <= 98304)
    return {tiles_about(op, P, G, K, F, kShapeThin16) <= cus / 2 ? kShapeThin8 : kShapeThin16, 1,
            cus, 1, 0.0f};
  // Few rows a group (at most a tile each, about): every shape streams the
  // weights at HBM rate, Small a little faster (64 tokens on 8 of 288 experts,
  // 4096 -> 1280: 235 us; Big 246, Half 243).  A few tiles of many steps are
  // cut into ranges, one for every CU at most (17 rows in 8 groups, 11264 ->
  // 256: 14 us in eight, 34 in one; 73 in 12, 2544 -> 480, 104 tiles of 40
  // steps: 14 us in four, 11 in one).
  if (op != kWeightGrad && z.ragged && P > kThinRows && P <= 16 * static_cast<int64_t>(G)) {
    const int64_t tiles = tile_count(op, P, G, K, F, true, kShapeSizes[kShapeSmall]);
    ProductPlan few{kShapeSmall, 1, cus, 1, product_us(z, tiles, kShapeSmall, 1, 1, cus)};
    for (int splits = 2; splits <= 8 && splits <= z.steps && tiles * splits <= cus; splits *= 2) {
      const float us = product_us(z, tiles, kShapeSmall, splits, 1, cus) + kRaggedJoin;
      if (us < few.us) few = {kShapeSmall, splits, cus, 1, us};
    }
    return few;
  }
  ProductPlan best{kShapeSmall, 1, cus, 1, 0.0f};
  for (int s = kShapeBig; s <= kShapeSmall; ++s) {
    const int64_t tiles = tiles_about(op, P, G, K, F, s);
    const int64_t most = most_splits(op, z, tiles, s, cus);
    for (int splits = 1; splits <= most; splits *= 2) {
      const int slices = s == kShapeBig && op != kWeightGrad && !z.ragged && splits == 1
                             ? last_round_slices(tiles, cus)
                             : 1;
      const float us = product_us(z, tiles, s, splits, slices, cus) +
                       (splits > kFewSplits ? kManyJoin : 0.0f);
      if (best.us == 0.0f || us < best.us) best = {s, splits, cus, slices, us};
    }
  }
  return best;
}

bool pair_plan(int64_t P, int G, int K, int F, int cus, ProductPlan* x, ProductPlan* w) {
  const Sizes zx = sizes_of(kInputGrad, P, G, K, F), zw = sizes_of(kWeightGrad, P, G, K, F);
  const ProductPlan ax = product_plan(kInputGrad, P, G, K, F, cus);
  const ProductPlan aw = product_plan(kWeightGrad, P, G, K, F, cus);
  float best_us = ax.us + aw.us + kSecondLaunch;
  bool found = false;
  auto consider = [&](int sx, int slices, int sw) {
    const ShapeCost &cx = cost_of(sx, slices), &cw = kCosts[sw];
    const float slots = static_cast<float>(cus) * cw.per_cu;
    const float nx = static_cast<float>(tiles_about(kInputGrad, P, G, K, F, sx) * slices);
    const float nw = static_cast<float>(tiles_about(kWeightGrad, P, G, K, F, sw));
    const float lx = static_cast<float>(zx.steps), lw = static_cast<float>(zw.steps);
    float us;
    if (nx + nw <= cus) {  // one round
      const float taken = (nx + nw) / cus;
      us = std::max(partly_us(cx, lx, taken), partly_us(cw, lw, taken));
    } else {
      // as much of the GPU's time as the tiles take, and of the last round
      // what a tile leaves over
      const float tx = lx * cx.full + cx.fixed, tw = lw * cw.full + cw.fixed;
      const float rounds = (nx + nw) / slots;
      const float last = rounds - static_cast<float>(static_cast<int>(rounds));
      // (long dense runs of Big tiles: one round saved; of thirteen sizes of 1e3
      // to 15e3 rows none is slower than apart by more than 1%, and 8192 x 5120
      // -> 7168 takes 943 us, apart 998, 1065 x 5960 -> 8248 219, apart 237)
      const bool even = sx == kShapeBig && slices == 1 && sw == kShapeBig && rounds >= 2.0f &&
                        !zx.ragged;
      us = std::max((nx * tx + nw * tw) / slots * (even ? 0.98f : kMixed) +
                        (last > 0.0f ? (1.0f - last) * tw * kLeftOver : 0.0f),
                    std::max(tx, tw) * kLongest);
      // dW's blocks come behind dx's: its tiles start when dx's last ones do,
      // and above a third of the CUs, about, two Small ones share one even then
      // (11353 x 6152 -> 336, Half: 251 us, apart 178; 3800 x 728 -> 608, 120
      // Small tiles of 60 steps: 38, apart 28; 2552 x 1360 -> 160, 66 of 40
      // steps: 17, apart 21)
      const int64_t slot = static_cast<int64_t>(slots), tiles = static_cast<int64_t>(nw);
      const float rest = static_cast<float>(tiles % slot);
      const bool shared = cw.per_cu > 1 && rest > kShared * cus;
      const float end = rest == 0.0f ? 0.0f : shared ? tw : partly_us(cw, lw, rest / cus);
      us = std::max(us, nx * tx / slots - tx + static_cast<float>(tiles / slot) * tw + end);
    }
    if (us < best_us) {
      best_us = us;
      found = true;
      *x = {sx, 1, cus, slices};
      *w = {sw, 1, cus, 1};
    }
  };
  for (int sw : {kShapeBig, kShapeHalf}) {
    consider(kShapeHalf, 1, sw);
    consider(kShapeBig, 1, sw);
    // (a cut tile's slices take the place of whole tiles in the last round only)
    if (!zx.ragged && tiles_about(kInputGrad, P, G, K, F, kShapeBig) < cus) {
      consider(kShapeBig, 2, sw);
      consider(kShapeBig, 4, sw);
    }
  }
  consider(kShapeSmall, 1, kShapeSmall);
  return found;
}

size_t product_part_bytes(int op, int64_t P, int G, int K, int F, const ProductPlan& plan) {
  if (plan.splits <= 1) return 0;
  const size_t rows = op == kWeightGrad ? static_cast<size_t>(G) * F : static_cast<size_t>(P);
  const size_t cols = op == kForward ? F : K;
  return (rows * cols + (op == kWeightGrad ? rows : 0)) * 4 * plan.splits;
}

namespace {

ProductArgs with_plan(int op, const ProductArgs& p, const ProductPlan& plan) {
  ProductArgs q = p;
  q.splits = plan.splits;
  q.cus = plan.cus;
  q.slices = plan.slices;
  if (op == kWeightGrad) {
    // A weight gradient that will not stay in the 256 MB last-level cache is
    // stored past the caches, which then keep the operands (1 GB of fp32: 389
    // us instead of 455; 185 MB: 346 instead of 336).
    q.stream = static_cast<int64_t>(q.G) * q.F * q.K * (q.y_f32 ? 4 : 2) > (int64_t(256) << 20);
    q.part_db = q.part + static_cast<int64_t>(q.splits) * q.G * q.F * q.K;
  }
  return q;
}

}  // namespace

hipError_t launch_product(int op, const ProductArgs& p, const ProductPlan& plan,
                          hipStream_t stream) {
  const ProductArgs q = with_plan(op, p, plan);
  if (op == kForward) return launch_forward(q, plan.shape, stream);
  if (op == kInputGrad) return launch_input_grad(q, plan.shape, stream);
  return launch_weight_grad(q, plan.shape, stream);
}

hipError_t launch_pair(const ProductArgs& x, const ProductPlan& px, const ProductArgs& w,
                       const ProductPlan& pw, hipStream_t stream) {
  return launch_grad_pair(with_plan(kInputGrad, x, px), px.shape, with_plan(kWeightGrad, w, pw),
                          pw.shape, stream);
}

hipError_t launch_source_rows(const int32_t* row_ids, int row_div, int64_t x_rows, int64_t P,
                              int32_t* src, hipStream_t stream) {
  source_rows_kernel<<<static_cast<unsigned>((P + kSourcePad + 255) / 256), 256, 0, stream>>>(
      row_ids, row_div, x_rows, P, src);
  return hipGetLastError();
}

size_t act_grad_part_bytes(int64_t T, int F) {
  const int rows = std::max(strip_rows(T), 1);
  return static_cast<size_t>((T + rows - 1) / rows) * F * 4;
}

hipError_t launch_act_grad(const uint16_t* dy, const uint16_t* z, int act, int64_t T, int F,
                           uint16_t* dz, float* db, int accumulate, float* part,
                           hipStream_t stream) {
  const int rows = strip_rows(T), strips = static_cast<int>((T + rows - 1) / rows);
  const dim3 grid((F + kStripCols - 1) / kStripCols, strips);
  const bool one = strips == 1;
  float* const sums = !db ? nullptr : one ? db : part;
  const bool add = one && accumulate;
  if (static_cast<int64_t>(grid.x) * strips < kStripMany)
    act_grad_kernel<16><<<grid, 64 * 16, 0, stream>>>(dy, z, act, T, F, dz, sums, rows, add);
  else
    act_grad_kernel<8><<<grid, 64 * 8, 0, stream>>>(dy, z, act, T, F, dz, sums, rows, add);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !db || one) return e;
  strip_sum_kernel<<<(F + 63) / 64, 256, 0, stream>>>(part, strips, F, db, accumulate);
  return hipGetLastError();
}

}  // namespace moe

// What the launches of the linear and grouped products share: each block's
// tile, the tile shapes, the kernel over them, and the join of split
// contractions.
#pragma once

#include <algorithm>

#include "product_tile.h"

namespace moe {

namespace {

constexpr int kGroupM = 8;  // row tiles walked together, so that they share column operands

__device__ __forceinline__ int clamp_row(int v, int64_t P) {
  return static_cast<int>(min<int64_t>(max(v, 0), P));
}

// Block -> unit.  Forward, input gradient and one group: each XCD takes a
// contiguous range (xcd_remap).  The weight gradient of ragged groups: runs of
// units dealt over the XCDs in turn, since contiguous ranges of experts of
// different sizes leave some XCDs long behind the others.  A run is a column
// of up to 8 row tiles, whose blocks share x's panel in their L2, else 4 units
// (48 experts of 1280 x 4096, five row tiles: runs of 5 375 us, 4 381, 16 409,
// 1 459; 64 of 4096 x 2048, sixteen: runs of 4 410 us, 5 421, 10 438).
// Returns -1 for a block without work.
__host__ __device__ __forceinline__ int run_of(int F, int bm) {
  const int tiles = (F + bm - 1) / bm;
  return tiles >= 4 && tiles <= kGroupM ? tiles : 4;
}
__host__ __device__ __forceinline__ int dealt_unit(int bid, int run, int nvalid) {
  const int xcd = bid % kNumXcd, slot = bid / kNumXcd;
  const int u = (slot / run * kNumXcd + xcd) * run + slot % run;
  return u < nvalid ? u : -1;
}

// Block -> unit of a launch whose last tiles, from `cut` on (a multiple of the
// XCDs), are cut into slices of rows: they follow the whole ones in every
// XCD's order.  *part: which slice.
__host__ __device__ __forceinline__ int cut_unit(int bid, int cut, int units, int slices,
                                                 int* part) {
  *part = 0;
  if (bid < cut) return xcd_remap(bid, cut);
  const int v = xcd_remap(bid - cut, (units - cut) * slices);
  if (v < 0) return -1;
  *part = v % slices;
  return cut + v / slices;
}

// Block bid's unit, false if it has none.  Forward and input gradient: the
// tiles of a group number ceil(rows / BM), known on the device only, so the
// block prefixes the groups' tile counts itself (at most 1024 groups, a few
// per thread) -- about 1 us, against a launch and a tile list in memory.
template <int OP, int BM, int BN, int THREADS>
__device__ __forceinline__ bool find_unit(const ProductArgs& p, int bid, int* sh, Unit* un) {
  const int tid = threadIdx.x;
  const int N = OP == kForward ? p.F : p.K;
  // db alone (no y): one column tile
  const int NT = OP == kWeightGrad && !p.y ? 1 : (N + BN - 1) / BN;
  if constexpr (OP == kWeightGrad) {
    const int MT = (p.F + BM - 1) / BM;
    const int per = p.G * MT * NT;
    const int u = p.offsets ? dealt_unit(bid, run_of(p.F, BM), per * p.splits)
                            : xcd_remap(bid, per * p.splits);
    if (u < 0) return false;
    un->split = u / per;
    const int v = u % per;
    un->g = v / (MT * NT);
    const int t = v % (MT * NT);
    const int first = t / (kGroupM * NT) * kGroupM;
    const int gm = min(kGroupM, MT - first);
    const int w = t - first * NT;
    un->row0 = (first + w % gm) * BM;
    un->rows = min(BM, p.F - un->row0);
    un->col0 = w / gm * BN;
    un->begin = p.offsets ? clamp_row(p.offsets[un->g], p.P) : 0;
    const int end = p.offsets ? clamp_row(p.offsets[un->g + 1], p.P) : static_cast<int>(p.P);
    un->len = max(0, end - un->begin);
    return true;
  }
  int tiles, base = 0, n = static_cast<int>(p.P), first_tile = 0, total;
  if (!p.offsets) {
    total = static_cast<int>((p.P + BM - 1) / BM);
  } else {
    const int c = (p.G + THREADS - 1) / THREADS;
    int mine = 0;
    for (int i = tid * c; i < min(tid * c + c, p.G); ++i) {
      const int b = clamp_row(p.offsets[i], p.P);
      mine += (max(0, clamp_row(p.offsets[i + 1], p.P) - b) + BM - 1) / BM;
    }
    const int lane = tid & 63, wid = tid >> 6;
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 63) sh[wid] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < wid) before += sh[w];
      total += sh[w];
    }
    total = __builtin_amdgcn_readfirstlane(total);
    const int u = xcd_remap(bid, total * NT * p.splits);
    if (u < 0) return false;
    int t = u % (total * NT) / NT;
    int at = before + incl - mine;
    if (t >= at && t < at + mine) {
      for (int i = tid * c; i < min(tid * c + c, p.G); ++i) {
        const int b = clamp_row(p.offsets[i], p.P);
        const int rows = max(0, clamp_row(p.offsets[i + 1], p.P) - b);
        const int k = (rows + BM - 1) / BM;
        if (t < at + k) {
          sh[16] = i;
          sh[17] = b;
          sh[18] = rows;
          sh[19] = at;
          break;
        }
        at += k;
      }
    }
    __syncthreads();
    un->g = __builtin_amdgcn_readfirstlane(sh[16]);
    base = __builtin_amdgcn_readfirstlane(sh[17]);
    n = __builtin_amdgcn_readfirstlane(sh[18]);
    first_tile = __builtin_amdgcn_readfirstlane(sh[19]);
    __syncthreads();
  }
  if (!p.offsets) un->g = 0;
  int part = 0, parts = 1;  // which of how many slices of the tile's rows
  int u;
  if (BM == 256 && p.whole >= 0) {
    const int cut = kNumXcd * (p.whole / kNumXcd);
    u = cut_unit(bid, cut, total * NT, p.slices, &part);
    if (u < 0) return false;
    if (u >= cut) parts = p.slices;
  } else {
    u = xcd_remap(bid, total * NT * p.splits);
    if (u < 0) return false;
  }
  un->split = u / (total * NT);
  const int v = u % (total * NT);
  tiles = (n + BM - 1) / BM;
  // inside the group: runs of kGroupM row tiles, the row tile fastest
  const int w = v - first_tile * NT;
  const int gfirst = w / (kGroupM * NT) * kGroupM;
  const int gm = min(kGroupM, tiles - gfirst);
  const int x = w - gfirst * NT;
  const int rt = gfirst + x % gm;
  un->row0 = base + rt * BM + part * (BM / parts);
  un->rows = min(BM / parts, n - rt * BM - part * (BM / parts));
  if (un->rows <= 0) return false;
  un->col0 = x / gm * BN;
  un->begin = base;
  un->len = n;
  return true;
}

// Tile shapes of the ring-buffered mainloop.  Big: many rows, whole rounds of
// the GPU; 8 waves of 128 x 64, A 2 and B 3 stages deep (160 KB of LDS).
// Duo: two blocks of four such waves a CU, so that one's start and epilogue
// overlap the other's products, at 1.5 times the operand traffic: short
// contractions.  Half and Small: fewer rows or columns, more blocks.  Three,
// Half and Flat also serve the remainders of groups and the cut tiles in Big's
// launches.
template <int OP> using Big = Tile<OP, 256, 256, 2, 4, 2, 3>;
template <int OP> using Half = Tile<OP, 128, 256, 2, 4, 3, 3>;
template <int OP> using Three = Tile<OP, 192, 256, 2, 4, 2, 3>;
template <int OP> using Duo = Tile<OP, 256, 128, 2, 2, 3, 3, 32>;
template <int OP> using Small = Tile<OP, 64, 64, 2, 2, 4, 4>;
template <int OP> using Flat = Tile<OP, 64, 256, 2, 4, 4, 4>;

// Block bid of a product.
template <int OP, class T, bool GATHER>
__device__ __forceinline__ void run_block(const ProductArgs& p, int bid, uint8_t* smem) {
  Unit un;
  if (!find_unit<OP, T::BM, T::BN, T::THREADS>(p, bid, reinterpret_cast<int*>(smem), &un)) return;
  if constexpr (OP == kWeightGrad) {
    if (p.accumulate && un.len == 0 && p.splits == 1) return;
    if (p.db && un.col0 == 0) {
      product_tile<OP, T, GATHER, true>(p, smem, un);
      return;
    }
  } else if constexpr (T::BM == 256 && T::BN == 256) {
    // fewer rows, the remainder of a group or a cut tile: the same columns
    // with less of A to load and to multiply
    static_assert(Flat<OP>::RING <= T::RING && Half<OP>::RING <= T::RING &&
                      Three<OP>::RING <= T::RING,
                  "the same LDS");
    static_assert(Flat<OP>::THREADS == T::THREADS && Half<OP>::THREADS == T::THREADS &&
                      Three<OP>::THREADS == T::THREADS,
                  "and waves");
    if (un.rows <= 64) {
      product_tile<OP, Flat<OP>, false, false>(p, smem, un);
      return;
    }
    if (un.rows <= 128) {
      product_tile<OP, Half<OP>, false, false>(p, smem, un);
      return;
    }
    if (un.rows <= 192) {
      product_tile<OP, Three<OP>, false, false>(p, smem, un);
      return;
    }
  }
  product_tile<OP, T, GATHER, false>(p, smem, un);
}

template <int OP, class T, bool GATHER>
__global__ __launch_bounds__(T::THREADS, 2) void product_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::RING];
  run_block<OP, T, GATHER>(p, blockIdx.x, smem);
}

// Sums the contraction ranges' partial results in order and finishes them.
// Thread i: eight consecutive columns of a row; the threads behind the last
// row: db.
// SPLITS is a constant so that all of a thread's loads are under way at once
// (3.9 us for 64 x 4096 from eight ranges; a loop over four took 4.7).
template <int OP, int SPLITS>
__global__ __launch_bounds__(256) void product_join(ProductArgs p) {
  const int N = OP == kForward ? p.F : p.K;
  const int64_t rows = OP == kWeightGrad ? static_cast<int64_t>(p.G) * p.F : p.P;
  const int per_row = N / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = i / per_row;
  if (row < rows) {
    const int col = static_cast<int>(i - row * per_row) * 8;
    const float* bias = p.bias;
    if (OP != kWeightGrad && p.offsets) {
      // the group whose rows hold this one: the last with offset <= row
      if (row < clamp_row(p.offsets[0], p.P) || row >= clamp_row(p.offsets[p.G], p.P)) return;
      int lo = 0, hi = p.G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.offsets[mid] <= row) lo = mid; else hi = mid;
      }
      if (bias) bias += static_cast<int64_t>(lo) * p.F;
    }
    if (OP == kWeightGrad && !p.y) return;
    F8 w[SPLITS];
#pragma unroll
    for (int s = 0; s < SPLITS; ++s) w[s] = load8(p.part + (s * rows + row) * N + col);
    F8 v = w[0];
#pragma unroll
    for (int s = 1; s < SPLITS; ++s)
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += w[s].v[q];
    if (OP == kForward)
      finish_one(p, v, bias, row, col, N);
    else
      put_grad8<false>(p, v, row * N + col);
  } else if (OP == kWeightGrad && p.db) {
    const int64_t j = i - rows * per_row;
    if (j >= rows) return;
    float v = 0.0f;
#pragma unroll
    for (int s = 0; s < SPLITS; ++s) v += p.part_db[s * rows + j];
    p.db[j] = p.accumulate ? p.db[j] + v : v;
  }
}

// The same for a weight gradient in more than eight ranges.  A thread takes
// eight consecutive values of an eighth of the ranges, in order and
// kJoinAhead loads at a time; the eighths' sums meet in LDS, in order too.
// The values of dW come first, then db's.
constexpr int kJoinItems = 32, kJoinParts = 8, kJoinAhead = 8;

__global__ __launch_bounds__(kJoinItems * kJoinParts) void product_join_many(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[kJoinParts - 1][kJoinItems * 8];
  const int64_t rows = static_cast<int64_t>(p.G) * p.F;
  const int64_t dw = p.y ? rows * p.K : 0, total = dw + (p.db ? rows : 0);
  const int lane = threadIdx.x % kJoinItems, sub = threadIdx.x / kJoinItems;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kJoinItems + lane) * 8;
  F8 v{};
  if (at < total) {
    const float* src = at < dw ? p.part + at : p.part_db + (at - dw);
    const int64_t stride = at < dw ? dw : rows;
    const int n = p.splits / kJoinParts;
    src += sub * n * stride;
    for (int s = 0; s < n; s += kJoinAhead) {
      F8 w[kJoinAhead];
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) w[i] = load8(src + min(s + i, n - 1) * stride);
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i)
        if (s + i < n)
#pragma unroll
          for (int q = 0; q < 8; ++q) v.v[q] += w[i].v[q];
    }
  }
  if (sub > 0) store8(&sums[sub - 1][lane * 8], v);
  __syncthreads();
  if (sub > 0 || at >= total) return;
#pragma unroll
  for (int i = 0; i < kJoinParts - 1; ++i) {
    const F8 o = load8(&sums[i][lane * 8]);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
  }
  if (at < dw)
    put_grad8<false>(p, v, at);
  else
    put_grad8<false>(p.db + (at - dw), v, p.accumulate);
}

enum Shape : int {
  kShapeBig, kShapeHalf, kShapeDuo, kShapeSmall,
  kShapeThin8, kShapeThin16,  // forward only: product_thin
  kNumShapes
};

constexpr int kThinRows = 16;  // rows of product_thin's tiles
// Contraction ranges that product_join sums; a weight gradient may have more.
constexpr int kFewSplits = 8;

struct ShapeSize {
  int bm, bn;
};
constexpr ShapeSize kShapeSizes[kNumShapes] = {{256, 256}, {128, 256},     {256, 128},
                                               {64, 64},   {kThinRows, 8}, {kThinRows, 16}};

// Tiles of a product, at most (the tiles of ragged groups are counted on the device).
int64_t tile_count(int op, int64_t P, int G, int K, int F, bool grouped, ShapeSize s) {
  const int64_t nt = ((op == kForward ? F : K) + s.bn - 1) / s.bn;
  if (op == kWeightGrad) return static_cast<int64_t>(G) * ((F + s.bm - 1) / s.bm) * nt;
  return (grouped ? P / s.bm + std::min<int64_t>(G, P) : (P + s.bm - 1) / s.bm) * nt;
}

// Blocks for that many units: whole rounds of the XCDs, of runs where they are dealt.
unsigned block_count(int64_t units, int run) {
  const int64_t round = static_cast<int64_t>(run) * kNumXcd;
  return static_cast<unsigned>((units + round - 1) / round * round);
}

// The grid of a product in tiles of T, and the launch's own fields of p.
template <int OP, class T>
unsigned grid_of(ProductArgs* p) {
  const int64_t units =
      tile_count(OP, p->P, p->G, OP == kWeightGrad && !p->y ? 1 : p->K, p->F,
                 p->offsets != nullptr, {T::BM, T::BN}) * p->splits;
  p->whole = -1;
  if (T::BM == 256 && T::BN == 256 && OP != kWeightGrad && !p->offsets && p->slices > 1) {
    p->whole = static_cast<int>(units - units % p->cus);
    const int64_t cut = p->whole / kNumXcd * kNumXcd;
    return static_cast<unsigned>(
        cut + ((units - cut) * p->slices + kNumXcd - 1) / kNumXcd * kNumXcd);
  }
  return block_count(units, OP == kWeightGrad && p->offsets ? run_of(p->F, T::BM) : 1);
}

template <int OP, class T>
hipError_t launch_tiles(ProductArgs p, hipStream_t stream) {
  const unsigned grid = grid_of<OP, T>(&p);
  if (grid == 0) return hipSuccess;
  if (OP == kWeightGrad && p.src && p.y)
    product_kernel<OP, T, OP == kWeightGrad><<<grid, T::THREADS, 0, stream>>>(p);
  else
    product_kernel<OP, T, false><<<grid, T::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

template <int OP>
hipError_t launch_op(const ProductArgs& p, int shape, hipStream_t stream) {
  hipError_t e;
  switch (shape) {
    case kShapeBig: e = launch_tiles<OP, Big<OP>>(p, stream); break;
    case kShapeHalf: e = launch_tiles<OP, Half<OP>>(p, stream); break;
    case kShapeDuo: e = launch_tiles<OP, Duo<OP>>(p, stream); break;
    default: e = launch_tiles<OP, Small<OP>>(p, stream); break;
  }
  if (e != hipSuccess || p.splits == 1) return e;
  if (OP == kWeightGrad && p.splits > kFewSplits) {
    const int64_t values = static_cast<int64_t>(p.G) * p.F * ((p.y ? p.K : 0) + (p.db ? 1 : 0));
    const int64_t per = kJoinItems * 8;
    product_join_many<<<static_cast<unsigned>((values + per - 1) / per),
                        kJoinItems * kJoinParts, 0, stream>>>(p);
    return hipGetLastError();
  }
  const int N = OP == kForward ? p.F : p.K;
  const int64_t rows = OP == kWeightGrad ? static_cast<int64_t>(p.G) * p.F : p.P;
  const int64_t threads = rows * (N / 8) + (OP == kWeightGrad && p.db ? rows : 0);
  const unsigned grid = static_cast<unsigned>((threads + 255) / 256);
  switch (p.splits) {
    case 2: product_join<OP, 2><<<grid, 256, 0, stream>>>(p); break;
    case 4: product_join<OP, 4><<<grid, 256, 0, stream>>>(p); break;
    case 8: product_join<OP, 8><<<grid, 256, 0, stream>>>(p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

// Launches of one product in a shape, and of both gradients together (both
// Small, or each Big or Half).
hipError_t launch_forward(const ProductArgs& p, int shape, hipStream_t stream);
hipError_t launch_input_grad(const ProductArgs& p, int shape, hipStream_t stream);
hipError_t launch_weight_grad(const ProductArgs& p, int shape, hipStream_t stream);
hipError_t launch_grad_pair(const ProductArgs& x, int sx, const ProductArgs& w, int sw,
                            hipStream_t stream);

}  // namespace moe

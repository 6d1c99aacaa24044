// Linear and grouped products on gfx950 matrix cores: y = x W^T with bias,
// activation and residual, and the gradients dx = dy W and dW = dy^T x, for
// one group of rows or for one group per expert with ragged sizes.

#include <algorithm>

#include "activation.h"
#include "products.h"

namespace moe {

namespace {

constexpr int kGroupM = 8;  // row tiles walked together, so that they share column operands

// The work of one block: a tile of one group's output and a contraction range.
struct Unit {
  int g;         // group
  int row0;      // first output row (forward, input gradient: a row of all P;
                 // weight gradient: an out feature)
  int rows;      // output rows in the tile, >= 1
  int col0;      // first output column
  int begin;     // weight gradient: the group's first row and row count
  int len;
  int split;
};

__device__ __forceinline__ int clamp_row(int v, int64_t P) {
  return static_cast<int>(min<int64_t>(max(v, 0), P));
}

// The block's unit, false if it has none.  Forward and input gradient: the
// tiles of a group number ceil(rows / BM), known on the device only, so the
// block prefixes the groups' tile counts itself (at most 1024 groups, a few
// per thread) -- about 1 us, against a launch and a tile list in memory.
template <int OP, int BM, int BN, int THREADS>
__device__ bool find_unit(const ProductArgs& p, int* sh, Unit* un) {
  const int tid = threadIdx.x;
  const int N = OP == kForward ? p.F : p.K;
  // db alone (no y): one column tile
  const int NT = OP == kWeightGrad && !p.y ? 1 : (N + BN - 1) / BN;
  if constexpr (OP == kWeightGrad) {
    const int MT = (p.F + BM - 1) / BM;
    const int per = p.G * MT * NT;
    const int u = xcd_remap(blockIdx.x, per * p.splits);
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
    const int u = xcd_remap(blockIdx.x, total * NT * p.splits);
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
    un->g = sh[16];
    base = sh[17];
    n = sh[18];
    first_tile = sh[19];
    __syncthreads();
  }
  if (!p.offsets) un->g = 0;
  const int u = xcd_remap(blockIdx.x, total * NT * p.splits);
  if (u < 0) return false;
  un->split = u / (total * NT);
  const int v = u % (total * NT);
  tiles = (n + BM - 1) / BM;
  // inside the group: runs of kGroupM row tiles, the row tile fastest
  const int w = v - first_tile * NT;
  const int gfirst = w / (kGroupM * NT) * kGroupM;
  const int gm = min(kGroupM, tiles - gfirst);
  const int x = w - gfirst * NT;
  const int rt = gfirst + x % gm;
  un->row0 = base + rt * BM;
  un->rows = min(BM, n - rt * BM);
  un->col0 = x / gm * BN;
  un->begin = base;
  un->len = n;
  return true;
}

// Bias, z, activation, residual and the store of eight consecutive columns.
// Rounded once per output, from the fp32 sum.
__device__ __forceinline__ void finish8(const ProductArgs& p, F8 v, const float* bias, int64_t row,
                                        int col, int N) {
  const int64_t at = row * N + col;
  if (bias) {
    const F8 b = load8(bias + col);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += b.v[q];
  }
  if (p.z) store8(p.z + at, v);
  if (p.act != MOE_ACT_NONE)
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] = activate(v.v[q], p.act);
  if (p.residual) {
    const F8 r = load8(p.residual + at);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += r.v[q];
  }
  if (p.y_f32) {
    float* y = static_cast<float*>(p.y) + at;
    if (p.accumulate) {
      const F8 o = load8(y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
    }
    store8(y, v);
  } else {
    uint16_t* y = static_cast<uint16_t*>(p.y) + at;
    if (p.accumulate) {
      const F8 o = load8(y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
    }
    store8(y, v);
  }
}

// x's row of row r, or -1.
__device__ __forceinline__ int64_t source_row(const ProductArgs& p, int r) {
  if (!p.src) return r;
  const int id = p.src[r];
  if (id < 0) return -1;
  const int64_t s = id / p.row_div;
  return s < p.x_rows ? s : -1;
}

// The plainest tile: 64 x 64, staged through registers, both operands laid
// down contraction-contiguous.
template <int OP>
__global__ __launch_bounds__(256) void product_simple(ProductArgs p) {
  constexpr int BM = 64, BN = 64, BK = 32, LD = BK + 8;
  __shared__ __attribute__((aligned(16))) uint16_t as[BM * LD], bs[BN * LD];
  __shared__ float out[BM * (BN + 4)];
  __shared__ int sh[32];
  Unit un;
  if (!find_unit<OP, BM, BN, 256>(p, sh, &un)) return;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int N = OP == kForward ? p.F : p.K;
  const int L = OP == kForward ? p.K : OP == kInputGrad ? p.F : un.len;
  const int KT = (L + BK - 1) / BK, per = (KT + p.splits - 1) / p.splits;
  const int k_first = min(KT, un.split * per), k_last = min(KT, k_first + per);
  const uint16_t* w = p.b + (OP == kWeightGrad ? 0 : static_cast<int64_t>(un.g) * p.F * p.K);
  f32x16 acc{};
  float dbsum = 0.0f;
  for (int kt = k_first; kt < k_last; ++kt) {
    const int k0 = kt * BK;
    u32x4 va{}, vb{};
    {  // A: dy^T for the weight gradient, else rows of x or dy
      if (OP == kWeightGrad) {
        const int k = k0 + tid / 8, c = un.row0 + tid % 8 * 8;
        if (k < L && c < p.F)
          va = *reinterpret_cast<const u32x4*>(p.a + static_cast<int64_t>(un.begin + k) * p.F + c);
      } else {
        const int r = tid / 4, k = k0 + tid % 4 * 8;
        if (r < un.rows && k < L) {
          const int64_t s = OP == kForward ? source_row(p, un.row0 + r) : un.row0 + r;
          if (s >= 0) va = *reinterpret_cast<const u32x4*>(p.a + s * L + k);
        }
      }
      if (OP == kForward) {
        const int r = un.col0 + tid / 4, k = k0 + tid % 4 * 8;
        if (r < N && k < L) vb = *reinterpret_cast<const u32x4*>(w + static_cast<int64_t>(r) * L + k);
      } else {
        const int k = k0 + tid / 8, c = un.col0 + tid % 8 * 8;
        if (k < L && c < N && (OP != kWeightGrad || p.y)) {
          const int64_t s = OP == kWeightGrad ? source_row(p, un.begin + k) : k;
          if (s >= 0) vb = *reinterpret_cast<const u32x4*>(w + s * N + c);
        }
      }
    }
    __syncthreads();
    auto put = [&](uint16_t* lds, const u32x4& v, bool strided) {
      if (!strided) {
        *reinterpret_cast<u32x4*>(lds + tid / 4 * LD + tid % 4 * 8) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          lds[(tid % 8 * 8 + q) * LD + tid / 8] = static_cast<uint16_t>(v[q / 2] >> (q % 2 * 16));
      }
    };
    put(as, va, OP == kWeightGrad);
    put(bs, vb, OP != kForward);
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
      const int o = 16 * ks + 8 * (lane >> 5);
      const bf16x8 fa = *reinterpret_cast<const bf16x8*>(as + ((wid >> 1) * 32 + (lane & 31)) * LD + o);
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(bs + ((wid & 1) * 32 + (lane & 31)) * LD + o);
      acc = mfma32(fb, fa, acc);
    }
    if (OP == kWeightGrad && p.db && un.col0 == 0 && tid < BM)
      for (int k = 0; k < BK; ++k) dbsum += bf16_to_f32(as[tid * LD + k]);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r)
    out[((wid >> 1) * 32 + (lane & 31)) * (BN + 4) + (wid & 1) * 32 + mfma32_row(r, lane)] = acc[r];
  __syncthreads();
  for (int i = tid; i < BM * BN / 8; i += 256) {
    const int r = i / (BN / 8), c = i % (BN / 8) * 8, col = un.col0 + c;
    if (r >= un.rows || col >= N || (OP == kWeightGrad && !p.y)) continue;
    F8 v;
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] = out[r * (BN + 4) + c + q];
    const int64_t row = (OP == kWeightGrad ? static_cast<int64_t>(un.g) * p.F : 0) + un.row0 + r;
    if (p.splits > 1) {
      const int64_t rows = OP == kWeightGrad ? static_cast<int64_t>(p.G) * p.F : p.P;
      store8(p.part + (un.split * rows + row) * N + col, v);
    } else {
      finish8(p, v, p.bias ? p.bias + static_cast<int64_t>(un.g) * p.F : nullptr, row, col, N);
    }
  }
  if (OP == kWeightGrad && p.db && un.col0 == 0 && tid < un.rows) {
    const int64_t i = static_cast<int64_t>(un.g) * p.F + un.row0 + tid;
    if (p.splits > 1)
      p.part_db[static_cast<int64_t>(un.split) * p.G * p.F + i] = dbsum;
    else
      p.db[i] = p.accumulate ? p.db[i] + dbsum : dbsum;
  }
}

// Sums the contraction ranges' partial results in order and finishes them.
// Thread i: eight consecutive columns of a row; the threads behind the last
// row: db.
template <int OP>
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
    F8 v{};
    for (int s = 0; s < p.splits; ++s) {
      const F8 w = load8(p.part + (s * rows + row) * N + col);
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += w.v[q];
    }
    finish8(p, v, bias, row, col, N);
  } else if (OP == kWeightGrad && p.db) {
    const int64_t j = i - rows * per_row;
    if (j >= rows) return;
    float v = 0.0f;
    for (int s = 0; s < p.splits; ++s) v += p.part_db[s * rows + j];
    p.db[j] = p.accumulate ? p.db[j] + v : v;
  }
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

// dz = dy act'(z) and the column sums of each strip of rows: a block takes
// a strip of 256 x 8 columns, a thread eight columns.
int strip_rows(int64_t T) { return 64 * static_cast<int>((T + 65535) / 65536); }

__global__ __launch_bounds__(256) void act_grad_kernel(const uint16_t* __restrict__ dy,
                                                       const uint16_t* __restrict__ z, int act,
                                                       int64_t T, int F, uint16_t* __restrict__ dz,
                                                       float* __restrict__ part, int strip) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= F) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * strip;
  const int64_t r1 = min<int64_t>(T, r0 + strip);
  F8 sum{};
#pragma unroll 4
  for (int64_t r = r0; r < r1; ++r) {
    F8 d = load8(dy + r * F + c);
    const F8 v = load8(z + r * F + c);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      d.v[q] *= act_slope(v.v[q], act);
      sum.v[q] += d.v[q];
    }
    store8(dz + r * F + c, d);
  }
  if (part) store8(part + static_cast<int64_t>(blockIdx.y) * F + c, sum);
}

__global__ __launch_bounds__(256) void strip_sum_kernel(const float* __restrict__ part, int strips,
                                                        int F, float* __restrict__ db,
                                                        int accumulate) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= F) return;
  float v = 0.0f;
  for (int s = 0; s < strips; ++s) v += part[static_cast<int64_t>(s) * F + c];
  db[c] = accumulate ? db[c] + v : v;
}

template <int OP>
hipError_t launch_op(const ProductArgs& p, hipStream_t stream) {
  const int N = OP == kForward ? p.F : p.K;
  const int64_t NT = (N + 63) / 64;
  const int64_t tiles = OP == kWeightGrad ? static_cast<int64_t>(p.G) * ((p.F + 63) / 64)
                        : p.offsets      ? p.P / 64 + std::min<int64_t>(p.G, p.P)
                                         : (p.P + 63) / 64;
  const int64_t units = tiles * NT * p.splits;
  if (units <= 0) return hipSuccess;
  const int64_t grid = (units + kNumXcd - 1) / kNumXcd * kNumXcd;
  product_simple<OP><<<static_cast<unsigned>(grid), 256, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = OP == kWeightGrad ? static_cast<int64_t>(p.G) * p.F : p.P;
  const int64_t threads = rows * (N / 8) + (OP == kWeightGrad && p.db ? rows : 0);
  product_join<OP><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

ProductPlan product_plan(int op, int64_t P, int G, int K, int F, int cus) {
  (void)op, (void)P, (void)G, (void)K, (void)F, (void)cus;
  return {0, 1};
}

size_t product_part_bytes(int op, int64_t P, int G, int K, int F, const ProductPlan& plan) {
  if (plan.splits <= 1) return 0;
  const size_t rows = op == kWeightGrad ? static_cast<size_t>(G) * F : static_cast<size_t>(P);
  const size_t cols = op == kForward ? F : K;
  return (rows * cols + (op == kWeightGrad ? rows : 0)) * 4 * plan.splits;
}

hipError_t launch_product(int op, const ProductArgs& p, const ProductPlan& plan,
                          hipStream_t stream) {
  ProductArgs q = p;
  q.splits = plan.splits;
  if (op == kForward) return launch_op<kForward>(q, stream);
  if (op == kInputGrad) return launch_op<kInputGrad>(q, stream);
  q.part_db = q.part + static_cast<int64_t>(q.splits) * q.G * q.F * q.K;
  return launch_op<kWeightGrad>(q, stream);
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
  const dim3 grid((F / 8 + 255) / 256, strips);
  act_grad_kernel<<<grid, 256, 0, stream>>>(dy, z, act, T, F, dz, db ? part : nullptr,
                                       rows);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !db) return e;
  strip_sum_kernel<<<(F + 255) / 256, 256, 0, stream>>>(part, strips, F, db, accumulate);
  return hipGetLastError();
}

}  // namespace moe

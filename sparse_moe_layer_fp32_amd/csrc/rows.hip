// Rows out to the experts and back, with weights, and their gradients.
//
//   dispatch          r[pos[t][j]] = x[t]
//   its gradient      dx[t] = base[t] + sum_j dr[pos[t][j]]
//   combine           y[t]  = base[t] + sum_j w[t][j] r[pos[t][j]]
//   its gradients     dr[pos[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], r[pos[t][j]]>
//
// Bound: HBM.  All four walk the tokens, so that a token's own row is read or
// written once, whatever top_k is, and every row of an expert once.  Sums are
// formed in fp32 in slot order.  A wave takes 8 columns a lane of one token, 512
// in all; of narrow rows (up to 256 columns) two, four or eight tokens at once.

#include "activation.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kRowThreads = 256;
constexpr int kSlots = 8;  // slots whose rows are under way together

__device__ __forceinline__ F8 scaled(const F8& v, float w) {
  F8 o;
#pragma unroll
  for (int q = 0; q < 8; ++q) o.v[q] = v.v[q] * w;
  return o;
}

// The token and first column of this lane; false if there is none.  LANES: how
// many lanes a token has in a wave.
template <int LANES>
__device__ __forceinline__ bool locate(const RowsArgs& p, int parts, int64_t* token, int* col) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * (kRowThreads / 64) +
                        __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (LANES == 64) {
    const uint32_t t = wave / parts;
    *token = t;
    *col = static_cast<int>((wave - t * parts) * 64 + lane) * 8;
  } else {
    *token = static_cast<int64_t>(wave) * (64 / LANES) + lane / LANES;
    *col = lane % LANES * 8;
  }
  return *token < p.tokens && *col < p.hidden;
}

// Positions of a token's slots j0 .. j0 + kSlots - 1, -1 where there is no row.
__device__ __forceinline__ void positions(const RowsArgs& p, int64_t token, int j0, int* at) {
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int v = j0 + j < p.top_k ? p.pos[token * p.top_k + j0 + j] : -1;
    at[j] = v >= 0 && v < p.rows ? v : -1;
  }
}

template <class T, class R, int LANES>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowsArgs p, int parts) {
  int64_t t;
  int c;
  if (!locate<LANES>(p, parts, &t, &c)) return;
  const F8 v = load8(static_cast<const T*>(p.tok) + t * p.hidden + c);
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    int at[kSlots];
    positions(p, t, j0, at);
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (at[j] >= 0)
        store8(static_cast<R*>(p.row_out) + static_cast<int64_t>(at[j]) * p.hidden + c, v);
  }
}

template <class T, class R, int LANES>
__global__ __launch_bounds__(kRowThreads) void combine_rows_kernel(RowsArgs p, int parts) {
  int64_t t;
  int c;
  if (!locate<LANES>(p, parts, &t, &c)) return;
  F8 sum{};
  if (p.base) sum = load8(static_cast<const T*>(p.base) + t * p.hidden + c);
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    int at[kSlots];
    positions(p, t, j0, at);
    F8 v[kSlots];
    float w[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      w[j] = 1.0f;
      if (at[j] < 0) continue;
      if (p.w) w[j] = p.w[t * p.top_k + j0 + j];
      v[j] = load8(static_cast<const R*>(p.row) + static_cast<int64_t>(at[j]) * p.hidden + c);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (at[j] >= 0)
#pragma unroll
        for (int q = 0; q < 8; ++q) sum.v[q] = fmaf(w[j], v[j].v[q], sum.v[q]);
  }
  store8(static_cast<T*>(p.tok_out) + t * p.hidden + c, sum);
}

// A block per token (of narrow rows, a wave): the dot products need whole rows.
// Lanes take columns in turn, their sums meet over the wave and then over the
// waves in order.
template <class T, class R, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void combine_grad_kernel(RowsArgs p) {
  __shared__ float sums[WAVES][kSlots];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    int at[kSlots];
    positions(p, t, j0, at);
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      dot[j] = 0.0f;
      w[j] = p.w && at[j] >= 0 ? p.w[t * p.top_k + j0 + j] : 1.0f;
    }
    for (int c = threadIdx.x * 8; c < p.hidden; c += 64 * WAVES * 8) {
      const F8 d = load8(static_cast<const T*>(p.tok) + t * p.hidden + c);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (at[j] < 0) continue;
        const int64_t i = static_cast<int64_t>(at[j]) * p.hidden + c;
        if (p.dw) {
          const F8 r = load8(static_cast<const R*>(p.row) + i);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot[j] = fmaf(d.v[q], r.v[q], dot[j]);
        }
        if (p.row_out) store8(static_cast<R*>(p.row_out) + i, scaled(d, w[j]));
      }
    }
    if (!p.dw) continue;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
      if (lane == 0) sums[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < p.top_k) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) v += sums[i][threadIdx.x];
      p.dw[t * p.top_k + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// One of the four pairs of types, and the lanes a token has.
template <class F>
void with_types(const RowsArgs& p, F f) {
  if (p.tok_f32) {
    if (p.row_f32) f(float{}, float{}); else f(float{}, uint16_t{});
  } else {
    if (p.row_f32) f(uint16_t{}, float{}); else f(uint16_t{}, uint16_t{});
  }
}

int lanes_of(int hidden) { return hidden > 256 ? 64 : hidden > 128 ? 32 : hidden > 64 ? 16 : 8; }

unsigned row_blocks(const RowsArgs& p, int lanes, int parts) {
  const int64_t waves = lanes == 64 ? p.tokens * parts : (p.tokens * lanes + 63) / 64;
  return static_cast<unsigned>((waves + kRowThreads / 64 - 1) / (kRowThreads / 64));
}

#define MOE_ROWS_LAUNCH(kernel)                                                          \
  const int lanes = lanes_of(p.hidden), parts = (p.hidden + 511) / 512;                  \
  const unsigned grid = row_blocks(p, lanes, parts);                                     \
  with_types(p, [&](auto t, auto r) {                                                    \
    using T = decltype(t);                                                               \
    using R = decltype(r);                                                               \
    switch (lanes) {                                                                     \
      case 64: kernel<T, R, 64><<<grid, kRowThreads, 0, stream>>>(p, parts); break;      \
      case 32: kernel<T, R, 32><<<grid, kRowThreads, 0, stream>>>(p, parts); break;      \
      case 16: kernel<T, R, 16><<<grid, kRowThreads, 0, stream>>>(p, parts); break;      \
      default: kernel<T, R, 8><<<grid, kRowThreads, 0, stream>>>(p, parts); break;       \
    }                                                                                    \
  });                                                                                    \
  return hipGetLastError()

}  // namespace

hipError_t launch_dispatch(const RowsArgs& p, hipStream_t stream) {
  if (p.tokens == 0 || p.rows == 0) return hipSuccess;
  MOE_ROWS_LAUNCH(dispatch_kernel);
}

hipError_t launch_combine_rows(const RowsArgs& p, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  MOE_ROWS_LAUNCH(combine_rows_kernel);
}

hipError_t launch_combine_grad(const RowsArgs& p, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>(p.tokens);
  with_types(p, [&](auto t, auto r) {
    using T = decltype(t);
    using R = decltype(r);
    if (p.hidden <= 512)
      combine_grad_kernel<T, R, 1><<<grid, 64, 0, stream>>>(p);
    else
      combine_grad_kernel<T, R, 4><<<grid, 256, 0, stream>>>(p);
  });
  return hipGetLastError();
}

}  // namespace moe

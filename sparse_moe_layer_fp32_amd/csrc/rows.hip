// Rows out to the experts and back, with weights, and their gradients.
//
//   dispatch          r[pos[t][j]] = x[t]
//   its gradient      dx[t] = base[t] + sum_j dr[pos[t][j]]
//   combine           y[t]  = base[t] + sum_j w[t][j] r[pos[t][j]]
//   its gradients     dr[pos[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], r[pos[t][j]]>
//
// Bound: HBM.  All four walk the tokens, so that a token's own row is read or
// written once, whatever top_k is, and every row of an expert once.  Sums are
// formed in fp32 in slot order.  A lane takes 8 columns of a token.  Bytes needed
// over time: 6.2 TB/s (sum over 8192 x 8 rows of 4096, base added: 109 us), 5.7
// (combine of 32768 x 8 pairs, half of them with rows, into fp32: 285 us; its
// gradients of 8191 x 3 rows of 7168: 147); a copy of 2 GiB 4.9.  Of few tokens,
// latency: 5 x 8 rows of 4096 2.5 us, combine of 64 x 8 3.6, its gradients 7.5, one
// after the other in a graph (alone 3.0 and 4.2, traced).

#include <algorithm>
#include <type_traits>

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

// The token and first column of this lane; false if there is none.  WHOLE: a wave
// has one token; else lanes take the chunks of all tokens one after the other.
template <bool WHOLE>
__device__ __forceinline__ bool locate(const RowsArgs& p, uint32_t parts, int64_t* token, int* col) {
  if (WHOLE) {
    const uint32_t wave = blockIdx.x * (kRowThreads / 64) +
                          __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t t = wave / parts;
    *token = t;
    *col = static_cast<int>((wave - t * parts) * 64 + (threadIdx.x & 63)) * 8;
  } else {
    const uint32_t chunk = blockIdx.x * kRowThreads + threadIdx.x;
    const uint32_t t = chunk / parts;
    *token = t;
    *col = static_cast<int>(chunk - t * parts) * 8;
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

// STREAM: with the non-temporal hint, on both sides (a constant: accesses that
// differ in the hint alone are merged without it).
template <bool STREAM, class E>
__device__ __forceinline__ F8 get8(const E* p) {
  return STREAM ? read8(p) : load8(p);
}
template <bool STREAM, class E>
__device__ __forceinline__ void put8(E* p, const F8& v) {
  if (STREAM)
    stream8(p, v);
  else
    store8(p, v);
}

template <class T, class R, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowsArgs p, uint32_t parts) {
  int64_t t;
  int c;
  if (!locate<WHOLE>(p, parts, &t, &c)) return;
  const F8 v = load8(static_cast<const T*>(p.tok) + t * p.hidden + c);
  for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
    int at[kSlots];
    positions(p, t, j0, at);
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (at[j] >= 0)
        put8<STREAM>(static_cast<R*>(p.row_out) + static_cast<int64_t>(at[j]) * p.hidden + c, v);
  }
}

template <class T, class R, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void combine_rows_kernel(RowsArgs p, uint32_t parts) {
  int64_t t;
  int c;
  if (!locate<WHOLE>(p, parts, &t, &c)) return;
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
      v[j] = get8<STREAM>(static_cast<const R*>(p.row) + static_cast<int64_t>(at[j]) * p.hidden + c);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (at[j] >= 0)
#pragma unroll
        for (int q = 0; q < 8; ++q) sum.v[q] = fmaf(w[j], v[j].v[q], sum.v[q]);
  }
  put8<STREAM>(static_cast<T*>(p.tok_out) + t * p.hidden + c, sum);
}

// SLOTS values of every lane summed over the wave: lane i gets value i % SLOTS.
// Each exchange halves the values a lane still holds, so that eight values take
// 10 exchanges and not 48.
template <int SLOTS>
__device__ __forceinline__ float wave_sums(const float* v, int lane) {
  float h[SLOTS];
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) h[i] = v[i];
#pragma unroll
  for (int n = SLOTS / 2; n >= 1; n /= 2) {  // n: the bit of the lane, and values left
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? h[i + n] : h[i], give = up ? h[i] : h[i + n];
      h[i] = keep + __shfl_xor(give, n);
    }
  }
#pragma unroll
  for (int off = SLOTS; off < 64; off <<= 1) h[0] += __shfl_xor(h[0], off);
  return h[0];
}

// WAVES waves per token: the dot products need whole rows.  Lanes take columns in
// turn, of all slots' rows at once, and their sums meet over the wave and then
// over the token's waves in order.  SLOTS: how many of a token's slots are taken
// together.
template <class T, class R, int WAVES, int SLOTS, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(RowsArgs p) {
  constexpr int TOKENS = kRowThreads / 64 / WAVES;  // per block
  __shared__ float sums[TOKENS][WAVES][SLOTS];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = wid / WAVES, wave = wid % WAVES;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TOKENS + token;
  const bool live = t < p.tokens;
  const T* const dy = static_cast<const T*>(p.tok) + t * p.hidden;
  for (int j0 = 0; j0 < p.top_k; j0 += SLOTS) {
    int64_t at[SLOTS];  // offset of the slot's row, -1 where there is none
    float w[SLOTS], dot[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const int64_t i = t * p.top_k + j0 + j;
      const int v = live && j0 + j < p.top_k ? p.pos[i] : -1;
      const bool have = v >= 0 && v < p.rows;
      at[j] = have ? static_cast<int64_t>(v) * p.hidden : -1;
      w[j] = p.w && have ? p.w[i] : 1.0f;
      dot[j] = 0.0f;
    }
    if (live)
      for (int c = (wave * 64 + lane) * 8; c < p.hidden; c += 64 * WAVES * 8) {
        const F8 d = load8(dy + c);
        F8 r[SLOTS];
        if (p.dw)
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (at[j] >= 0) r[j] = get8<STREAM>(static_cast<const R*>(p.row) + at[j] + c);
        if (p.row_out)
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (at[j] >= 0)
              put8<STREAM>(static_cast<R*>(p.row_out) + at[j] + c, scaled(d, w[j]));
        if (p.dw)
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (at[j] >= 0)
#pragma unroll
              for (int q = 0; q < 8; ++q) dot[j] = fmaf(d.v[q], r[j].v[q], dot[j]);
      }
    if (!p.dw) continue;
    float v = wave_sums<SLOTS>(dot, lane);
    if (WAVES > 1) {
      if (lane < SLOTS) sums[token][wave][lane] = v;
      __syncthreads();
      if (lane < SLOTS) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += sums[token][i][lane];
      }
      __syncthreads();
    }
    if (live && wave == 0 && lane < SLOTS && j0 + lane < p.top_k)
      p.dw[t * p.top_k + j0 + lane] = v;
  }
}

// One of the four pairs of types.
template <class F>
void with_types(const RowsArgs& p, F f) {
  if (p.tok_f32) {
    if (p.row_f32) f(float{}, float{}); else f(float{}, uint16_t{});
  } else {
    if (p.row_f32) f(uint16_t{}, float{}); else f(uint16_t{}, uint16_t{});
  }
}

// Sums of streamed rows are streamed too (8192 x 8 rows of 4096 into 67 MB: 100 us,
// from 109 with sums that stay; with a kernel that reads them at once 128, 130).
bool streams(const RowsArgs& p) {
  return rows_past_cache(p.tokens, p.rows, p.top_k, int64_t(p.hidden) * (p.row_f32 ? 4 : 2));
}

// Waves per token of the weights' gradient (us with 1 and 4, k = 8: 8192 x 256 20,
// 57; 8192 x 1024 66, 109; 1024 x 1024 12.3, 11.3; 8192 x 2048 149, 138; 64 x 4096
// 18.6, 8.6; 8192 x 4096 278, 234).
int grad_waves(const RowsArgs& p) {
  return p.hidden > 1024 || (p.hidden > 512 && p.tokens < 4096) ? 4 : 1;
}

template <class F>
void with_constant(bool v, F f) {
  if (v) f(std::true_type{}); else f(std::false_type{});
}

// Waves of one token each, or of narrow rows lanes packed.
#define MOE_ROWS_LAUNCH(kernel)                                                                 \
  const bool whole = p.hidden >= 512;                                                           \
  const int parts = whole ? (p.hidden + 511) / 512 : p.hidden / 8;                              \
  const int64_t threads = p.tokens * parts * (whole ? 64 : 1);                                  \
  const unsigned grid = static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads);       \
  with_types(p, [&](auto t, auto r) {                                                           \
    using T = decltype(t);                                                                      \
    using R = decltype(r);                                                                      \
    with_constant(streams(p), [&](auto s) {                                                     \
      constexpr bool S = decltype(s)::value;                                                    \
      if (whole)                                                                                \
        kernel<T, R, true, S><<<grid, kRowThreads, 0, stream>>>(p, parts);                      \
      else                                                                                      \
        kernel<T, R, false, S><<<grid, kRowThreads, 0, stream>>>(p, parts);                     \
    });                                                                                         \
  });                                                                                           \
  return hipGetLastError()

}  // namespace

// Rows that do not stay in the 256 MB last-level cache between their writer and
// their reader go past it (8192 x 8 rows of 4096, 537 MB: the sum over slots 108
// us, from 131, dispatch 109, from 118); others stay, whatever room the buffer has
// (1024 x 8, 67 MB: dispatch and a kernel that reads the rows 34.0 us, past the cache
// 39.1; the gradients 24.2 and 29.1; the sum by itself 14.7 either way).
bool rows_past_cache(int64_t tokens, int64_t rows, int top_k, int64_t row_bytes) {
  return std::min(rows, tokens * top_k) * row_bytes > (int64_t(256) << 20);
}

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
  const int waves = grad_waves(p);
  const unsigned grid = static_cast<unsigned>((p.tokens * waves + 3) / 4);
  with_types(p, [&](auto t, auto r) {
    using T = decltype(t);
    using R = decltype(r);
    with_constant(streams(p), [&](auto s) {
      constexpr bool S = decltype(s)::value;
      with_constant(p.top_k <= 4, [&](auto few) {
        constexpr int N = decltype(few)::value ? 4 : 8;
        if (waves == 1)
          combine_grad_kernel<T, R, 1, N, S><<<grid, kRowThreads, 0, stream>>>(p);
        else
          combine_grad_kernel<T, R, 4, N, S><<<grid, kRowThreads, 0, stream>>>(p);
      });
    });
  });
  return hipGetLastError();
}

}  // namespace moe

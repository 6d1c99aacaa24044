// SwiGLU between an expert's products, and its gradient.
//
//   gc = min(g, L), uc = clamp(u, -L, L) (L <= 0: no clamp), s = sigmoid(gc)
//   h  = gc s uc
//   dg = dh uc s (1 + gc (1 - s))  where g <= L, else 0
//   du = dh gc s                   where |u| <= L, else 0
// (llm-atlas Step-3.5-Flash card, raw field swiglu_limits: the clamp.)
//
// Bound: HBM.  One thread moves eight consecutive columns, 16 bytes of each
// operand, so a wave touches whole 128-byte lines; gate and up are read once
// and may be the two halves of one product's rows (row stride ld).

#include "activation.h"
#include "products.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <bool GRAD>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gate,
    const uint16_t* __restrict__ up, uint16_t* __restrict__ dgate, uint16_t* __restrict__ dup,
    uint16_t* __restrict__ h, int64_t rows, int chunks, int64_t ld, float limit) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = i / chunks;
  if (r >= rows) return;
  const int c = static_cast<int>(i - r * chunks) * 8;
  const int64_t at = r * ld + c, ath = r * 8 * chunks + c;
  const F8 g = load8(gate + at), u = load8(up + at);
  F8 hv, dg, du, d;
  if (GRAD) d = load8(dh + ath);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float gc = g.v[q], uc = u.v[q];
    bool gin = true, uin = true;
    if (limit > 0.0f) {  // comparisons, so that a NaN stays one
      gin = !(gc > limit);
      uin = !(fabsf(uc) > limit);
      gc = gin ? gc : limit;
      uc = uin ? uc : copysignf(limit, uc);
    }
    const float s = sigmoid_fast(gc);
    const float a = gc * s;
    hv.v[q] = a * uc;
    if (GRAD) {
      dg.v[q] = gin ? d.v[q] * uc * (s + a * (1.0f - s)) : 0.0f;
      du.v[q] = uin ? d.v[q] * a : 0.0f;
    }
  }
  if (!GRAD || h) store8(h + ath, hv);
  if (GRAD) {
    store8(dgate + at, dg);
    store8(dup + at, du);
  }
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* gate, const uint16_t* up, uint16_t* h, int64_t rows,
                         int inter, int64_t ld, float limit, hipStream_t stream) {
  const int64_t blocks = (rows * (inter / 8) + kThreads - 1) / kThreads;
  if (blocks <= 0) return hipSuccess;
  swiglu_kernel<false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      nullptr, gate, up, nullptr, nullptr, h, rows, inter / 8, ld, limit);
  return hipGetLastError();
}

hipError_t launch_swiglu_grad(const uint16_t* dh, const uint16_t* gate, const uint16_t* up,
                              uint16_t* dgate, uint16_t* dup, uint16_t* h, int64_t rows, int inter,
                              int64_t ld, float limit, hipStream_t stream) {
  const int64_t blocks = (rows * (inter / 8) + kThreads - 1) / kThreads;
  if (blocks <= 0) return hipSuccess;
  swiglu_kernel<true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      dh, gate, up, dgate, dup, h, rows, inter / 8, ld, limit);
  return hipGetLastError();
}

}  // namespace moe

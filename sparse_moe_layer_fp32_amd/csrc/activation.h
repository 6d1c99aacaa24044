// The activations of the linear product and their slopes, in fp32, and wide
// bf16 loads and stores.
#pragma once

#include "common.h"
#include "moe.h"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-v); v_exp_f32 and v_rcp_f32 are each about 1 ulp.  e^-v = inf
// for large negative v gives 0.
__device__ __forceinline__ float sigmoid_fast(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

// 1 - Phi(|v|) = erfc(|v| / sqrt 2) / 2, the upper tail of the standard normal
// distribution; *gauss gets e^(-v v / 2).  The tail is t poly(t) e^(-v v / 2)
// with t = 1 / (1 + 0.305 |v|), where t poly(t) = erfcx(|v| / sqrt 2) / 2 was
// fitted for its largest RELATIVE error over 0 <= |v| <= 13.5, 9.4e-8 (eight
// terms; seven: 7.8e-7), since for v < 0 the tail alone is the value of GELU.
// With fp32 roundings the tail is off by 5e-7 of itself up to |v| = 3 and by
// 8e-6 at 13 (the exponent's rounding, v v / 2 times 2^-24 and more).  15
// instructions; the library erfcf and the gaussian take 59, which the wide
// products' epilogues have no matrix work to hide behind (8192 x 4096 -> 11264
// with GELU: 658 us; 653 with the five terms of a formula for the absolute
// error, 4.7e-4 off at v = -4 and 2e-2 at -10).
__device__ __forceinline__ float normal_tail(float v, float* gauss) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.305f, 1.0f));
  float q = fmaf(0.03669919f, t, -0.15298831f);
  q = fmaf(q, t, 0.18571687f);
  q = fmaf(q, t, -0.0379768f);
  q = fmaf(q, t, 0.12102166f);
  q = fmaf(q, t, 0.10342087f);
  q = fmaf(q, t, 0.12246682f);
  q = fmaf(q, t, 0.12163974f);
  const float e = __builtin_amdgcn_exp2f(v * v * (-0.5f * kLog2e));
  *gauss = e;
  return q * t * e;
}

constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_RELU:
      return v < 0.0f ? 0.0f : v;  // NaN stays
    case MOE_ACT_GELU: {  // v Phi(v) = max(v, 0) - |v| (1 - Phi(|v|)); |v| capped so that
      float e;            // infinity times a tail of 0 stays 0
      return fmaxf(v, 0.0f) - fminf(fabsf(v), 1e18f) * normal_tail(v, &e);
    }
    case MOE_ACT_GELU_TANH:  // v (1 + tanh(q)) / 2 = v sigmoid(2 q)
      return v * sigmoid_fast(2.0f * kGeluC * v * fmaf(kGeluA * v, v, 1.0f));
    case MOE_ACT_SILU:
      return v * sigmoid_fast(v);
    default:
      return v;
  }
}

__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case MOE_ACT_RELU:
      return v > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_GELU: {
      float e;
      const float tail = normal_tail(v, &e);
      return fmaf(v * 0.39894228040143268f, e, v < 0.0f ? tail : 1.0f - tail);
    }
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoid_fast(2.0f * kGeluC * v * fmaf(kGeluA * v, v, 1.0f));
      // kept finite: s (1 - s) is 0 long before
      const float dq = fminf(2.0f * kGeluC * fmaf(3.0f * kGeluA * v, v, 1.0f), 1e30f);
      return s + v * s * (1.0f - s) * dq;
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid_fast(v);
      return s + v * s * (1.0f - s);
    }
    default:
      return 1.0f;
  }
}

// Eight consecutive values, bf16 (16 bytes) or fp32 (32 bytes).
struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack8(const u32x4& w) {
  F8 f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f.v[2 * q] = bf16_lo(w[q]);
    f.v[2 * q + 1] = bf16_hi(w[q]);
  }
  return f;
}
__device__ __forceinline__ F8 load8(const uint16_t* p) {
  return unpack8(*reinterpret_cast<const u32x4*>(p));
}
__device__ __forceinline__ F8 load8(const float* p) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
// The same with the non-temporal hint, for data that is read once.
__device__ __forceinline__ F8 read8(const uint16_t* p) {
  return unpack8(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}
__device__ __forceinline__ F8 read8(const float* p) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
// Rounds to nearest even with v_cvt_pk_bf16_f32 (NaN stays NaN).
__device__ __forceinline__ u32x4 pack8(const F8& f) {
  u32x4 w;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bf16x2 p{static_cast<__bf16>(f.v[2 * q]), static_cast<__bf16>(f.v[2 * q + 1])};
    w[q] = __builtin_bit_cast(uint32_t, p);
  }
  return w;
}
__device__ __forceinline__ void store8(uint16_t* p, const F8& f) {
  *reinterpret_cast<u32x4*>(p) = pack8(f);
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
}
__device__ __forceinline__ void stream8(float* p, const F8& f) {
  __builtin_nontemporal_store(f32x4{f.v[0], f.v[1], f.v[2], f.v[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{f.v[4], f.v[5], f.v[6], f.v[7]},
                              reinterpret_cast<f32x4*>(p) + 1);
}
__device__ __forceinline__ void stream8(uint16_t* p, const F8& f) {
  __builtin_nontemporal_store(pack8(f), reinterpret_cast<u32x4*>(p));
}

}  // namespace

}  // namespace moe

// Elementwise arithmetic of the epilogues: bf16 packing, GeLU, the gated
// activations and their derivatives.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/libtp.h"
#include "ptx_sm100.cuh"

namespace tp {

constexpr float kLog2e = 1.4426950408889634f;

// The standard normal distribution at x: Phi(x) = (1 + erf(x / sqrt 2)) / 2
// and phi(x) = exp(-x^2 / 2) / sqrt(2 pi), with erf by Abramowitz & Stegun,
// "Handbook of Mathematical Functions", formula 7.1.26: for z >= 0,
// erf z = 1 - t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-z^2),
// t = 1 / (1 + p z), |error| <= 1.5e-7, and erf(-z) = -erf z.  With
// z = |x| / sqrt 2 the factor exp(-z^2) is the exp(-x^2 / 2) of phi, so one
// reciprocal and one exponential give both.  GeLU(x) = x Phi(x) (the erf
// form) and GeLU'(x) = Phi(x) + x phi(x).  Two values at a time, on sm_100's
// two-wide fp32 instructions (each lane rounded as the one-wide form): on
// short-K GEMMs the epilogue's instruction issue, not the tensor core, sets
// the pace.
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }

__device__ __forceinline__ void normal_cdf_pdf2(float2 x, float2& cdf, float2& pdf) {
  const float2 z = __fmul2_rn(make_float2(fabsf(x.x), fabsf(x.y)), f2(0.70710678118654752f));
  const float2 d = __ffma2_rn(f2(0.3275911f), z, f2(1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  float2 p = __ffma2_rn(t, f2(1.061405429f), f2(-1.453152027f));
  p = __ffma2_rn(t, p, f2(1.421413741f));
  p = __ffma2_rn(t, p, f2(-0.284496736f));
  p = __ffma2_rn(t, p, f2(0.254829592f));
  const float2 poly = __fmul2_rn(t, p);
  const float2 arg = __fmul2_rn(__fmul2_rn(x, f2(-0.5f * kLog2e)), x);
  const float2 e = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));  // exp(-x^2 / 2)
  const float2 q = __fmul2_rn(__fmul2_rn(f2(0.5f), poly), e);         // (1 - erf z) / 2
  const float2 r = __fadd2_rn(f2(1.0f), make_float2(-q.x, -q.y));
  cdf = make_float2(x.x >= 0.0f ? r.x : q.x, x.y >= 0.0f ? r.y : q.y);
  pdf = __fmul2_rn(f2(0.39894228040143268f), e);
}

// GeLU on eight values, in pairs.
__device__ __forceinline__ void gelu8(float* x) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(x[i], x[i + 1]);
    float2 cdf, pdf;
    normal_cdf_pdf2(v, cdf, pdf);
    const float2 g = __fmul2_rn(v, cdf);
    x[i] = g.x;
    x[i + 1] = g.y;
  }
}

// x *= GeLU'(y) on eight values, in pairs; with hh, also hh = GeLU(y).
__device__ __forceinline__ void dgelu8(float* x, const float* y, float* hh) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(y[i], y[i + 1]);
    float2 cdf, pdf;
    normal_cdf_pdf2(v, cdf, pdf);
    if (hh != nullptr) {
      const float2 g = __fmul2_rn(v, cdf);
      hh[i] = g.x;
      hh[i + 1] = g.y;
    }
    const float2 r = __fmul2_rn(make_float2(x[i], x[i + 1]), __ffma2_rn(v, pdf, cdf));
    x[i] = r.x;
    x[i + 1] = r.y;
  }
}

// The gate's activation of two values and its derivative: SiLU x sigma(x),
// sigma(x) = 1 / (1 + exp(-x)), derivative sigma (1 + x (1 - sigma)); or the
// GeLU above.
__device__ __forceinline__ float2 gate_act2(float2 v, int act, float2& d) {
  float2 w;
  if (act == TP_ACT_SILU) {
    const float2 e = __fmul2_rn(v, f2(-kLog2e));
    const float2 q = __fadd2_rn(f2(1.0f), make_float2(ex2_approx(e.x), ex2_approx(e.y)));
    w = make_float2(rcp_approx(q.x), rcp_approx(q.y));
    d = __fmul2_rn(w, __ffma2_rn(v, __fadd2_rn(f2(1.0f), make_float2(-w.x, -w.y)), f2(1.0f)));
  } else {
    float2 pdf;
    normal_cdf_pdf2(v, w, pdf);
    d = __ffma2_rn(v, pdf, w);
  }
  return __fmul2_rn(v, w);
}

__device__ __forceinline__ float2 gate_act2(float2 v, int act) {
  float2 d;
  return gate_act2(v, act, d);
}

// The same on eight values; the derivative only with da.
__device__ __forceinline__ void gate_act8(const float* x, int act, float* av, float* da) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 d;
    const float2 r = gate_act2(make_float2(x[i], x[i + 1]), act, d);
    av[i] = r.x;
    av[i + 1] = r.y;
    if (da != nullptr) {
      da[i] = d.x;
      da[i + 1] = d.y;
    }
  }
}

// x *= u on eight values, in pairs.
__device__ __forceinline__ void mul8(float* x, const float* u) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 r = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(u[i], u[i + 1]));
    x[i] = r.x;
    x[i + 1] = r.y;
  }
}

// Backward of h = act(g) u on eight values: x = dh becomes dg = dh u act'(g);
// du = dh act(g); hh = h.
__device__ __forceinline__ void dglu8(float* x, const float* g, const float* u, int act, float* du,
                                      float* hh) {
  float da[8];
  gate_act8(g, act, hh, da);
#pragma unroll
  for (int i = 0; i < 8; ++i) du[i] = x[i] * hh[i];
  mul8(x, u);
  mul8(x, da);
  mul8(hh, u);
}

// x += b on eight values, in pairs.
__device__ __forceinline__ void add8(float* x, const float* b) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 r = __fadd2_rn(make_float2(x[i], x[i + 1]), make_float2(b[i], b[i + 1]));
    x[i] = r.x;
    x[i + 1] = r.y;
  }
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(p[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  return u;
}

constexpr float kF16Max = 65504.0f;

// fp16 is spaced 2^-24 apart below 2^-14, so where the largest of 32 neighbouring
// values is below 2^-17, what is kept of it is coarser than bf16 (half a step,
// 2^-25, is over 2^-8 of it).  Zeros are kept exactly.
constexpr float kF16Small = 7.62939453125e-6f;
__device__ __forceinline__ bool f16_too_small(float largest) {
  return largest > 0.0f && largest < kF16Small;
}
__device__ __forceinline__ float absmax8(const float* f, float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// Eight fp32 values to fp16, saturated to the finite range; returns whether
// any finite value had to be clamped.
__device__ __forceinline__ uint4 pack8_f16(float* f, bool& clamped) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (fabsf(f[i]) > kF16Max) {
      clamped = true;
      f[i] = copysignf(kF16Max, f[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  return u;
}

// Eight fp32 values as two bf16 terms: the rounded values and the rounded rests
// (16 mantissa bits together, the range of fp32).
__device__ __forceinline__ uint4 split8(const float* f, uint4& rest) {
  const uint4 hi = pack8(f);
  float h[8], r[8];
  unpack8(hi, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = isinf(h[i]) ? 0.0f : f[i] - h[i];
  rest = pack8(r);
  return hi;
}

// Eight fp16 values as fp32.
__device__ __forceinline__ void unpack8_f16(const uint4& u, float* f) {
  const __half2* p = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(p[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

}  // namespace tp

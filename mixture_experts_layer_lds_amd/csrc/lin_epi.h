// The dense projection's epilogue (bias, activation, residual, saved pre-activation), shared by the
// kernels of linear.hip and those on 4-bit weights.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

enum { LIN_NONE = 0, LIN_RELU = 1, LIN_GELU = 2, LIN_SILU = 3, LIN_SWIGLU = 4 };

// The normal distribution's upper tail at x = |z| and, through *e, exp(-x^2 / 2):
// tail(x) = t P(t) exp(-x^2 / 2), t = 1 / (1 + p x), P the polynomial whose largest relative error
// against erfcx(x / sqrt 2) / (2 t) is least for 0 <= x <= 14.5, where the exponential underflows
// (found by reweighted least squares): 3.2e-8 in degree 8, 4.7e-6 in degree 5.  The error stays relative
// to the tail, so GELU keeps its leading digits for negative z too, where 1 + erf cancels: in degree
// 8 6e-7 of the value down to -3 and 3e-6 at -8 (the exponent's rounding), at most 2.4e-7 in all.
// BRIEF, degree 5, is for results that are rounded to bf16 next, half a step of which is 400 times its
// error: 8192 x 14336 x 256 with GELU takes 144 us with it and 157 with degree 8, 8192 x 14336 x 4096 with
// bias and Z kept 766 and 772.
template <bool BRIEF>
__device__ __forceinline__ float normal_tail(float z, float* e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), BRIEF ? 0.31f : 0.35f, 1.0f));
  *e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);
  float p;
  if constexpr (BRIEF) {
    p = -0.07392915311f;
    p = fmaf(p, t, 0.18045038015f);
    p = fmaf(p, t, 0.01574467415f);
    p = fmaf(p, t, 0.13342980380f);
    p = fmaf(p, t, 0.12044127104f);
    p = fmaf(p, t, 0.12386070275f);
  } else {
    p = -0.02915787324f;
    p = fmaf(p, t, 0.14403086901f);
    p = fmaf(p, t, -0.25583893061f);
    p = fmaf(p, t, 0.15931960940f);
    p = fmaf(p, t, -0.02321228944f);
    p = fmaf(p, t, 0.10555247962f);
    p = fmaf(p, t, 0.11982129514f);
    p = fmaf(p, t, 0.13986350596f);
    p = fmaf(p, t, 0.13962130249f);
  }
  return p * t * *e;
}

// act(z) of one element (not SwiGLU).  GELU is the exact form
// z Phi(z) = max(z, 0) - |z| tail(|z|).  T: the type that the result is rounded to.
template <int ACT, typename T>
__device__ __forceinline__ float lin_act1(float z) {
  if constexpr (ACT == LIN_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays
  if constexpr (ACT == LIN_GELU) {
    float e;
    const float q = normal_tail<sizeof(T) == 2>(z, &e);
    return fmaf(q != 0.0f ? -fabsf(z) : 0.0f, q, z < 0.0f ? 0.0f : z);  // (infinity times a tail of 0 is 0)
  }
  if constexpr (ACT == LIN_SILU) return z * sigmoid_f32(z);
  return z;
}
// dy act'(z).  ReLU selects: where its unit is off, dy adds nothing even if it is infinite or NaN.
template <int ACT>
__device__ __forceinline__ float lin_bwd1(float dy, float z) {
  if constexpr (ACT == LIN_RELU) return z > 0.0f ? dy : 0.0f;
  if constexpr (ACT == LIN_GELU) {
    float e;
    const float q = normal_tail<false>(z, &e);  // (bound by memory; dbias is fp32)
    return dy * ((z < 0.0f ? q : 1.0f - q) + (e != 0.0f ? z : 0.0f) * e * 0.39894228040143268f);
  }
  if constexpr (ACT == LIN_SILU) {
    const float s = sigmoid_f32(z);
    return dy * (s * (1.0f + z * (1.0f - s)));
  }
  return dy;
}
// f(integral_constant<int, act>) for the activation act (SwiGLU as NONE: it is not elementwise).
template <class F>
__device__ __forceinline__ void lin_by_act(int act, F f) {
  if (act == LIN_RELU) f(std::integral_constant<int, LIN_RELU>{});
  else if (act == LIN_GELU) f(std::integral_constant<int, LIN_GELU>{});
  else if (act == LIN_SILU) f(std::integral_constant<int, LIN_SILU>{});
  else f(std::integral_constant<int, LIN_NONE>{});
}
template <typename T, int N>
__device__ __forceinline__ void lin_act(float* z, int act) {
  lin_by_act(act, [&](auto A) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] = lin_act1<decltype(A)::value, T>(z[u]);
  });
}

// What the epilogue does with z [m][n]; pointers may be null, res may be out.
template <typename T>
struct LinEpi {
  const float* bias;
  const T* res;
  int64_t ldr;
  T* Z;
  int64_t ldz;
  T* out;
  int64_t ldo;
  int act;
};

// Four consecutive elements of T as fp32.
template <typename T> __device__ __forceinline__ f32x4 lin_ld4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const f32x4*>(p);
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
                 __uint_as_float(v[1] & 0xffff0000u)};
  }
}
template <typename T> __device__ __forceinline__ void lin_st4(T* p, f32x4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4*>(p) = v;
  else *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// The epilogue of four consecutive columns c of row r: z is z there (bias not yet added), for
// SwiGLU the gate's, zu the up projection's.
template <typename T>
__device__ __forceinline__ void lin_epi4(const LinEpi<T>& ep, int64_t r, int c, int n, bool glu, f32x4 z, f32x4 zu) {
  if (ep.bias) {
    z += *reinterpret_cast<const f32x4*>(ep.bias + c);
    if (glu) zu += *reinterpret_cast<const f32x4*>(ep.bias + n + c);
  }
  if (ep.Z) {
    lin_st4(ep.Z + r * ep.ldz + c, z);
    if (glu) lin_st4(ep.Z + r * ep.ldz + n + c, zu);
  }
  float f[4] = {z[0], z[1], z[2], z[3]};
  if (glu) {
#pragma unroll
    for (int u = 0; u < 4; ++u) f[u] = f[u] * sigmoid_f32(f[u]) * zu[u];
  } else {
    lin_act<T, 4>(f, ep.act);
  }
  f32x4 o = {f[0], f[1], f[2], f[3]};
  if (ep.res) o += lin_ld4(ep.res + r * ep.ldr + c);
  lin_st4(ep.out + r * ep.ldo + c, o);
}

// Adds SK partial products [SK][m][np] in slice order and applies the epilogue (linear.hip); np: n, or 2 n for
// SwiGLU.
hipError_t launch_lin_finish(const float* part, int SK, int m, int n, int np, const LinEpi<bf16>& ep, hipStream_t st);

}  // namespace moe

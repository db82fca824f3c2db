// activation.cuh -- the gated units' functions: silu, gelu and their derivatives.
#pragma once

#include "net_common.cuh"

namespace gs {

// 2^v and 1 / v as the hardware's single instructions; results and arguments below
// 2^-126 count as zero, which is below the error of every use here.
__device__ __forceinline__ float power2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Phi and its density for two values.  16-bit types take Abramowitz and Stegun's formula
// 7.1.26 for the error function, which needs the one exponential that the derivative has
// too; in this arithmetic Phi is off by up to 2.6e-7, a thousandth of fp16's rounding of
// values near 1 (in the tail, where Phi is small, by up to a third of itself: below that
// rounding of v Phi's terms).  It takes two values an instruction (gated units of 8160 x
// 1361 fp16: 72 us, 75 without).  The same elsewhere in these kernels costs the aligned form registers, and
// thereby warps: 238 us in place of 230 at 32640 x 2816 bf16.  fp32 takes the complementary
// error function, which keeps its relative accuracy in the tail.
struct Phi {
  float2 p, density;  // Phi(v), phi(v)
};
template <typename T>
__device__ __forceinline__ Phi normal(float2 v) {
  if constexpr (sizeof(T) == 4) {
    const float2 w = mul2(mul2(v, v), both(-0.72134752044448170f));  // -v^2 / 2 in powers of two
    return Phi{make_float2(0.5f * erfcf(v.x * -0.70710678118654752f),
                           0.5f * erfcf(v.y * -0.70710678118654752f)),
               mul2(make_float2(power2(w.x), power2(w.y)), both(0.39894228040143268f))};
  } else {
    const float2 z = make_float2(fabsf(v.x) * 0.70710678118654752f, fabsf(v.y) * 0.70710678118654752f);
    const float2 y = fma2(both(0.3275911f), z, both(1.f));
    const float2 t = make_float2(reciprocal(y.x), reciprocal(y.y));
    const float2 w = mul2(mul2(z, z), both(-1.4426950408889634f));
    const float2 ex = make_float2(power2(w.x), power2(w.y));
    float2 q = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
    q = fma2(q, t, both(0.5f * 1.421413741f));
    q = fma2(q, t, both(0.5f * -0.284496736f));
    q = fma2(q, t, both(0.5f * 0.254829592f));
    const float2 tail = mul2(mul2(q, t), ex), rest = fma2(tail, both(-1.f), both(1.f));
    return Phi{make_float2(v.x < 0.f ? tail.x : rest.x, v.y < 0.f ? tail.y : rest.y),
               mul2(ex, both(0.39894228040143268f))};
  }
}
// act(v) and its derivative for two values.
__device__ __forceinline__ float sigmoid(float v) {
  return reciprocal(1.f + power2(v * -1.4426950408889634f));
}
template <typename T, int ACT>
__device__ __forceinline__ float2 act_value(float2 v) {
  if (ACT == GS_ACT_SILU) return make_float2(v.x * sigmoid(v.x), v.y * sigmoid(v.y));
  return mul2(v, normal<T>(v).p);
}
template <typename T, int ACT>
__device__ __forceinline__ void act_both(float2 v, float2& f, float2& df) {
  if (ACT == GS_ACT_SILU) {
    const float s = sigmoid(v.x), u = sigmoid(v.y);
    f = make_float2(v.x * s, v.y * u);
    df = make_float2(s * (1.f + v.x * (1.f - s)), u * (1.f + v.y * (1.f - u)));
  } else {
    const Phi n = normal<T>(v);
    f = mul2(v, n.p);
    df = fma2(v, n.density, n.p);
  }
}

}  // namespace gs

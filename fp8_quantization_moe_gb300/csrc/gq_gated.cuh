// gq_gated.cuh -- the activations of the gated feed-forward block, and what
// its kernels share.  With the projections x (gate) and u (up) of a row,
//     act(x)  = x * sigma(z),        h = act(x) * u
//     act'(x) = sigma(z) + x * sigma(z) * (1 - sigma(z)) * dz/dx
// where sigma is the logistic function and z = x (a + b x^2): a = 1, b = 0
// gives silu, a = 2 sqrt(2 / pi), b = 0.044715 a the tanh form of gelu, since
// 0.5 (1 + tanh(y)) = sigma(2 y).
#pragma once

#include "gq_fp8.h"
#include "gq_tcgen05.cuh"

namespace gq {
namespace gated {

struct Act {
  float a, b;
};

inline Act act_of(int activation) {
  const float a = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  return activation == GQ_ACT_GELU ? Act{a, a * 0.044715f} : Act{1.0f, 0.0f};
}

// z(x).  The square is held at 2^100, where sigma is 0 or 1 in any case, so
// that no product of an infinity and a zero arises.
__device__ __forceinline__ float act_z(Act p, float x) {
  return x * __fmaf_rn(p.b, fminf(x * x, 0x1p100f), p.a);
}

// sigma(z).  The reciprocal is within one unit in the last place; past exp's
// overflow it gives 0.
__device__ __forceinline__ float sigma(float z) { return rcp_approx(1.0f + expf(-z)); }

// x := act(x) * u for several values, two at a time, with sigma from the
// hardware's power of two, whose argument adds |z| 2^-23: for values that are
// sums of rounded products anyway.  a x + b x^3 may overflow to the infinity that
// it stands for; x is held at fp32's lowest value, so that an infinity times a
// vanished sigma is no NaN (a NaN comes through sigma).
// Measured, 38,000 rows, K 224 to N 3680, gelu to fp8: 204 us, of which 70 are
// this; one value at a time 231; a reciprocal shared by two values, against the
// special function unit's 16 results a cycle, with a branch for the far ones, 274.
template <int kN>
__device__ __forceinline__ void gate(Act p, float (&x)[kN], const float (&u)[kN]) {
  const float a = p.a * -1.4426950408889634f, b = p.b * -1.4426950408889634f;
#pragma unroll
  for (int j = 0; j < kN; j += 2) {
    float k[2] = {a, a}, z[2], e[2], d[2], s[2];
    if (b != 0.0f) {
      float q[2];
      mul2(q[0], q[1], x[j], x[j + 1], x[j], x[j + 1]);
      fma2(k[0], k[1], __float_as_uint(q[0]), __float_as_uint(q[1]), b);
    }
    mul2(z[0], z[1], x[j], x[j + 1], k[0], k[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(z[i]));
    add2(d[0], d[1], e[0], e[1], 1.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] = rcp_approx(d[i]);
    mul2(s[0], s[1], s[0], s[1], fmaxf(x[j], -0x1.fffffep127f), fmaxf(x[j + 1], -0x1.fffffep127f));
    mul2(x[j], x[j + 1], s[0], s[1], u[j], u[j + 1]);
  }
}

// act(x) from x and sigma(z): its limit 0 where sigma has vanished.
__device__ __forceinline__ float act_value(float x, float s) { return s == 0.0f ? 0.0f : x * s; }

// act'(x): sigma(z) alone where sigma (1 - sigma) has vanished.
__device__ __forceinline__ float act_slope(Act p, float x, float s) {
  const float t = s * (1.0f - s);
  const float dz = __fmaf_rn(3.0f * p.b, fminf(x * x, 0x1p100f), p.a);
  return t == 0.0f ? s : __fmaf_rn(x * t, dz, s);
}

}  // namespace gated
}  // namespace gq

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

// The same from the hardware's power of two, whose argument adds |z| 2^-23: for
// values that are sums of rounded products anyway.
__device__ __forceinline__ float sigma_approx(float z) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  return rcp_approx(1.0f + e);
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

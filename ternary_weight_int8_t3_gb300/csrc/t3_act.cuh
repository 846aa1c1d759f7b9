// t3_act.cuh -- the activations of an epilogue and their derivatives, and what
// an epilogue takes besides the product.
#pragma once
#include <cstdint>

#include "t3.h"

namespace t3 {

// z = (x row_scale) col_scale + bias, pre = z, out = act(z) + residual; any
// pointer may be null.
struct EpilogueArgs {
  const float *row_scale, *col_scale, *bias;
  const void* residual;
  void* pre;
  int act;
};

// Two products over one A (0: the gate's, 1: the other's): z_i = (x_i row_scale) scale_i +
// bias_i, pre_i = z_i, out = act(z_0) z_1; any pointer may be null.
struct GluArgs {
  const float* row_scale;
  const float *scale[2], *bias[2];
  void* pre[2];
  int act;
};

namespace vec {

// The logistic function from one exponential that cannot overflow, with
// e = exp(-|z|) and r = 1 / (1 + e):
//   sigmoid(z) = r for z >= 0 and e r below, sigmoid(-z) the other one,
//   sigmoid(z) sigmoid(-z) = e r r;
// each keeps its relative precision however far z is from zero.
struct Logistic {
  float pos, neg, slope;  // sigmoid(z), sigmoid(-z), their product
};
// exp2 and the reciprocal are the hardware's approximations (2 ulp and 1 ulp),
// results below the float range flushed to 0.
__device__ __forceinline__ Logistic logistic(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * fabsf(z)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  const float er = e * r;
  Logistic s;
  s.pos = z >= 0.0f ? r : er;
  s.neg = z >= 0.0f ? er : r;
  s.slope = er * r;
  return s;
}

// Activation ACT of z, and its derivative.  GELU is the tanh form written as
// z sigmoid(2 u) with u = sqrt(2 / pi) (z + 0.044715 z^3), since
// (1 + tanh u) / 2 = sigmoid(2 u).
constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(z) alone, as 1 / (1 + exp(-z)): 0 once the exponential is infinite.
__device__ __forceinline__ float sigmoid_scaled(float minus_z_log2e) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(minus_z_log2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == T3_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == T3_ACT_RELU2) return z < 0.0f ? 0.0f : z * z;
  if constexpr (ACT == T3_ACT_SILU) return z * sigmoid_scaled(-kLog2e * z);
  if constexpr (ACT == T3_ACT_GELU) return z * sigmoid_scaled(z * fmaf(-kLog2e * kGeluC * kGeluA, z * z, -kLog2e * kGeluC));
  return z;
}

__device__ __forceinline__ float act_any(float z, int kind) {
  switch (kind) {
    case T3_ACT_RELU: return act<T3_ACT_RELU>(z);
    case T3_ACT_RELU2: return act<T3_ACT_RELU2>(z);
    case T3_ACT_SILU: return act<T3_ACT_SILU>(z);
    case T3_ACT_GELU: return act<T3_ACT_GELU>(z);
    default: return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == T3_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == T3_ACT_RELU2) return z < 0.0f ? 0.0f : 2.0f * z;
  if constexpr (ACT == T3_ACT_SILU) {
    const Logistic s = logistic(z);
    return s.slope == 0.0f ? s.pos : fmaf(z, s.slope, s.pos);  // far out: no infinity times zero
  }
  if constexpr (ACT == T3_ACT_GELU) {
    const float z2 = z * z;
    const Logistic s = logistic(kGeluC * z * fmaf(kGeluA, z2, 1.0f));
    return s.slope == 0.0f ? s.pos
                           : fmaf(z * s.slope, kGeluC * fmaf(3.0f * kGeluA, z2, 1.0f), s.pos);
  }
  return 1.0f;
}

}  // namespace vec
}  // namespace t3

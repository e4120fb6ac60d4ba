// Activations and their slopes in fp32 (the codes are gptq_act's).
#pragma once
#include "gptq.h"

#include <hip/hip_runtime.h>

namespace gq {

// 1 / (1 + exp(-x)) within a few ulps; exp's overflow gives 0.
__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi): 1 + tanh(v) = 2 sigmoid(2 v)
constexpr float kGeluB = 0.044715f;

// Phi(z), the normal distribution function.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case GPTQ_ACT_RELU: return z < 0.f ? 0.f : z;          // NaN stays
    case GPTQ_ACT_GELU: return z * normal_cdf(z);
    case GPTQ_ACT_GELU_TANH: return z * sigmoid_f32(kGeluA * z * fmaf(kGeluB * z, z, 1.f));
    case GPTQ_ACT_SILU: return z * sigmoid_f32(z);
    default: return z;
  }
}

// Value and slope. The slopes' factors are formed of z cut to +-64, where all
// of them have reached 0 or 1 in fp32: no product of an infinity and 0.
__device__ __forceinline__ float act_both(int act, float z, float& slope) {
  const float c = fabsf(z) > 64.f ? copysignf(64.f, z) : z;
  switch (act) {
    case GPTQ_ACT_RELU:
      slope = z > 0.f ? 1.f : (z == z ? 0.f : z);
      return z < 0.f ? 0.f : z;
    case GPTQ_ACT_GELU: {
      // Phi(-|z|) = erfc(|z| / sqrt 2) / 2 by formula 7.1.26 of Abramowitz and
      // Stegun (erfc within 1.5e-7), which shares its exponential with the slope
      const float a = fabsf(c), e = __expf(-0.5f * a * a);
      const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678118654752f, a, 1.f));
      const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                               0.254829592f);
      const float tail = 0.5f * q * e, p = z < 0.f ? tail : 1.f - tail;
      slope = fmaf(c * 0.3989422804014327f, e, p);
      return z * p;
    }
    case GPTQ_ACT_GELU_TANH: {
      const float s = sigmoid_f32(kGeluA * z * fmaf(kGeluB * z, z, 1.f));
      slope = fmaf(c * s * (1.f - s) * kGeluA, fmaf(3.f * kGeluB * c, c, 1.f), s);
      return z * s;
    }
    case GPTQ_ACT_SILU: {
      const float s = sigmoid_f32(z);
      slope = fmaf(c * s, 1.f - s, s);
      return z * s;
    }
    default:
      slope = 1.f;
      return z;
  }
}

}  // namespace gq

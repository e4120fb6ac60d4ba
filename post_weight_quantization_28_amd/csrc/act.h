// Activations and their slopes in fp32 (the codes are gptq_act's).
#pragma once
#include "gptq.h"

#include <hip/hip_runtime.h>

namespace gq {

// 1 / (1 + exp(-x)), relative to itself within 8 2^-24 for positive x and (1.3 |x| +
// 8) 2^-24 for negative ones (the rounding of x log2 e is absolute in the exponent);
// exp's overflow gives 0.
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
      // Phi(-|z|) = erfc(|z| / sqrt 2) / 2 with an exponential that the slope needs
      // too: exp(x^2) erfc(x) is t times a polynomial in t = 1 / (1 + 0.3925 x)
      // within 1.1e-7 of itself for all x up to 46 (fitted to the least largest
      // relative error; 5e-7 in fp32), so that the tail is as good as the middle.
      const float a = fabsf(c), e = __expf(-0.5f * a * a);
      const float t = __builtin_amdgcn_rcpf(fmaf(0.3925f * 0.70710678118654752f, a, 1.f));
      float q = fmaf(t, 0.052698649466f, -0.207043841481f);
      q = fmaf(t, q, 0.226035580039f);
      q = fmaf(t, q, -0.043806929141f);
      q = fmaf(t, q, 0.161438837647f);
      q = fmaf(t, q, 0.162571072578f);
      q = fmaf(t, q, 0.205268085003f);
      q = fmaf(t, q, 0.221392959356f);
      q = t * fmaf(t, q, 0.22144556046f);
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

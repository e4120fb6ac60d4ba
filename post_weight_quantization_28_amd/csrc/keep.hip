// Activations kept in 8 bits for the backward pass.
//
// A group is 32 consecutive columns of one row (the last group of a row may
// be short). With amax the group's largest magnitude, 2^p <= amax < 2^(p+1),
// the step is 2^(p - 6) (p at least -120), and
//   c = clamp(rint(x / step), -127, 127)   (round half to even),
//   x_hat = c step:
// |x - x_hat| <= step / 2 <= amax / 128, except that a value within half a
// step of 2^(p+1) is off by up to a whole step. The step is kept as its
// fp32 exponent field, one byte (1..248). A power of two costs up to one of
// the eight bits against amax / 127, and buys that x_hat has at most 7
// significant bits: it is exact in bf16, so the matrix cores form the
// weight gradient from the kept values without another rounding
// (experts.hip), and scaling by the step is exact everywhere. The byte 255
// marks a group that held an infinity or a NaN: its codes are 0 and all its
// values come back as NaN, so that such a step cannot pass unnoticed.
//
// Rows are kept at a pitch of 32 ceil(n / 32) codes, the columns past n as
// zeros. Both kernels are bound by memory; a thread moves 8 columns (16
// bytes of bf16), the four threads of a group share its maximum by two
// lane exchanges.
#include "common.h"
#include "dma.h"

namespace gq {

typedef unsigned int kp_u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int kp_u32x2_t __attribute__((ext_vector_type(2)));
typedef float kp_f32x4_t __attribute__((ext_vector_type(4)));

template <bool BF, bool VEC>
__device__ __forceinline__ void kp_load8(const void* X, int64_t off, int nc, float (&v)[8]) {
  if (VEC && nc == 8) {
    if constexpr (BF) {
      const kp_u32x4_t u = *reinterpret_cast<const kp_u32x4_t*>(static_cast<const uint16_t*>(X) + off);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const float* p = static_cast<const float*>(X) + off;
      const kp_f32x4_t a = *reinterpret_cast<const kp_f32x4_t*>(p);
      const kp_f32x4_t b = *reinterpret_cast<const kp_f32x4_t*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i < nc)
        v[i] = BF ? bf16_to_f32(static_cast<const uint16_t*>(X)[off + i]) : static_cast<const float*>(X)[off + i];
    }
  }
}

template <bool BF, bool VEC>
__global__ void __launch_bounds__(256)
k_keep_save(const void* __restrict__ X, int64_t ldx, int64_t T, int64_t n, int64_t units,
            int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // units is a multiple of 4
  const bool in = i < T * units;
  const int64_t t = in ? i / units : 0, u = in ? i - t * units : 0;
  const int64_t c = 8 * u;
  const int nc = in ? (int)max((int64_t)0, min((int64_t)8, n - c)) : 0;
  float v[8];
  kp_load8<BF, VEC>(X, t * ldx + c, nc, v);
  // magnitudes compare as integers; an infinity or NaN has the field 255
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  if (!in) return;
  const int field = (int)(top >> 23);
  const int byte = field == 255 ? 255 : max(field - 6, 1);
  // 1 / step = 2^(127 - byte) in two factors, both normal; products with a
  // power of two are exact unless they underflow, and such values round to 0
  const int up = 127 - byte;
  const int a = up >> 1;
  const float f1 = __uint_as_float((uint32_t)(127 + a) << 23);
  const float f2 = __uint_as_float((uint32_t)(127 + up - a) << 23);
  uint32_t w[2] = {0u, 0u};
  if (byte != 255) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fminf(fmaxf(rintf(v[e] * f1 * f2), -127.f), 127.f);
      w[e >> 2] |= ((uint32_t)(int)r & 0xFFu) << (8 * (e & 3));
    }
  }
  *reinterpret_cast<kp_u32x2_t*>(codes + t * (8 * units) + c) = (kp_u32x2_t){w[0], w[1]};
  if ((u & 3) == 0) exps[t * (units / 4) + (u >> 2)] = (uint8_t)byte;
}

template <bool BF, bool VEC>
__global__ void __launch_bounds__(256)
k_keep_restore(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t T, int64_t n,
               int64_t units, void* __restrict__ X, int64_t ldx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * units) return;
  const int64_t t = i / units, u = i - t * units, c = 8 * u;
  const int nc = (int)max((int64_t)0, min((int64_t)8, n - c));
  const kp_u32x2_t w = *reinterpret_cast<const kp_u32x2_t*>(codes + t * (8 * units) + c);
  const uint32_t b = exps[t * (units / 4) + (u >> 2)];
  const float step = __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * step;
  if (VEC && nc == 8) {
    if constexpr (BF) {
      kp_u32x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j)   // exact in bf16: the low halves are zero
        o[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xFFFF0000u);
      *reinterpret_cast<kp_u32x4_t*>(static_cast<uint16_t*>(X) + t * ldx + c) = o;
    } else {
      float* p = static_cast<float*>(X) + t * ldx + c;
      *reinterpret_cast<kp_f32x4_t*>(p) = (kp_f32x4_t){v[0], v[1], v[2], v[3]};
      *reinterpret_cast<kp_f32x4_t*>(p + 4) = (kp_f32x4_t){v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nc) {
        if constexpr (BF) static_cast<uint16_t*>(X)[t * ldx + c + e] = (uint16_t)(__float_as_uint(v[e]) >> 16);
        else static_cast<float*>(X)[t * ldx + c + e] = v[e];
      }
  }
}

static bool kp_aligned(const void* p, int64_t ld, int esize) {
  return ((uintptr_t)p & 15) == 0 && (ld * esize) % 16 == 0;
}

hipError_t launch_keep_save(hipStream_t s, const void* X, int bf16, int64_t T, int64_t n, int64_t ldx,
                            int8_t* codes, uint8_t* exps) {
  if (T <= 0 || n <= 0) return hipSuccess;
  const int64_t units = 4 * ceil_div(n, 32);
  const dim3 grid((unsigned)ceil_div(T * units, 256)), block(256);
  const bool vec = kp_aligned(X, ldx, bf16 ? 2 : 4);
  if (bf16 && vec) hipLaunchKernelGGL((k_keep_save<true, true>), grid, block, 0, s, X, ldx, T, n, units, codes, exps);
  else if (bf16) hipLaunchKernelGGL((k_keep_save<true, false>), grid, block, 0, s, X, ldx, T, n, units, codes, exps);
  else if (vec) hipLaunchKernelGGL((k_keep_save<false, true>), grid, block, 0, s, X, ldx, T, n, units, codes, exps);
  else hipLaunchKernelGGL((k_keep_save<false, false>), grid, block, 0, s, X, ldx, T, n, units, codes, exps);
  return hipGetLastError();
}

hipError_t launch_keep_restore(hipStream_t s, const int8_t* codes, const uint8_t* exps, int64_t T, int64_t n,
                               void* X, int bf16, int64_t ldx) {
  if (T <= 0 || n <= 0) return hipSuccess;
  const int64_t units = 4 * ceil_div(n, 32);
  const dim3 grid((unsigned)ceil_div(T * units, 256)), block(256);
  const bool vec = kp_aligned(X, ldx, bf16 ? 2 : 4);
  if (bf16 && vec) hipLaunchKernelGGL((k_keep_restore<true, true>), grid, block, 0, s, codes, exps, T, n, units, X, ldx);
  else if (bf16) hipLaunchKernelGGL((k_keep_restore<true, false>), grid, block, 0, s, codes, exps, T, n, units, X, ldx);
  else if (vec) hipLaunchKernelGGL((k_keep_restore<false, true>), grid, block, 0, s, codes, exps, T, n, units, X, ldx);
  else hipLaunchKernelGGL((k_keep_restore<false, false>), grid, block, 0, s, codes, exps, T, n, units, X, ldx);
  return hipGetLastError();
}

}  // namespace gq

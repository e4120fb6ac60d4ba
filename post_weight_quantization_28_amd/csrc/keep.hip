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
typedef kp_u32x4_t kp_u32x4_any_t __attribute__((aligned(2)));
typedef kp_f32x4_t kp_f32x4_any_t __attribute__((aligned(4)));

// Whole units move in 16-byte pieces at any alignment (VEC: rows that are
// 16-byte aligned), a row's last columns one by one. 8192 rows of 1915 bf16
// columns: save 23 us column by column, 12 in pieces, restore 23 and 10.

template <bool BF, bool VEC>
__device__ __forceinline__ void kp_load8(const void* X, int64_t off, int nc, float (&v)[8]) {
  if (nc == 8) {
    if constexpr (BF) {
      const uint16_t* p = static_cast<const uint16_t*>(X) + off;
      kp_u32x4_t u;
      if constexpr (VEC) u = *reinterpret_cast<const kp_u32x4_t*>(p);
      else u = *reinterpret_cast<const kp_u32x4_any_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const float* p = static_cast<const float*>(X) + off;
      kp_f32x4_t a, b;
      if constexpr (VEC) {
        a = *reinterpret_cast<const kp_f32x4_t*>(p);
        b = *reinterpret_cast<const kp_f32x4_t*>(p + 4);
      } else {
        a = *reinterpret_cast<const kp_f32x4_any_t*>(p);
        b = *reinterpret_cast<const kp_f32x4_any_t*>(p + 4);
      }
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
k_keep_save(const void* __restrict__ X, int64_t ldx, uint32_t T, uint32_t n, uint32_t units,
            int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;   // units is a multiple of 4
  const uint32_t q = i / units;
  const bool in = q < T;
  const int64_t t = in ? q : 0;
  const uint32_t u = in ? i - q * units : 0, c = 8 * u;
  const int nc = in && c < n ? (int)min(8u, n - c) : 0;
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
  *reinterpret_cast<kp_u32x2_t*>(codes + t * (8 * (int64_t)units) + c) = (kp_u32x2_t){w[0], w[1]};
  if ((u & 3) == 0) exps[t * (int64_t)(units / 4) + (u >> 2)] = (uint8_t)byte;
}

// STREAM: non-temporal stores for large results (360 MB: 90 against 98 us).
template <bool BF, bool VEC, bool STREAM>
__global__ void __launch_bounds__(256)
k_keep_restore(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, uint32_t T, uint32_t n,
               uint32_t units, void* __restrict__ X, int64_t ldx) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t q = i / units, u = i - q * units, c = 8 * u;
  if (q >= T) return;
  const int64_t t = q;
  const int nc = c < n ? (int)min(8u, n - c) : 0;
  const kp_u32x2_t w = *reinterpret_cast<const kp_u32x2_t*>(codes + t * (8 * (int64_t)units) + c);
  const uint32_t b = exps[t * (int64_t)(units / 4) + (u >> 2)];
  const float step = __uint_as_float(b == 255u ? 0x7FC00000u : b << 23);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * step;
  if (nc == 8) {
    if constexpr (BF) {
      kp_u32x4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j)   // exact in bf16: the low halves are zero
        o[j] = (__float_as_uint(v[2 * j]) >> 16) | (__float_as_uint(v[2 * j + 1]) & 0xFFFF0000u);
      uint16_t* at = static_cast<uint16_t*>(X) + t * ldx + c;
      if constexpr (STREAM) __builtin_nontemporal_store(o, reinterpret_cast<kp_u32x4_t*>(at));
      else if constexpr (VEC) *reinterpret_cast<kp_u32x4_t*>(at) = o;
      else *reinterpret_cast<kp_u32x4_any_t*>(at) = o;
    } else {
      float* at = static_cast<float*>(X) + t * ldx + c;
      const kp_f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      if constexpr (STREAM) {
        __builtin_nontemporal_store(a, reinterpret_cast<kp_f32x4_t*>(at));
        __builtin_nontemporal_store(b, reinterpret_cast<kp_f32x4_t*>(at + 4));
      } else if constexpr (VEC) {
        *reinterpret_cast<kp_f32x4_t*>(at) = a;
        *reinterpret_cast<kp_f32x4_t*>(at + 4) = b;
      } else {
        *reinterpret_cast<kp_f32x4_any_t*>(at) = a;
        *reinterpret_cast<kp_f32x4_any_t*>(at + 4) = b;
      }
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
  const uint32_t units = (uint32_t)(4 * ceil_div(n, 32));
  const dim3 grid((unsigned)ceil_div(T * (int64_t)units, 256)), block(256);
  const bool vec = kp_aligned(X, ldx, bf16 ? 2 : 4);
  if (bf16 && vec) hipLaunchKernelGGL((k_keep_save<true, true>), grid, block, 0, s, X, ldx, (uint32_t)T, (uint32_t)n, units, codes, exps);
  else if (bf16) hipLaunchKernelGGL((k_keep_save<true, false>), grid, block, 0, s, X, ldx, (uint32_t)T, (uint32_t)n, units, codes, exps);
  else if (vec) hipLaunchKernelGGL((k_keep_save<false, true>), grid, block, 0, s, X, ldx, (uint32_t)T, (uint32_t)n, units, codes, exps);
  else hipLaunchKernelGGL((k_keep_save<false, false>), grid, block, 0, s, X, ldx, (uint32_t)T, (uint32_t)n, units, codes, exps);
  return hipGetLastError();
}

hipError_t launch_keep_restore(hipStream_t s, const int8_t* codes, const uint8_t* exps, int64_t T, int64_t n,
                               void* X, int bf16, int64_t ldx) {
  if (T <= 0 || n <= 0) return hipSuccess;
  const uint32_t units = (uint32_t)(4 * ceil_div(n, 32));
  const dim3 grid((unsigned)ceil_div(T * (int64_t)units, 256)), block(256);
  const bool vec = kp_aligned(X, ldx, bf16 ? 2 : 4);
  const bool stream = vec && T * n * (bf16 ? 2 : 4) > kStreamBytes;
  const auto kernel = bf16 ? (stream ? k_keep_restore<true, true, true>
                                     : (vec ? k_keep_restore<true, true, false> : k_keep_restore<true, false, false>))
                           : (stream ? k_keep_restore<false, true, true>
                                     : (vec ? k_keep_restore<false, true, false> : k_keep_restore<false, false, false>));
  hipLaunchKernelGGL(kernel, grid, block, 0, s, codes, exps, (uint32_t)T, (uint32_t)n, units, X, ldx);
  return hipGetLastError();
}

}  // namespace gq

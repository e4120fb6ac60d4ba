// Distillation from a teacher's top logits: the divergence of the student's
// distribution over V entries from the teacher's over K of them, and its
// gradient.
//
//   s = z / tau,  lse = log sum_v exp s_v,  q_v = exp(s_v - lse)
//   loss = sum_k p_k (log p_k - log q_{id_k})
//   dz_v = g / tau (M q_v - sum_{k: id_k = v} p_k),   M = sum_k p_k
//
// Bound by reading the logits once (and writing their gradient once): one pass
// keeps a running maximum and sum per lane and joins them at the end. A
// workgroup has a row (the gradient: or a part of one, where rows are few); no
// result depends on timing. 4096 rows of 131072 bf16 logits: the loss 219 to 231
// us (4.7 TB/s), the gradient 411 to 418 (5.2 TB/s), what a copy of as many bytes
// takes.
#include "common.h"

#include <algorithm>

namespace gq {

typedef unsigned int di_u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int di_u32x2_t __attribute__((ext_vector_type(2)));
typedef di_u32x4_t di_u32x4_any_t __attribute__((aligned(2)));
typedef di_u32x2_t di_u32x2_any_t __attribute__((aligned(2)));
typedef __bf16 di_bf16x2_t __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;

template <bool BF>
struct DiType {
  static constexpr int P = BF ? 8 : 4;              // values of a 16-byte piece
  static constexpr int BYTES = BF ? 2 : 4;
};

template <bool BF>
__device__ __forceinline__ float di_load1(const void* p, int64_t i) {
  if constexpr (BF) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ di_u32x4_t di_piece(const void* p, int64_t i) {   // values i .. i + P - 1, any alignment
  return *reinterpret_cast<const di_u32x4_any_t*>(static_cast<const char*>(p) + i * DiType<BF>::BYTES);
}
template <bool BF>
__device__ __forceinline__ void di_values(di_u32x4_t w, float (&f)[DiType<BF>::P]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}
__device__ __forceinline__ uint32_t di_pack2(float a, float b) {
  const di_bf16x2_t p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
template <bool BF>
__device__ __forceinline__ void di_store1(void* p, int64_t i, float v) {
  if constexpr (BF) static_cast<uint16_t*>(p)[i] = (uint16_t)di_pack2(v, 0.f);
  else static_cast<float*>(p)[i] = v;
}
template <bool BF, int N>
__device__ __forceinline__ void di_store(void* p, int64_t i, const float (&f)[N]) {
  char* at = static_cast<char*>(p) + i * DiType<BF>::BYTES;
  if constexpr (!BF) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      reinterpret_cast<di_u32x4_any_t*>(at)[j] = (di_u32x4_t){__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]),
                                                              __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3])};
  } else if constexpr (N == 8) {
    *reinterpret_cast<di_u32x4_any_t*>(at) = (di_u32x4_t){di_pack2(f[0], f[1]), di_pack2(f[2], f[3]),
                                                          di_pack2(f[4], f[5]), di_pack2(f[6], f[7])};
  } else {
    *reinterpret_cast<di_u32x2_any_t*>(at) = (di_u32x2_t){di_pack2(f[0], f[1]), di_pack2(f[2], f[3])};
  }
}

// 2^x (within an ulp; 0 for -inf)
__device__ __forceinline__ float di_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// A part of the sum: sum exp((z - m) / tau) = l. m = -inf, l = 0: nothing yet,
// or logits of -inf alone.
struct DiSum {
  float m, l;
};
__device__ __forceinline__ float di_ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ DiSum di_join(DiSum a, DiSum b, float c) {
  const float m = fmaxf(a.m, b.m), r = di_ref(m);
  // a NaN among the logits is in its l (a maximum passes it over)
  return DiSum{m, a.l * di_exp2((a.m - r) * c) + b.l * di_exp2((b.m - r) * c)};
}

// Sums (maxima) over the workgroup, in a fixed order, in every thread.
template <int THREADS, class F>
__device__ __forceinline__ float di_all(float v, float* red, F&& f) {
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) v = f(v, __shfl_xor(v, i));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = f(v, red[w]);
  return v;
}
template <int THREADS>
__device__ __forceinline__ float di_add(float v, float* red) {
  return di_all<THREADS>(v, red, [](float a, float b) { return a + b; });
}
template <int THREADS>
__device__ __forceinline__ float di_max(float v, float* red) {
  return di_all<THREADS>(v, red, [](float a, float b) { return fmaxf(a, b); });
}

// The teacher's entries of a row: thread t has entries t, t + THREADS, ...
template <int THREADS>
struct DiTeacher {
  static constexpr int PER = kDistillMaxK / THREADS;
  int id[PER];           // -1: none (ids outside [0, V) are not entries)
  float lp[PER];         // log p
  float p[PER];          // 0 for no entry
};
template <int THREADS>
__device__ __forceinline__ void di_load_teacher(const DistillArgs& a, int64_t row, DiTeacher<THREADS>& te) {
#pragma unroll
  for (int i = 0; i < te.PER; ++i) {
    const int k = threadIdx.x + THREADS * i;
    te.id[i] = -1;
    te.lp[i] = -INFINITY;
    if (k < a.K) {
      const int id = a.ids[row * a.K + k];
      if (id >= 0 && id < a.V) {
        te.id[i] = id;
        te.lp[i] = a.teacher[row * a.K + k];
      }
    }
  }
}
// p and log p; returns their mass (0: nothing to learn in this row).
template <int THREADS>
__device__ __forceinline__ float di_probabilities(const DistillArgs& a, DiTeacher<THREADS>& te, float* red) {
  float sum = 0.f, top = 0.f, inv = 1.f, ln = 0.f;
  if (!a.log_probs) {
    float hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < te.PER; ++i) hi = fmaxf(hi, te.lp[i]);
    top = di_ref(di_max<THREADS>(hi, red));
#pragma unroll
    for (int i = 0; i < te.PER; ++i) {
      te.lp[i] = (te.lp[i] - top) * a.inv_temp;
      te.p[i] = expf(te.lp[i]);
      sum += te.p[i];
    }
    sum = di_add<THREADS>(sum, red);
    if (sum == 0.f) return 0.f;
    inv = 1.f / sum;
    ln = logf(sum);
  }
  float mass = 0.f;
#pragma unroll
  for (int i = 0; i < te.PER; ++i) {
    te.lp[i] -= ln;
    te.p[i] = a.log_probs ? expf(te.lp[i]) : te.p[i] * inv;
    mass += te.p[i];
  }
  return di_add<THREADS>(mass, red);
}

// Loss and lse of a row from its sum. zt: the student's logits at the
// teacher's entries.
template <int THREADS>
__device__ __forceinline__ void di_finish(const DistillArgs& a, int64_t row, DiSum s, DiTeacher<THREADS>& te,
                                          const float (&zt)[DiTeacher<THREADS>::PER], float* red) {
  const float ll = logf(s.l), r = di_ref(s.m);
  const float mass = di_probabilities(a, te, red);
  float loss = 0.f;
  if (mass != 0.f) {
#pragma unroll
    for (int i = 0; i < te.PER; ++i)    // p (log p - log q); an entry without mass adds nothing wherever its logit is
      if (te.p[i] != 0.f) loss += te.p[i] * (te.lp[i] - ((zt[i] - r) * a.inv_temp - ll));
    loss = di_add<THREADS>(loss, red);
  }
  if (threadIdx.x == 0) {
    a.loss[row] = loss;
    a.lse[row] = s.m * a.inv_temp + ll;
  }
}

// The sum of a row, in every thread (sums: one per wave, in LDS).
template <bool BF, int THREADS>
__device__ __forceinline__ DiSum di_row_sum(const char* z, int cols, float inv_temp, DiSum* sums) {
  constexpr int P = DiType<BF>::P, U = 4, WAVES = THREADS / 64;
  const int tid = threadIdx.x, np = cols / P;
  const float c = kLog2e * inv_temp;
  DiSum s = {-INFINITY, 0.f};
  auto take = [&](const float* f, int n) {
    float m = s.m;
#pragma unroll
    for (int i = 0; i < n; ++i) m = fmaxf(m, f[i]);
    const float r = di_ref(m);
    float l = s.l * di_exp2((s.m - r) * c);
#pragma unroll
    for (int i = 0; i < n; ++i) l += di_exp2((f[i] - r) * c);
    s = DiSum{m, l};
  };
  int p = tid;
  for (; p + (U - 1) * THREADS < np; p += U * THREADS) {
    di_u32x4_t w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = di_piece<BF>(z, (int64_t)(p + u * THREADS) * P);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[P];
      di_values<BF>(w[u], f);
      take(f, P);
    }
  }
  for (; p < np; p += THREADS) {
    float f[P];
    di_values<BF>(di_piece<BF>(z, (int64_t)p * P), f);
    take(f, P);
  }
  if (tid < cols - np * P) {
    const float f = di_load1<BF>(z, np * P + tid);
    take(&f, 1);
  }
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) s = di_join(s, DiSum{__shfl_xor(s.m, i), __shfl_xor(s.l, i)}, c);
  if ((tid & 63) == 0) sums[tid >> 6] = s;
  __syncthreads();
  s = sums[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s = di_join(s, sums[w], c);
  return s;
}

template <bool BF, int THREADS>
__global__ void __launch_bounds__(THREADS)
k_distill(DistillArgs a) {
  __shared__ float red[THREADS / 64];
  __shared__ DiSum sums[THREADS / 64];
  const int64_t row = blockIdx.x;
  const char* z = static_cast<const char*>(a.Z) + row * a.ldz * DiType<BF>::BYTES;
  DiTeacher<THREADS> te;
  float zt[te.PER];                                // the student's logits at the teacher's entries
  di_load_teacher<THREADS>(a, row, te);
#pragma unroll
  for (int i = 0; i < te.PER; ++i) zt[i] = te.id[i] >= 0 ? di_load1<BF>(z, te.id[i]) : 0.f;
  const DiSum s = di_row_sum<BF, THREADS>(z, (int)a.V, a.inv_temp, sums);
  di_finish<THREADS>(a, row, s, te, zt, red);
}

// Columns of part p of a row (whole pieces but for the last).
struct DiPart {
  int64_t lo, hi;
};
__device__ __forceinline__ DiPart di_part(const DistillArgs& a, int p) {
  const int64_t lo = (int64_t)p * a.part_cols;
  return DiPart{lo, min(lo + a.part_cols, (int64_t)a.V)};
}

// What fp32 rounds off lse is relative in every q: 2^-18 at 128, 2^-14 (of a bf16
// result's 2^-9) at 2048. In rows whose lse is larger (all logits at the type's
// lowest value, a large common offset, a low temperature) it would grow without
// bound (q = 1 for 1 / V): one workgroup takes the row, forms its largest logit and
// sum again as the loss has them, and writes all of it, so that dZ may still be Z.
// 4096 such rows of 131072 bf16 logits 653 us for 449, 61 of 32003 13.5 for 6.8, 8
// of 131072 41 for 8.
template <bool OBF>
constexpr float kDiFar = OBF ? 2048.f : 128.f;

// The gradient: q of every entry is written first, then the teacher's entries
// are written over it by the workgroup that owns their columns (their logits
// were read before, so that dZ may be Z). An id that stands more than once in
// a row gets all of its p, added in their order by each of its threads: they
// all store the same value.
template <bool BF, bool OBF>
__global__ void __launch_bounds__(256)
k_distill_grad(DistillArgs a) {
  constexpr int THREADS = 256, P = DiType<BF>::P, U = 4;
  __shared__ float red[THREADS / 64];
  __shared__ int sid[kDistillMaxK];
  __shared__ float sp[kDistillMaxK];
  __shared__ DiSum sums[THREADS / 64];
  const int64_t row = blockIdx.x / a.parts;
  DiPart part = di_part(a, blockIdx.x % a.parts);
  const int tid = threadIdx.x;
  const char* z = static_cast<const char*>(a.Z) + (row * a.ldz + part.lo) * DiType<BF>::BYTES;
  DiTeacher<THREADS> te;
  float zt[te.PER];
  di_load_teacher<THREADS>(a, row, te);
  auto load_logits = [&]() {
#pragma unroll
    for (int i = 0; i < te.PER; ++i) {
      zt[i] = 0.f;
      if (te.id[i] >= part.lo && te.id[i] < part.hi) zt[i] = di_load1<BF>(z, te.id[i] - part.lo);
    }
  };
  load_logits();
  const float lse = a.lse_in[row], g = a.grad[row] * a.inv_temp;
  const float mass = di_probabilities<THREADS>(a, te, red);
  const bool none = mass == 0.f;                   // nothing to learn: zeros, whatever the logits are
  const float f = g * mass;
  float top = 0.f, ll = lse;                       // log q = (z - top) / tau - ll
  if (!none && !(fabsf(lse) <= kDiFar<OBF>)) {
    if (part.lo > 0) return;                       // (all workgroups of the row come here)
    part.hi = a.V;
    load_logits();
    const DiSum s = di_row_sum<BF, THREADS>(z, (int)a.V, a.inv_temp, sums);
    top = di_ref(s.m);
    ll = logf(s.l);
  }
  char* out = static_cast<char*>(a.dZ) + (row * a.ldd + part.lo) * DiType<OBF>::BYTES;
  const int cols = (int)(part.hi - part.lo), np = cols / P;
#pragma unroll
  for (int i = 0; i < te.PER; ++i) {
    const int k = tid + THREADS * i;
    if (k < a.K) {
      sid[k] = te.id[i];
      sp[k] = te.p[i];
    }
  }
  auto value = [&](float v) { return none ? 0.f : f * di_exp2(fmaf(v - top, a.inv_temp, -ll) * kLog2e); };
#pragma unroll
  for (int i = 0; i < te.PER; ++i) zt[i] = value(zt[i]);
  __syncthreads();                                 // the teacher's logits are read
  int p = tid;
  for (; p + (U - 1) * THREADS < np; p += U * THREADS) {
    di_u32x4_t w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = di_piece<BF>(z, (int64_t)(p + u * THREADS) * P);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[P];
      di_values<BF>(w[u], v);
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = value(v[i]);
      di_store<OBF, P>(out, (int64_t)(p + u * THREADS) * P, v);
    }
  }
  for (; p < np; p += THREADS) {
    float v[P];
    di_values<BF>(di_piece<BF>(z, (int64_t)p * P), v);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = value(v[i]);
    di_store<OBF, P>(out, (int64_t)p * P, v);
  }
  if (tid < cols - np * P) di_store1<OBF>(out, np * P + tid, value(di_load1<BF>(z, np * P + tid)));
  __syncthreads();                                 // the stores above come before those below
  if (none) return;
#pragma unroll
  for (int i = 0; i < te.PER; ++i) {
    if (te.id[i] < part.lo || te.id[i] >= part.hi) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k)
      if (sid[k] == te.id[i]) sum += sp[k];
    di_store1<OBF>(out, te.id[i] - part.lo, zt[i] - g * sum);
  }
}

// ---------------------------------------------------------------- host
// Rows below four workgroups per CU go with 1024 threads each, whatever their
// length: 61 rows of 32003 fp32 values 8.4 us in one launch; in parts of 2048
// values or more with a second launch that joins them 4.6 + 4.5, and a workspace.
hipError_t launch_distill(hipStream_t s, const DistillArgs& a) {
  const dim3 grid((unsigned)a.T);
  const bool few = a.T < 1024 && a.V > 2048;
  if (a.z_bf16 && few) hipLaunchKernelGGL((k_distill<true, 1024>), grid, dim3(1024), 0, s, a);
  else if (few) hipLaunchKernelGGL((k_distill<false, 1024>), grid, dim3(1024), 0, s, a);
  else if (a.z_bf16) hipLaunchKernelGGL((k_distill<true, 256>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_distill<false, 256>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_distill_grad(hipStream_t s, const DistillArgs& args) {
  DistillArgs a = args;
  // parts of a row: until there are four workgroups per CU, of at least 2048 values
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(ceil_div(1024, a.T), a.V / 2048));
  a.part_cols = ceil_div(ceil_div(a.V, parts), 8) * 8;
  a.parts = (int)ceil_div(a.V, a.part_cols);
  const dim3 grid((unsigned)(a.T * a.parts)), block(256);
  if (a.z_bf16 && a.dz_bf16) hipLaunchKernelGGL((k_distill_grad<true, true>), grid, block, 0, s, a);
  else if (a.z_bf16) hipLaunchKernelGGL((k_distill_grad<true, false>), grid, block, 0, s, a);
  else if (a.dz_bf16) hipLaunchKernelGGL((k_distill_grad<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_distill_grad<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace gq

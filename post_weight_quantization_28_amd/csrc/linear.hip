// Packed layers with bias, activation, gate and residual, and their gradient.
//
//   z = X[rows[p]] W_hat_e^T + bias[e],  Y[p] = act(z) (or act(g) u) + residual[p]
//   dZ = dY act'(z)  (or (dY u act'(g), dY act(g))),  dbias[e] = sum_p dZ[p],
//   dX[p] = dZ[p] W_hat_e
//
// The product is experts.hip's.
#include "act.h"
#include "common.h"

#include <algorithm>

namespace gq {

typedef unsigned int li_u32x4_t __attribute__((ext_vector_type(4)));
typedef li_u32x4_t li_u32x4_any_t __attribute__((aligned(2)));
typedef __bf16 li_bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float li_load(const void* p, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ uint32_t li_pack2(float a, float b) {
  const li_bf16x2_t p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ void li_store(void* p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<uint16_t*>(p)[i] = (uint16_t)li_pack2(v, 0.f);
  else static_cast<float*>(p)[i] = v;
}

// The segment of a row: the last one that starts at or before it.
__device__ __forceinline__ int li_expert(const int32_t* __restrict__ offsets, int E, int64_t row) {
  int lo = 0, hi = E;                      // offsets[lo] <= row, offsets[hi] > row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- forward
__global__ void __launch_bounds__(256)
k_linear_end(const float* __restrict__ part, int64_t m, LinearArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / a.d, c = i - row * a.d;
  if (row >= a.mm.R) return;
  const int32_t* offsets = a.mm.offsets;
  if (offsets && (row < offsets[0] || row >= offsets[a.mm.E])) return;
  const float* b = a.bias;
  if (b && offsets) b += li_expert(offsets, a.mm.E, row) * m;
  float v[2];
  for (int h = 0; h <= a.gated; ++h) {
    v[h] = part[row * m + h * a.d + c] + (b ? b[h * a.d + c] : 0.f);
    if (a.Z) li_store(a.Z, a.z_bf16, row * a.ldz + h * a.d + c, v[h]);
  }
  float y = act_value(a.act, v[0]);
  if (a.gated) y *= v[1];
  if (a.res) y += li_load(a.res, a.res_bf16, row * a.ldr + c);
  li_store(a.Y, a.y_bf16, row * a.ldy + c, y);
}

size_t linear_workspace(int64_t R, int E, int64_t n, int64_t m, int group) {
  return (expert_split(R, E, n, m, group, 0, false).part_bytes + 255) / 256 * 256 + (size_t)R * m * sizeof(float);
}

hipError_t launch_linear(hipStream_t s, const LinearArgs& a) {
  const int64_t m = a.mm.d_out;
  ExpertArgs e = a.mm;
  float* z = reinterpret_cast<float*>(static_cast<char*>(a.ws) +
                                      (expert_split(e.R, e.E, e.n, m, e.group, 0, false).part_bytes + 255) / 256 * 256);
  e.part = a.ws;
  e.Y = z;
  e.y_bf16 = 0;
  e.ldy = m;
  const hipError_t err = launch_expert_mm(s, e);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(k_linear_end, dim3((unsigned)ceil_div(e.R * a.d, 256)), dim3(256), 0, s, z, m, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
// dZ and the partial sums of dbias, bound by their bytes. A workgroup owns
// kLgRows rows of one segment and 256 columns of dY: 32 lanes of eight
// columns side by side, eight rows at a time. Its column sums go to
// part[tile][m], and a second launch adds a segment's tiles in their order.
constexpr int kLgRows = 64;

// Row tiles of all segments, an upper bound known to the host.
static int64_t li_tiles(int64_t R, int E) { return std::min<int64_t>(R, ceil_div(R, kLgRows) + E - 1); }

// The segment of row tile rt, its rows and the number of its first tile; e = -1
// past the last one. Called by whole waves.
struct LiSeg {
  int e, lo, hi, first;
};
__device__ __forceinline__ LiSeg li_find(const int32_t* __restrict__ offsets, int E, int R, int rt) {
  if (offsets == nullptr) return LiSeg{(int64_t)rt * kLgRows < R ? 0 : -1, 0, R, 0};
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < E) {
      lo = min(max(offsets[e0 + lane], 0), R);
      hi = min(max(offsets[e0 + lane + 1], lo), R);
    }
    const int nt = (hi - lo + kLgRows - 1) / kLgRows;
    int inc = nt;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const int v = __shfl_up(inc, i);
      if (lane >= i) inc += v;
    }
    const uint64_t past = __ballot(before + inc > rt);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      return LiSeg{e0 + l, __shfl(lo, l), __shfl(hi, l), before + __shfl(inc - nt, l)};
    }
    before += __shfl(inc, 63);
  }
  return LiSeg{-1, 0, 0, 0};
}

// Eight values from column c of a row (`have` of them exist), at any alignment.
template <bool BF>
__device__ __forceinline__ void li_row8(const void* p, int64_t at, int have, float (&f)[8]) {
  if (have >= 8) {
    if constexpr (BF) {
      const li_u32x4_t w = *reinterpret_cast<const li_u32x4_any_t*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const li_u32x4_t w = *reinterpret_cast<const li_u32x4_any_t*>(static_cast<const float*>(p) + at + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * h + i] = __uint_as_float(w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < have ? li_load(p, BF, at + i) : 0.f;
  }
}
__device__ __forceinline__ void li_store8(uint16_t* p, int have, const float (&f)[8]) {
  if (have >= 8) {
    *reinterpret_cast<li_u32x4_any_t*>(p) =
        (li_u32x4_t){li_pack2(f[0], f[1]), li_pack2(f[2], f[3]), li_pack2(f[4], f[5]), li_pack2(f[6], f[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) p[i] = (uint16_t)li_pack2(f[i], 0.f);
  }
}

template <bool YBF, bool ZBF, bool GATED>
__global__ void __launch_bounds__(256)
k_linear_dz(LinearGradArgs a) {
  __shared__ float sums[GATED ? 2 : 1][8][256];
  const uint32_t nct = (uint32_t)((a.d + 255) / 256);
  const int rt = blockIdx.x / nct;
  const int64_t c0 = (int64_t)(blockIdx.x % nct) * 256;
  const LiSeg sg = li_find(a.mm.offsets, a.mm.E, a.mm.R, rt);
  if (sg.e < 0) return;
  const int r0 = sg.lo + (rt - sg.first) * kLgRows, r1 = min(r0 + kLgRows, sg.hi);
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c = c0 + 8 * cl;
  const int have = (int)min((int64_t)8, a.d - c);
  float sg_[8] = {}, su_[8] = {};
  if (have > 0) {
    for (int r = r0 + rl; r < r1; r += 8) {
      float dy[8], z[8], u[8], dg[8], du[8];
      li_row8<YBF>(a.dY, r * a.ldy + c, have, dy);
      if (a.Z) li_row8<ZBF>(a.Z, r * a.ldz + c, have, z);
      if constexpr (GATED) li_row8<ZBF>(a.Z, r * a.ldz + a.d + c, have, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float slope = 1.f, v = 0.f;
        if (a.Z) v = act_both(a.act, z[i], slope);
        dg[i] = dy[i] * slope;
        if constexpr (GATED) {
          dg[i] = dy[i] * u[i] * slope;
          du[i] = dy[i] * v;
          su_[i] += du[i];
        }
        sg_[i] += dg[i];
      }
      if (a.dZ) {
        li_store8(a.dZ + r * a.lddz + c, have, dg);
        if constexpr (GATED) li_store8(a.dZ + r * a.lddz + a.d + c, have, du);
      }
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[0][rl][8 * cl + i] = sg_[i];
    if constexpr (GATED) sums[1][rl][8 * cl + i] = su_[i];
  }
  __syncthreads();
  const int64_t col = c0 + threadIdx.x;
  if (col >= a.d) return;
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sums[h][i][threadIdx.x];
    a.part[(int64_t)rt * a.m + h * a.d + col] = v;
  }
}

__global__ void __launch_bounds__(256)
k_linear_dbias(const float* __restrict__ part, const int32_t* __restrict__ offsets, int E, int R, int64_t m,
               float* __restrict__ dbias) {
  const int e = blockIdx.y, lane = threadIdx.x & 63;
  int first = 0, count = (R + kLgRows - 1) / kLgRows;
  if (offsets) {
    // tiles of the segments before this one
    for (int e0 = 0; e0 <= e; e0 += 64) {
      int nt = 0;
      if (e0 + lane <= e) {
        const int lo = min(max(offsets[e0 + lane], 0), R), hi = min(max(offsets[e0 + lane + 1], lo), R);
        nt = (hi - lo + kLgRows - 1) / kLgRows;
      }
      if (e0 + 64 > e) count = __shfl(nt, e - e0);
      int t = e0 + lane < e ? nt : 0;
#pragma unroll
      for (int i = 32; i > 0; i >>= 1) t += __shfl_xor(t, i);
      first += t;
    }
  }
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= m) return;
  float v = 0.f;
  for (int t = 0; t < count; ++t) v += part[(int64_t)(first + t) * m + c];
  dbias[(int64_t)e * m + c] = v;
}

int64_t linear_bias_parts(int64_t R, int E, int64_t m) { return li_tiles(R, E) * m; }
int64_t linear_grad_threads(int64_t R, int E, int64_t d) { return R > 0 ? li_tiles(R, E) * ceil_div(d, 256) * 256 : 0; }

template <bool GATED>
static void dz_go(hipStream_t s, const LinearGradArgs& a) {
  const dim3 grid((unsigned)(li_tiles(a.mm.R, a.mm.E) * ceil_div(a.d, 256))), block(256);
  if (a.dy_bf16 && a.z_bf16) hipLaunchKernelGGL((k_linear_dz<true, true, GATED>), grid, block, 0, s, a);
  else if (a.dy_bf16) hipLaunchKernelGGL((k_linear_dz<true, false, GATED>), grid, block, 0, s, a);
  else if (a.z_bf16) hipLaunchKernelGGL((k_linear_dz<false, true, GATED>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_linear_dz<false, false, GATED>), grid, block, 0, s, a);
}

hipError_t launch_linear_grad(hipStream_t s, const LinearGradArgs& a) {
  if (a.mm.R > 0 && (a.dZ || a.dbias)) {
    if (a.gated) dz_go<true>(s, a);
    else dz_go<false>(s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (a.dbias) {
    hipLaunchKernelGGL(k_linear_dbias, dim3((unsigned)ceil_div(a.m, 256), (unsigned)a.mm.E), dim3(256), 0, s, a.part,
                       a.mm.offsets, a.mm.E, a.mm.R, a.m, a.dbias);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return a.mm.R > 0 ? launch_expert_mm_grad(s, a.mm) : hipSuccess;
}

}  // namespace gq

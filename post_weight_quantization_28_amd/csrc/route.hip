// Tokens in the order of their experts, and back.
//
// A mixture of experts sends token t to the experts ids[t][0..k). The packed
// layers of this library work on contiguous rows, so the T k slots
// i = t k + j are put in the stable order of their expert:
//   offsets[e] = #{kept slots with an expert below e},
//   inverse[i] = offsets[ids[i]] + #{kept slots i' < i with the same expert},
//   rows[inverse[i]] = t.
// A slot whose id is outside [0, E) is dropped: inverse[i] = -1, and the
// last T k - offsets[E] entries of rows are -1. The way there copies
// Xs[inverse[i]] = X[t]; the way back is Y[t] = sum_j w[t][j] Ys[inverse[t k + j]],
// whose gradients are dYs[inverse[i]] = w[i] dY[t] and
// dw[i] = <dY[t], Ys[inverse[i]]>; the gradient of the way there is the way
// back with weights of one.
//
// The order is a counting sort whose ranks come from ballots, never from
// atomics that return a place, so it does not depend on timing. Everything
// here is bound by memory (or, for a few tokens, by the launches): the
// copies are organised by token, so each row of X is read once (dY: once for
// four slots) and its copies leave from registers, and the way back adds the
// k rows in the order of j in fp32 and rounds once.
#include "common.h"
#include "dma.h"

#include <algorithm>

namespace gq {

typedef unsigned int rt_u32x4_t __attribute__((ext_vector_type(4)));
typedef float rt_f32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- the order
constexpr int kRtSteps = 4;          // 64-slot steps per wave
constexpr int kRtMaxBuckets = kRouteMaxExperts + 1;   // the last bucket: dropped slots

__device__ __forceinline__ int rt_bucket(const int32_t* __restrict__ ids, int64_t ldi, int k, int64_t i, int E) {
  const int64_t t = i / k;
  const int id = ids[t * ldi + (i - t * k)];
  return (unsigned)id < (unsigned)E ? id : E;
}

// Lanes of the wave that hold the same bucket (active lanes only).
__device__ __forceinline__ uint64_t rt_peers(int b, bool active, int nbits) {
  uint64_t m = __ballot(active);
  for (int i = 0; i < nbits; ++i) {
    const bool bit = (b >> i) & 1;
    const uint64_t v = __ballot(active && bit);
    m &= bit ? v : ~v;
  }
  return m;
}

// Ranks of this wave's slots inside their buckets: loc[s] counts the wave's
// earlier slots of the same bucket, and hist (this wave's row, zeroed)
// receives the wave's totals.
__device__ __forceinline__ void rt_rank(const int32_t* __restrict__ ids, int64_t ldi, int k, int64_t first,
                                        int64_t R, int E, int nbits, uint16_t* hist, int (&bk)[kRtSteps],
                                        int (&loc)[kRtSteps]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < kRtSteps; ++s) {
    const int64_t i = first + 64 * s + lane;
    bk[s] = i < R ? rt_bucket(ids, ldi, k, i, E) : -1;
  }
#pragma unroll
  for (int s = 0; s < kRtSteps; ++s) {
    const bool act = bk[s] >= 0;
    const uint64_t peers = rt_peers(bk[s], act, nbits);
    const uint64_t before = peers & ((1ull << lane) - 1ull);
    int base = 0;
    if (act) {
      base = hist[bk[s]];
      loc[s] = base + __popcll(before);
    }
    // one lane per bucket adds the step's count; the fences keep the order of
    // the wave's LDS accesses, whose lanes see each other's values
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (act && before == 0) hist[bk[s]] = (uint16_t)(base + __popcll(peers));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Exclusive sums of v[0..nb) in place (all threads of the block; tmp: one
// int per wave). Thread t owns ceil(nb / threads) consecutive entries.
template <int THREADS>
__device__ void rt_scan(int* v, int nb, int* tmp) {
  const int per = (nb + THREADS - 1) / THREADS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b0 = threadIdx.x * per, b1 = min(nb, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += v[b];
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) tmp[wave] = inc;
  __syncthreads();
  int run = inc - sum;
  for (int w = 0; w < wave; ++w) run += tmp[w];
  for (int b = b0; b < b1; ++b) {
    const int c = v[b];
    v[b] = run;
    run += c;
  }
  __syncthreads();
}

// One workgroup's slots in order. base (LDS): the first place of each
// bucket; the wave offsets come from the waves' histograms.
__device__ __forceinline__ void rt_place(const int (&bk)[kRtSteps], const int (&loc)[kRtSteps], int64_t first,
                                         int64_t R, int k, int E, const int* base, const uint16_t* hist, int nb,
                                         int wave, int32_t* __restrict__ rows, int32_t* __restrict__ inverse) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < kRtSteps; ++s) {
    const int64_t i = first + 64 * s + lane;
    if (i >= R) continue;
    int p = base[bk[s]] + loc[s];
    for (int w = 0; w < wave; ++w) p += hist[w * nb + bk[s]];
    const bool kept = bk[s] < E;
    rows[p] = kept ? (int32_t)(i / k) : -1;
    inverse[i] = kept ? p : -1;
  }
}

// All slots in one workgroup of 16 waves (R <= kRouteOneBlock): one launch,
// which is what a decoding step pays for.
__global__ void __launch_bounds__(1024)
k_route_one(const int32_t* __restrict__ ids, int64_t ldi, int64_t R, int k, int E, int nbits,
            int32_t* __restrict__ offsets, int32_t* __restrict__ rows, int32_t* __restrict__ inverse) {
  __shared__ uint16_t hist[16 * kRtMaxBuckets];
  __shared__ int base[kRtMaxBuckets];
  __shared__ int tmp[16];
  const int nb = E + 1, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < 16 * nb; i += 1024) hist[i] = 0;
  __syncthreads();
  // wave-major slots, as many steps per wave as the slots need
  const int64_t steps = ceil_div(R, 16 * 64);
  const int64_t first = (int64_t)wave * steps * 64;
  const int64_t end = min(R, first + steps * 64);
  int bk[kRtSteps], loc[kRtSteps];
  rt_rank(ids, ldi, k, first, end, E, nbits, hist + wave * nb, bk, loc);
  __syncthreads();
  for (int b = threadIdx.x; b < nb; b += 1024) {
    int c = 0;
    for (int w = 0; w < 16; ++w) c += hist[w * nb + b];
    base[b] = c;
  }
  __syncthreads();
  rt_scan<1024>(base, nb, tmp);
  for (int b = threadIdx.x; b < nb; b += 1024) offsets[b] = base[b];
  rt_place(bk, loc, first, end, k, E, base, hist, nb, wave, rows, inverse);
}

// Larger batches, three launches: bucket counts of each block of
// kRouteBlockSlots slots (count[b][block]), ...
__global__ void __launch_bounds__(256)
k_route_count(const int32_t* __restrict__ ids, int64_t ldi, int64_t R, int k, int E, int nblocks,
              int32_t* __restrict__ count) {
  __shared__ int h[kRtMaxBuckets];
  for (int b = threadIdx.x; b <= E; b += 256) h[b] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kRouteBlockSlots;
#pragma unroll
  for (int s = 0; s < kRtSteps; ++s) {
    const int64_t i = i0 + 256 * s + threadIdx.x;
    if (i < R) atomicAdd(&h[rt_bucket(ids, ldi, k, i, E)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b <= E; b += 256) count[(int64_t)b * nblocks + blockIdx.x] = h[b];
}

// ... their exclusive sums along the blocks, one workgroup per bucket, and
// the buckets' totals, ...
__global__ void __launch_bounds__(256)
k_route_scan(int32_t* __restrict__ count, int nblocks, int32_t* __restrict__ total) {
  __shared__ int tmp[4];
  int32_t* __restrict__ c = count + (int64_t)blockIdx.x * nblocks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int b0 = 0; b0 < nblocks; b0 += 256) {
    const int b = b0 + threadIdx.x;
    const int v = b < nblocks ? c[b] : 0;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 63) tmp[wave] = inc;
    __syncthreads();
    int run = carry + inc - v, all = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) run += tmp[w];
      all += tmp[w];
    }
    if (b < nblocks) c[b] = run;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) total[blockIdx.x] = carry;
}

// ... and the places.
__global__ void __launch_bounds__(256)
k_route_place(const int32_t* __restrict__ ids, int64_t ldi, int64_t R, int k, int E, int nbits, int nblocks,
              const int32_t* __restrict__ count, const int32_t* __restrict__ total,
              int32_t* __restrict__ offsets, int32_t* __restrict__ rows, int32_t* __restrict__ inverse) {
  __shared__ uint16_t hist[4 * kRtMaxBuckets];
  __shared__ int base[kRtMaxBuckets];
  __shared__ int tmp[4];
  const int nb = E + 1, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < 4 * nb; i += 256) hist[i] = 0;
  for (int b = threadIdx.x; b < nb; b += 256) base[b] = total[b];
  __syncthreads();
  rt_scan<256>(base, nb, tmp);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < nb; b += 256) offsets[b] = base[b];
  const int64_t first = (int64_t)blockIdx.x * kRouteBlockSlots + (int64_t)wave * (64 * kRtSteps);
  int bk[kRtSteps], loc[kRtSteps];
  rt_rank(ids, ldi, k, first, R, E, nbits, hist + wave * nb, bk, loc);
  __syncthreads();
  for (int b = threadIdx.x; b < nb; b += 256) base[b] += count[(int64_t)b * nblocks + blockIdx.x];
  __syncthreads();
  rt_place(bk, loc, first, R, k, E, base, hist, nb, wave, rows, inverse);
}

size_t route_workspace(int64_t R, int64_t E) {
  if (R <= kRouteOneBlock) return 0;
  const int64_t nblocks = ceil_div(R, kRouteBlockSlots);
  return (size_t)(E + 1) * (size_t)(nblocks + 1) * sizeof(int32_t);
}

hipError_t launch_route(hipStream_t s, const int32_t* ids, int64_t ldi, int64_t T, int k, int E, int32_t* offsets,
                        int32_t* rows, int32_t* inverse, void* ws) {
  const int64_t R = T * k;
  int nbits = 0;
  while ((E >> nbits) != 0) ++nbits;      // buckets 0..E
  if (R <= kRouteOneBlock) {
    hipLaunchKernelGGL(k_route_one, dim3(1), dim3(1024), 0, s, ids, ldi, R, k, E, nbits, offsets, rows, inverse);
    return hipGetLastError();
  }
  const int nblocks = (int)ceil_div(R, kRouteBlockSlots);
  int32_t* total = static_cast<int32_t*>(ws);
  int32_t* count = total + (E + 1);
  hipLaunchKernelGGL(k_route_count, dim3(nblocks), dim3(256), 0, s, ids, ldi, R, k, E, nblocks, count);
  hipLaunchKernelGGL(k_route_scan, dim3(E + 1), dim3(256), 0, s, count, nblocks, total);
  hipLaunchKernelGGL(k_route_place, dim3(nblocks), dim3(256), 0, s, ids, ldi, R, k, E, nbits, nblocks, count, total,
                     offsets, rows, inverse);
  return hipGetLastError();
}

// ---------------------------------------------------------------- rows there and back
// The rows of Ys are read once, so where they are aligned they are loaded past
// the caches, whatever their number, and dY with them, which the gradient reads
// once for each four slots of a token. Past the caches and through them, 2048
// columns, 8 slots: the way back of 8192 tokens (268 MB of Ys) 55 and 58 us, its
// gradient 99 and 122, of 2048 tokens 33 and 31, of 512 tokens 9.7 and 9.2; the
// way back right after the way there is alike up to 2048 tokens (8192: 115 and
// 120 for both). One slot of 4096 tokens of 4096 columns: 14.7 and 12.4.
// A unit is 8 columns: 16 bytes of bf16, 32 of fp32.
//   kAligned: every row of both sides is 16-byte aligned and n % 8 == 0, so
//     units move as whole 16-byte pieces;
//   kAnywhere: n >= 8; pieces of any alignment, a row's last unit moved back to
//     end with the row (the columns that two units share get the same value
//     from both);
//   kSingly: columns one by one, for rows of less than a unit.
// 4096 tokens, 8 slots each, rows of 1915: the way there, the way back and its
// gradient 28, 38 and 78 us with kAnywhere, 67, 79 and 193 column by column.
enum { kSingly, kAnywhere, kAligned };
typedef rt_u32x4_t rt_u32x4_any_t __attribute__((aligned(2)));
typedef rt_f32x4_t rt_f32x4_any_t __attribute__((aligned(4)));

template <bool BF, int MODE>
__device__ __forceinline__ void rt_load8(const void* base, int64_t off, int ncols, float (&v)[8]) {
  if constexpr (MODE != kSingly && BF) {
    rt_u32x4_t u;
    if constexpr (MODE == kAligned)
      u = __builtin_nontemporal_load(reinterpret_cast<const rt_u32x4_t*>(static_cast<const uint16_t*>(base) + off));
    else u = *reinterpret_cast<const rt_u32x4_any_t*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else if constexpr (MODE != kSingly) {
    const float* p = static_cast<const float*>(base) + off;
    rt_f32x4_t a, b;
    if constexpr (MODE == kAligned) {
      a = __builtin_nontemporal_load(reinterpret_cast<const rt_f32x4_t*>(p));
      b = __builtin_nontemporal_load(reinterpret_cast<const rt_f32x4_t*>(p + 4));
    } else {
      a = *reinterpret_cast<const rt_f32x4_any_t*>(p);
      b = *reinterpret_cast<const rt_f32x4_any_t*>(p + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i < ncols)
        v[i] = BF ? bf16_to_f32(static_cast<const uint16_t*>(base)[off + i]) : static_cast<const float*>(base)[off + i];
    }
  }
}

__device__ __forceinline__ uint32_t rt_pack2(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

template <bool BF, int MODE>
__device__ __forceinline__ void rt_store8(void* base, int64_t off, int ncols, const float (&v)[8]) {
  if constexpr (MODE != kSingly && BF) {
    const rt_u32x4_t u = {rt_pack2(v[0], v[1]), rt_pack2(v[2], v[3]), rt_pack2(v[4], v[5]), rt_pack2(v[6], v[7])};
    uint16_t* p = static_cast<uint16_t*>(base) + off;
    if constexpr (MODE == kAligned) *reinterpret_cast<rt_u32x4_t*>(p) = u;
    else *reinterpret_cast<rt_u32x4_any_t*>(p) = u;
  } else if constexpr (MODE != kSingly) {
    const rt_f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    float* p = static_cast<float*>(base) + off;
    if constexpr (MODE == kAligned) {
      *reinterpret_cast<rt_f32x4_t*>(p) = a;
      *reinterpret_cast<rt_f32x4_t*>(p + 4) = b;
    } else {
      *reinterpret_cast<rt_f32x4_any_t*>(p) = a;
      *reinterpret_cast<rt_f32x4_any_t*>(p + 4) = b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < ncols) {
        if constexpr (BF) static_cast<uint16_t*>(base)[off + i] = (uint16_t)rt_pack2(v[i], 0.f);
        else static_cast<float*>(base)[off + i] = v[i];
      }
  }
}

// Xs[inverse[t k + j]] = X[t], copied bit by bit: one thread per piece (a U) of
// X's rows, `width` pieces a row. The pitches are in bytes, and a row's last
// piece is moved back to end with it (bytes: its length). ANY: 16-byte pieces
// of any alignment. STREAM: non-temporal stores (268 MB of copies, 8 per row:
// 37 against 51 us).
template <typename U, bool STREAM, bool ANY>
__global__ void __launch_bounds__(256)
k_dispatch(const char* __restrict__ X, int64_t ldx, uint32_t T, uint32_t width, int64_t bytes, int k,
           const int32_t* __restrict__ inverse, int R, char* __restrict__ Xs, int64_t lds) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t t = i / width;
  if (t >= T) return;
  const int64_t c = min((int64_t)(i - t * width) * (int64_t)sizeof(U), bytes - (int64_t)sizeof(U));
  const char* in = X + (int64_t)t * ldx + c;
  U v;
  if constexpr (ANY) v = *reinterpret_cast<const rt_u32x4_any_t*>(in);
  else v = *reinterpret_cast<const U*>(in);
  const int32_t* __restrict__ inv = inverse + (int64_t)t * k;
  for (int j = 0; j < k; ++j) {
    const int p = inv[j];
    if ((unsigned)p < (unsigned)R) {
      char* out = Xs + (int64_t)p * lds + c;
      if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<U*>(out));
      else if constexpr (ANY) *reinterpret_cast<rt_u32x4_any_t*>(out) = v;
      else *reinterpret_cast<U*>(out) = v;
    }
  }
}

// Y[t] = sum_j w[t][j] Ys[inverse[t k + j]]. Four rows are loaded before the
// first is added, so a thread has up to 64 bytes of bf16 in flight (8192 tokens,
// 8 slots, 2048 columns: 55 us, with eight rows 66; kernels of their own for one
// and two slots are within 3 % of this one).
constexpr int kCombineRows = 4;
template <bool YSBF, bool YBF, int MODE>
__global__ void __launch_bounds__(256)
k_combine(const void* __restrict__ Ys, int64_t lds, int R, const int32_t* __restrict__ inverse,
          const float* __restrict__ w, uint32_t T, uint32_t n, uint32_t units, int k, void* __restrict__ Y, int64_t ldy) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t t = i / units;
  if (t >= T) return;
  uint32_t c = 8u * (i - t * units);
  if constexpr (MODE == kAnywhere) c = min(c, n - 8u);
  const int nc = (int)min(8u, n - c);
  const int64_t s0 = (int64_t)t * k;
  constexpr int KB = kCombineRows;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += KB) {
    float v[KB][8], wj[KB];
    int p[KB];
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      const bool in = j0 + u < k;
      p[u] = in ? inverse[s0 + j0 + u] : -1;
      wj[u] = w && in ? w[s0 + j0 + u] : 1.f;
    }
#pragma unroll
    for (int u = 0; u < KB; ++u)
      if ((unsigned)p[u] < (unsigned)R) rt_load8<YSBF, MODE>(Ys, (int64_t)p[u] * lds + c, nc, v[u]);
#pragma unroll
    for (int u = 0; u < KB; ++u)
      if ((unsigned)p[u] < (unsigned)R) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(wj[u], v[u][e], sum[e]);
      }
  }
  rt_store8<YBF, MODE>(Y, (int64_t)t * ldy + c, nc, sum);
}

// dYs[inverse[t k + j]] = w[t][j] dY[t], dw[t][j] = <dY[t], Ys[inverse[t k + j]]>.
// kCgSlots slots per pass over the columns, whose rows of Ys are all loaded
// before the first is used, so dY is read once for up to that many. One
// workgroup per token makes its passes; with few tokens each pass has a
// workgroup (8 slots, 2048 columns: 64 tokens 4.6 against 6.5 us, 512 9.6 and
// 12.9, 1024 17.4 and 17.7, 2048 30.5 and 32.6: beyond it matters little). The
// dot products are fp32: a thread's columns in order, then
// the lanes and the waves in a fixed tree. A dropped slot has dw = 0 and writes
// no row.
constexpr int kCgSlots = 4;
template <bool DYBF, bool YSBF, bool OBF, int MODE>
__global__ void __launch_bounds__(256)
k_combine_grad(const void* __restrict__ dY, int64_t ldy, const void* __restrict__ Ys, int64_t lds, int64_t R,
               const int32_t* __restrict__ inverse, const float* __restrict__ w, int64_t n, int64_t units, int k,
               void* __restrict__ dYs, int64_t ldo, float* __restrict__ dw) {
  __shared__ float red[4][kCgSlots];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = blockIdx.y * kCgSlots; j0 < k; j0 += gridDim.y * kCgSlots) {
    float dot[kCgSlots], wj[kCgSlots];
    int p[kCgSlots];
#pragma unroll
    for (int u = 0; u < kCgSlots; ++u) {
      const int j = j0 + u;
      const int q = j < k ? inverse[t * k + j] : -1;
      p[u] = q < R ? q : -1;
      wj[u] = p[u] >= 0 ? w[t * k + j] : 0.f;
      dot[u] = 0.f;
    }
    for (int64_t i = threadIdx.x; i < units; i += 256) {
      const int64_t c = MODE == kAnywhere ? min(8 * i, n - 8) : 8 * i;
      const int nc = (int)min((int64_t)8, n - c), seen = (int)(8 * i - c);   // columns of the unit before
      float g[8];
      rt_load8<DYBF, MODE>(dY, t * ldy + c, nc, g);
      float y[kCgSlots][8];
#pragma unroll
      for (int u = 0; u < kCgSlots; ++u)
        if (p[u] >= 0) rt_load8<YSBF, MODE>(Ys, (int64_t)p[u] * lds + c, nc, y[u]);
#pragma unroll
      for (int u = 0; u < kCgSlots; ++u) {
        if (p[u] < 0) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = fmaf(g[e], y[u][e], dot[u]);
          dot[u] = MODE == kAnywhere && e < seen ? dot[u] : d;
          o[e] = wj[u] * g[e];
        }
        rt_store8<OBF, MODE>(dYs, (int64_t)p[u] * ldo + c, nc, o);
      }
    }
#pragma unroll
    for (int u = 0; u < kCgSlots; ++u) {
      float v = dot[u];
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
      if (lane == 0) red[wave][u] = v;
    }
    __syncthreads();
    const int u = threadIdx.x;
    if (u < kCgSlots && j0 + u < k) dw[t * k + j0 + u] = (red[0][u] + red[1][u]) + (red[2][u] + red[3][u]);
    __syncthreads();
  }
}

static bool rows_aligned(const void* p, int64_t ld, int esize) {
  return ((uintptr_t)p & 15) == 0 && (ld * esize) % 16 == 0;
}

template <typename U, bool STREAM, bool ANY>
static void dispatch_go(hipStream_t s, const void* X, int64_t ldx, int64_t T, int64_t bytes, int k,
                        const int32_t* inverse, int64_t R, void* Xs, int64_t lds) {
  const int64_t width = ceil_div(bytes, (int64_t)sizeof(U));
  hipLaunchKernelGGL((k_dispatch<U, STREAM, ANY>), dim3((unsigned)ceil_div(T * width, 256)), dim3(256), 0, s,
                     static_cast<const char*>(X), ldx, (uint32_t)T, (uint32_t)width, bytes, k, inverse, (int)R,
                     static_cast<char*>(Xs), lds);
}

hipError_t launch_dispatch(hipStream_t s, const void* X, int esize, int64_t T, int64_t n, int64_t ldx, int k,
                           const int32_t* inverse, int64_t R, void* Xs, int64_t lds) {
  if (T <= 0 || n <= 0 || k <= 0) return hipSuccess;
  const bool aligned = rows_aligned(X, ldx, esize) && rows_aligned(Xs, lds, esize) && (n * esize) % 16 == 0;
  const int64_t bytes = n * esize;
  const auto go = !aligned ? (bytes >= 16 ? dispatch_go<rt_u32x4_t, false, true>
                              : esize == 2 ? dispatch_go<uint16_t, false, false> : dispatch_go<uint32_t, false, false>)
                  : T * k * bytes > kStreamBytes ? dispatch_go<rt_u32x4_t, true, false>
                                                 : dispatch_go<rt_u32x4_t, false, false>;
  go(s, X, ldx * esize, T, bytes, k, inverse, R, Xs, lds * esize);
  return hipGetLastError();
}

template <bool YSBF, bool YBF, int MODE>
static void combine_mode(hipStream_t s, const CombineArgs& a) {
  const int64_t units = ceil_div(a.n, 8);
  hipLaunchKernelGGL((k_combine<YSBF, YBF, MODE>), dim3((unsigned)ceil_div(a.T * units, 256)), dim3(256), 0, s, a.Ys,
                     a.lds, (int)a.R, a.inverse, a.w, (uint32_t)a.T, (uint32_t)a.n, (uint32_t)units, a.k, a.Y, a.ldy);
}

template <bool YSBF, bool YBF>
static void combine_go(hipStream_t s, const CombineArgs& a) {
  if (a.n % 8 == 0 && rows_aligned(a.Ys, a.lds, YSBF ? 2 : 4) && rows_aligned(a.Y, a.ldy, YBF ? 2 : 4))
    combine_mode<YSBF, YBF, kAligned>(s, a);
  else if (a.n >= 8) combine_mode<YSBF, YBF, kAnywhere>(s, a);
  else combine_mode<YSBF, YBF, kSingly>(s, a);
}

hipError_t launch_combine(hipStream_t s, const CombineArgs& a) {
  if (a.T <= 0 || a.n <= 0) return hipSuccess;
  if (a.ys_bf16) a.y_bf16 ? combine_go<true, true>(s, a) : combine_go<true, false>(s, a);
  else a.y_bf16 ? combine_go<false, true>(s, a) : combine_go<false, false>(s, a);
  return hipGetLastError();
}

template <bool DYBF, bool YSBF, bool OBF, int MODE>
static void combine_grad_mode(hipStream_t s, const CombineGradArgs& a) {
  const int64_t passes = ceil_div(a.k, kCgSlots);
  const dim3 grid((unsigned)a.T, (unsigned)(a.T * passes <= 1024 ? passes : 1));
  hipLaunchKernelGGL((k_combine_grad<DYBF, YSBF, OBF, MODE>), grid, dim3(256), 0, s, a.dY, a.ldy, a.Ys, a.lds, a.R,
                     a.inverse, a.w, a.n, ceil_div(a.n, 8), a.k, a.dYs, a.ldo, a.dw);
}

template <bool DYBF, bool YSBF, bool OBF>
static void combine_grad_go(hipStream_t s, const CombineGradArgs& a) {
  if (a.n % 8 == 0 && rows_aligned(a.dY, a.ldy, DYBF ? 2 : 4) && rows_aligned(a.Ys, a.lds, YSBF ? 2 : 4) &&
      rows_aligned(a.dYs, a.ldo, OBF ? 2 : 4))
    combine_grad_mode<DYBF, YSBF, OBF, kAligned>(s, a);
  else if (a.n >= 8) combine_grad_mode<DYBF, YSBF, OBF, kAnywhere>(s, a);
  else combine_grad_mode<DYBF, YSBF, OBF, kSingly>(s, a);
}

hipError_t launch_combine_grad(hipStream_t s, const CombineGradArgs& a) {
  if (a.T <= 0 || a.k <= 0) return hipSuccess;
  switch ((a.dy_bf16 ? 4 : 0) | (a.ys_bf16 ? 2 : 0) | (a.out_bf16 ? 1 : 0)) {
    case 0: combine_grad_go<false, false, false>(s, a); break;
    case 1: combine_grad_go<false, false, true>(s, a); break;
    case 2: combine_grad_go<false, true, false>(s, a); break;
    case 3: combine_grad_go<false, true, true>(s, a); break;
    case 4: combine_grad_go<true, false, false>(s, a); break;
    case 5: combine_grad_go<true, false, true>(s, a); break;
    case 6: combine_grad_go<true, true, false>(s, a); break;
    default: combine_grad_go<true, true, true>(s, a); break;
  }
  return hipGetLastError();
}

}  // namespace gq

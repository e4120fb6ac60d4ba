// Packed layers with bias, activation, gate and residual, and their gradient.
//
//   z = X[rows[p]] W_hat_e^T + bias[e],  Y[p] = act(z) (or act(g) u) + residual[p]
//   dZ = dY act'(z)  (or (dY u act'(g), dY act(g))),  dbias[e] = sum_p dZ[p],
//   dX[p] = dZ[p] W_hat_e
//
// Forward: the kernels of the experts' products with what stands behind the
// product at their end, where the sums are in registers. It costs the bytes of
// the residual and of the kept z, against writing and reading R x m fp32 sums in
// a launch of its own (captured: 2048 rows of 4096 x 11008 gated 484 to 395 us,
// 4084 rows over 32 experts of 2048 x 1408 gated with z kept 157 to 133, one token
// of 4096 x 4096 with four waves 17.1 to 15.3). Only where K is in parts (few
// tiles) is it a launch of its own, which adds the parts (64 rows of 11008: 5.4 of
// 32 us).
#include "act.h"
#include "common.h"
#include "expert_tiles.h"

#include <algorithm>

namespace gq {

typedef ex_u32x4_t li_u32x4_t;
typedef ex_u32x4_any_t li_u32x4_any_t;
typedef ex_u32x2_t li_u32x2_any_t __attribute__((aligned(2)));
typedef ex_f32x4_t li_f32x4_any_t __attribute__((aligned(4)));

__device__ __forceinline__ float li_load(const void* p, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
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

// Four values of a row (`have` of them exist), at any alignment.
__device__ __forceinline__ ex_f32x4_t li_load4(const void* p, int bf16, int64_t at, int have) {
  ex_f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (have < 4) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < have) v[i] = li_load(p, bf16, at + i);
  } else if (bf16) {
    const ex_u32x2_t w = *reinterpret_cast<const li_u32x2_any_t*>(static_cast<const uint16_t*>(p) + at);
    v = (ex_f32x4_t){__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                     __uint_as_float(w[1] & 0xFFFF0000u)};
  } else {
    v = *reinterpret_cast<const li_f32x4_any_t*>(static_cast<const float*>(p) + at);
  }
  return v;
}
__device__ __forceinline__ void li_store4(void* p, int bf16, int64_t at, int have, ex_f32x4_t v) {
  if (have < 4) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < have) store_out(p, bf16, at + i, v[i]);
  } else if (bf16) {
    *reinterpret_cast<li_u32x2_any_t*>(static_cast<uint16_t*>(p) + at) = (ex_u32x2_t){ex_pack2(v[0], v[1]), ex_pack2(v[2], v[3])};
  } else {
    *reinterpret_cast<li_f32x4_any_t*>(static_cast<float*>(p) + at) = v;
  }
}

// ---------------------------------------------------------------- forward
// What stands behind the product. GATED: z0 of the gate, z1 of the other factor.
template <bool GATED_>
struct LinearEnd {
  static constexpr bool GATED = GATED_, STORES = true;
  // LDS of a wave: a block of 32 x 32 sums (two when gated), rows 36 apart: 16-byte pieces, all banks
  static constexpr uint32_t ROW = 144, BLOCK = 32 * ROW, LDS = BLOCK * (GATED ? 2 : 1);
  const float* bias; int64_t d;
  int act;
  const void* res; int res_bf16; int64_t ldr;
  void* Z; int z_bf16; int64_t ldz;
  void* Y; int y_bf16; int64_t ldy;
  explicit LinearEnd(const LinearArgs& a)
      : bias(a.bias), d(a.d), act(a.act), res(a.res), res_bf16(a.res_bf16), ldr(a.ldr), Z(a.Z), z_bf16(a.z_bf16), ldz(a.ldz),
        Y(a.Y), y_bf16(a.y_bf16), ldy(a.ldy) {}

  __device__ __forceinline__ float bias_of(int e, int h, int64_t o) const {
    return bias ? bias[(e * (GATED ? 2 : 1) + h) * d + o] : 0.f;
  }
  // one output, z without its bias
  __device__ __forceinline__ void one(int e, int64_t row, int64_t o, float z0, float z1) const {
    z0 += bias_of(e, 0, o);
    if (GATED) z1 += bias_of(e, 1, o);
    if (Z) {
      store_out(Z, z_bf16, row * ldz + o, z0);
      if (GATED) store_out(Z, z_bf16, row * ldz + d + o, z1);
    }
    float y = act_value(act, z0);
    if (GATED) y *= z1;
    if (res) y += li_load(res, res_bf16, row * ldr + o);
    store_out(Y, y_bf16, row * ldy + o, y);
  }

  // The 32 x 32 block(s) in LDS: eight rows at a time, four columns a lane.
  __device__ __forceinline__ void block(int e, int row0, int hi, int64_t o0, uint32_t lds) const {
    const int lane = threadIdx.x & 63, col = 4 * (lane & 7);
    const int64_t o = o0 + col;
    const int have = (int)min((int64_t)4, d - o);
    if (have <= 0) return;
    ex_f32x4_t b0 = {0.f, 0.f, 0.f, 0.f}, b1 = b0;
    if (bias) {
      b0 = li_load4(bias, 0, (int64_t)e * (GATED ? 2 : 1) * d + o, have);
      if (GATED) b1 = li_load4(bias, 0, ((int64_t)e * 2 + 1) * d + o, have);
    }
#pragma unroll 1
    for (int it = 0; it < 4; ++it) {
      const int r = 8 * it + (lane >> 3);
      const int64_t row = row0 + r;
      if (row >= hi) break;
      typedef __attribute__((address_space(3))) const ex_f32x4_t lds_f32x4_t;
      ex_f32x4_t z0 = *reinterpret_cast<lds_f32x4_t*>(lds + r * ROW + 4 * col), z1 = z0, y;
      z0 += b0;
      if (GATED) z1 = *reinterpret_cast<lds_f32x4_t*>(lds + BLOCK + r * ROW + 4 * col) + b1;
      if (Z) {
        li_store4(Z, z_bf16, row * ldz + o, have, z0);
        if (GATED) li_store4(Z, z_bf16, row * ldz + d + o, have, z1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = act_value(act, z0[i]) * (GATED ? z1[i] : 1.f);
      if (res) y += li_load4(res, res_bf16, row * ldr + o, have);
      li_store4(Y, y_bf16, row * ldy + o, have, y);
    }
  }

  // A wave's MI x NI blocks of 32 x 32 accumulators (value(mi, ni, r)), rows from
  // row0 on, the tile's first output o0, the wave's first block of columns block0.
  template <int MI, int NI, class V>
  __device__ __forceinline__ void store(int e, int row0, int hi, int64_t o0, int block0, uint32_t lds, V&& value) const {
    static_assert(!GATED || NI % 2 == 0, "a lane has both factors");
    const int lane = threadIdx.x & 63;
    const uint32_t at = lds + 4 * (lane >> 5) * ROW + 4 * (lane & 31);
    auto put = [&](auto M, auto N, uint32_t to) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        *reinterpret_cast<__attribute__((address_space(3))) float*>(to + (8 * (r >> 2) + (r & 3)) * ROW) = value(M, N, r);
    };
    auto rows = [&](auto M) {
      auto columns = [&](auto N) {
        if constexpr (decltype(N)::value < NI && !(GATED && decltype(N)::value % 2)) {
          put(M, N, at);
          if constexpr (GATED) put(M, ex_const<decltype(N)::value + 1>{}, at + BLOCK);
          asm volatile("" ::: "memory");                   // (a wave's own LDS operations keep their order)
          block(e, row0 + 32 * M, hi, o0 + (GATED ? 16 : 32) * (block0 + N), lds);
          asm volatile("" ::: "memory");
        }
      };
      if constexpr (decltype(M)::value < MI) for_four(columns);
    };
    for_four(rows);
  }
};

// Few rows: the matrix-vector form (MvWave), 32 packed rows (16 pairs when
// gated) of up to TILE rows of X.
template <int BITS, bool WIDE, bool GATED, int TILE, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 4)
k_linear_mv(ExArgs p, LinearEnd<GATED> finish) {
  constexpr int OB = 2, COLS = GATED ? 16 : 32;            // outputs
  __shared__ __align__(16) uint8_t smem[WAVES][MvWave<BITS, WIDE, OB, 1, TILE>::BYTES];
  __shared__ float red[WAVES][OB][4][64];
  const Seg sg = find_tile(p.offsets, p.E, p.R, TILE, blockIdx.y);
  if (sg.e < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15;
  const int64_t o0 = (int64_t)blockIdx.x * COLS;
  int64_t orow[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b)
    orow[b] = sg.e * p.d_out + (GATED ? b * finish.d : 0) + min(o0 + (GATED ? 0 : 16 * b) + li, finish.d - 1);
  const MvRows<OB> w(p.qw, p.scales, p.zeros, orow, p.n, p.group, BITS);
  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int nrows = min(sg.hi - sg.row0, TILE);
  mv_sum<BITS, WIDE, OB, 1, TILE>(w, p.n, p.group, wave, WAVES, nrows, 0, lds_addr(smem[wave]),
                                  mv_vec(p.scales, p.zeros, p.n, p.group),
                                  [&](int r) { return p.A + source_row(p.rows, sg.row0 + r, p.T) * p.lda; }, tot);
#pragma unroll
  for (int b = 0; b < OB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][b][r][lane] = tot[b][r];
  __syncthreads();
  for (int i = threadIdx.x; i < (GATED ? 1 : OB) * 256; i += 64 * WAVES) {
    const int b = i >> 8, r = (i >> 6) & 3, l = i & 63, row = 4 * (l >> 4) + r;
    const int64_t o = o0 + 16 * b + (l & 15);
    if (o >= finish.d || row >= nrows) continue;
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
      for (int v = 0; v < WAVES; ++v) z[h] += red[v][GATED ? h : b][r][l];
    finish.one(sg.e, sg.row0 + row, o, z[0], z[1]);
  }
}

// K in parts: their sums in order, and what follows. (Parts are of few tiles: at
// most 2^14 rows.)
template <bool GATED>
__global__ void __launch_bounds__(256)
k_linear_end(const float* __restrict__ part, int splits, int64_t m, const int32_t* __restrict__ offsets, int E, int R,
             LinearEnd<GATED> finish) {
  const int64_t row = blockIdx.y, o = (int64_t)blockIdx.x * 256 + threadIdx.x, d = finish.d;
  if (o >= d || (offsets && (row < offsets[0] || row >= offsets[E]))) return;
  const int e = finish.bias && offsets ? li_expert(offsets, E, row) : 0;
  float z[2] = {0.f, 0.f};
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h)
    for (int s = 0; s < splits; ++s) z[h] += part[(s * (int64_t)R + row) * m + h * d + o];
  finish.one(e, row, o, z[0], z[1]);
}

size_t linear_workspace(int64_t R, int E, int64_t n, int64_t m, int group) {
  return expert_split(R, E, n, m, group, 0, false).part_bytes;
}

// Eight waves share K where workgroups are few: 4096 x 4096 for one token (128
// workgroups) 9.0 us with four waves, 7.8 with eight, 11008 x 4096 (344) 11.6 and
// 10.5, gated (688) 17.5 and 18.9 captured.
template <int BITS, bool WIDE, bool GATED, int TILE>
static void linear_mv(hipStream_t s, const LinearArgs& a) {
  const ExArgs p = ex_args(a.mm, TILE, 1, 1);
  const dim3 grid((unsigned)ceil_div(a.d, GATED ? 16 : 32), (unsigned)p.nrt);
  if ((int64_t)grid.x * std::min<int64_t>(p.nrt, a.mm.R) <= 512)
    hipLaunchKernelGGL((k_linear_mv<BITS, WIDE, GATED, TILE, 8>), grid, dim3(512), 0, s, p, LinearEnd<GATED>(a));
  else
    hipLaunchKernelGGL((k_linear_mv<BITS, WIDE, GATED, TILE, 4>), grid, dim3(256), 0, s, p, LinearEnd<GATED>(a));
}

template <int BITS, bool GATED, class TL, int GS>
static void linear_tiles(hipStream_t s, const LinearArgs& a) {
  static_assert(TL::WM * TL::WN * LinearEnd<GATED>::LDS <= 2 * (TL::BM + TL::BN) * 128, "the blocks fit the tiles' LDS");
  ExArgs p = ex_args(a.mm, TL::BM, TL::BN, a.mm.d_out);
  p.nct = (int)ceil_div(a.d, GATED ? TL::BN / 2 : TL::BN);
  p.per_split = (int)ceil_div(a.mm.n, kExBK);
  hipLaunchKernelGGL((k_expert_mm<BITS, TL, GS, LinearEnd<GATED>>), tile_grid(p.nrt, p.nct), dim3(TL::THREADS), 0, s, p,
                     LinearEnd<GATED>(a));
}
template <int BITS, bool GATED, class TL>
static void linear_group(hipStream_t s, const LinearArgs& a) {
  if constexpr (BITS == 4) {
    if (a.mm.group == 128) return linear_tiles<4, GATED, TL, 2>(s, a);
    if constexpr (TL::BM == 64) {
      if (a.mm.group == 64) return linear_tiles<4, GATED, TL, 1>(s, a);
    }
  }
  linear_tiles<BITS, GATED, TL, 0>(s, a);
}

// 64-row tiles in which a wave has two blocks of columns.
using ExTile64Pair = ExTile<1, 2, 2, 2, 4, 4>;

// The matrix-vector form beyond the 16 rows an expert of the plain product. Where
// tiles are few, 64-row tiles have K in parts, and a launch that adds these.
// Matrix-vector form and 64-row tiles, captured, us:
//  * four parts or more: 17, 32, 40 and 48 rows of 11008 x 4096 19.5, 20.5, 27 and
//    29 against 28, 28, 29 and 31 (64 rows: equal), 32 gated 32 and 43; 40 rows for
//    each of 8 experts of 1024 x 4096 21.5 and 32; groups of 64 with 24, 32 and 40
//    rows 24, 25, 34 and 28, 28, 29
//  * two or three: 24 rows of 28672 x 8192 72 and 77, 48 rows 100 and 82; 24 for
//    each of 8 of 4096 x 4096 43 and 54; groups of 64 95 and 86, 55 and 58
//  * one: 24 rows for each of 32 of 1408 x 2048 41 and 46, of 64 76 and 71 (gated
//    135 and 121), 32 of each of 32 48 and 46
//  * 3 bits, whose tiles are slower: 24 and 48 rows of 11008 x 4096 24, 33 and 48,
//    51; 48 of each of 8 of 4096 x 4096 82 and 122; 47 of each of 32 of 1408 x 2048
//    70 and 77
// Eight threads a packed row here, two in the tiles: beyond 2^29 rows only the
// tiles' launch has fewer than 2^32.
constexpr int64_t kMvMaxBlocks = (((int64_t)1 << 32) - 512) / 256;
static bool linear_few(const LinearArgs& a) {
  if (!bf16_rows_vec(a.mm.A, a.mm.lda, a.mm.n)) return false;
  if (ceil_div(a.mm.d_out, 32) > kMvMaxBlocks) return false;
  const int64_t avg = ceil_div(a.mm.R, a.mm.E);
  if (a.mm.bits == 3) return avg <= 48;
  const int parts = expert_split(a.mm.R, a.mm.E, a.mm.n, a.mm.d_out, a.mm.group, 0, false).splits;
  const bool wide = a.mm.group % 128 == 0;
  return avg <= (parts >= 4 ? (wide ? 48 : 32) : parts > 1 && wide ? 24 : 16);
}

template <int BITS, bool GATED>
static hipError_t linear_go(hipStream_t s, const LinearArgs& a) {
  const int bm = linear_few(a) ? 16 : expert_bm(a.mm, 0);
  if (bm == 16) {
    const bool wide = a.mm.group % 128 == 0, low = a.mm.R <= 8 * (int64_t)a.mm.E;
    if (wide && low) linear_mv<BITS, true, GATED, 8>(s, a);
    else if (wide) linear_mv<BITS, true, GATED, 16>(s, a);
    else if (low) linear_mv<BITS, false, GATED, 8>(s, a);
    else linear_mv<BITS, false, GATED, 16>(s, a);
    return hipGetLastError();
  }
  const ExpertSplit sp = expert_split(a.mm.R, a.mm.E, a.mm.n, a.mm.d_out, a.mm.group, 0, false);
  if (bm != 256 && sp.splits > 1) {
    ExpertArgs e = a.mm;
    e.part = a.ws;
    e.parts_only = true;
    const hipError_t err = launch_expert_mm(s, e);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_linear_end<GATED>, dim3((unsigned)ceil_div(a.d, 256), (unsigned)e.R), dim3(256), 0, s,
                       static_cast<const float*>(a.ws), sp.splits, e.d_out, e.offsets, e.E, e.R, LinearEnd<GATED>(a));
    return hipGetLastError();
  }
  if (bm == 256) {
    if constexpr (BITS == 4) {
      ExArgs p = ex_args(a.mm, 256, 256, a.mm.d_out);
      p.nct = (int)ceil_div(a.d, GATED ? 128 : 256);
      hipLaunchKernelGGL(k_expert_ring<LinearEnd<GATED>>, tile_grid(p.nrt, p.nct), dim3(512), 0, s, p, LinearEnd<GATED>(a));
    }
  } else if (bm == 64) {
    linear_group<BITS, GATED, std::conditional_t<GATED, ExTile64Pair, ExTile64>>(s, a);
  } else {
    linear_group<BITS, GATED, ExTile128>(s, a);
  }
  return hipGetLastError();
}

hipError_t launch_linear(hipStream_t s, const LinearArgs& a) {
  if (a.mm.bits == 2) return a.gated ? linear_go<2, true>(s, a) : linear_go<2, false>(s, a);
  if (a.mm.bits == 3) return a.gated ? linear_go<3, true>(s, a) : linear_go<3, false>(s, a);
  return a.gated ? linear_go<4, true>(s, a) : linear_go<4, false>(s, a);
}

// ---------------------------------------------------------------- gradient
// dZ is rounded to bf16, the product's operand, once, also for an fp32 dX: two
// pieces of it would double that product (4096 rows of 11008 x 4096: 344 us, 1150
// for an fp32 dX, whose weights are in three pieces). An fp32 dX is off by 0.0017 of
// itself for that, a bf16 one, with its own rounding and the weights', by 0.0029.
//
// dZ and the partial sums of dbias, bound by their bytes. A workgroup owns
// kLgRows rows of one segment and 256 columns of dY: 32 lanes of eight
// columns side by side, eight rows side by side. Its column sums go to
// part[tile][m], and a second launch adds a segment's tiles in their order.
// 4096 rows of 11008 with gelu 67 us (270 MB, 55 us at the rate of a copy), 1934
// of 2 x 1408 with silu 14.6; with 64 rows, two on their way at a time, and
// erfcf 93 and 21.
constexpr int kLgRows = 32;

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
        (li_u32x4_t){ex_pack2(f[0], f[1]), ex_pack2(f[2], f[3]), ex_pack2(f[4], f[5]), ex_pack2(f[6], f[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) p[i] = (uint16_t)ex_pack2(f[i], 0.f);
  }
}

// One activation's code (the switch over them stands outside of the loops).
template <int ACT, bool YBF, bool ZBF, bool GATED>
__device__ __forceinline__ void li_dz(const LinearGradArgs& a, int r0, int r1, int64_t c, int have, float (&sg)[8],
                                      float (&su)[8]) {
  constexpr int U = kLgRows / 8;                           // rows of a lane, all on their way at once
  const int rl = threadIdx.x >> 5;
  const int r = r0 + rl;
  {
    float dy[U][8], z[U][8], u[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = min(r + 8 * i, r1 - 1);
      li_row8<YBF>(a.dY, row * a.ldy + c, have, dy[i]);
      if (a.Z) li_row8<ZBF>(a.Z, row * a.ldz + c, have, z[i]);
      if constexpr (GATED) li_row8<ZBF>(a.Z, row * a.ldz + a.d + c, have, u[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = r + 8 * i;
      if (row >= r1) break;
      float dg[8], du[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float slope = 1.f, v = z[i][e];
        if constexpr (ACT != GPTQ_ACT_NONE) v = act_both(ACT, v, slope);
        dg[e] = dy[i][e] * slope;
        if constexpr (GATED) {
          dg[e] = dy[i][e] * u[i][e] * slope;
          du[e] = dy[i][e] * v;
          su[e] += du[e];
        }
        sg[e] += dg[e];
      }
      if (a.dZ) {
        li_store8(a.dZ + row * a.lddz + c, have, dg);
        if constexpr (GATED) li_store8(a.dZ + row * a.lddz + a.d + c, have, du);
      }
    }
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
    switch (a.act) {
      case GPTQ_ACT_RELU: li_dz<GPTQ_ACT_RELU, YBF, ZBF, GATED>(a, r0, r1, c, have, sg_, su_); break;
      case GPTQ_ACT_GELU: li_dz<GPTQ_ACT_GELU, YBF, ZBF, GATED>(a, r0, r1, c, have, sg_, su_); break;
      case GPTQ_ACT_GELU_TANH: li_dz<GPTQ_ACT_GELU_TANH, YBF, ZBF, GATED>(a, r0, r1, c, have, sg_, su_); break;
      case GPTQ_ACT_SILU: li_dz<GPTQ_ACT_SILU, YBF, ZBF, GATED>(a, r0, r1, c, have, sg_, su_); break;
      default: li_dz<GPTQ_ACT_NONE, YBF, ZBF, GATED>(a, r0, r1, c, have, sg_, su_); break;
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

// A segment's tiles in four parts, each in its order, then the parts. 64 columns
// a workgroup. `tiles`: li_tiles, what part holds. Segments that overlap (offsets
// that fall) may have more between them: those beyond have no sums and count for
// nothing, and the sums of their numbers stop there, so that none leaves 32 bits.
__global__ void __launch_bounds__(256)
k_linear_dbias(const float* __restrict__ part, const int32_t* __restrict__ offsets, int E, int R, int tiles, int64_t m,
               float* __restrict__ dbias) {
  __shared__ float sums[4][64];
  const int e = blockIdx.y, lane = threadIdx.x & 63, q = threadIdx.x >> 6;
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
      for (int i = 32; i > 0; i >>= 1) t = min(t + __shfl_xor(t, i), tiles);
      first = min(first + t, tiles);
    }
    count = min(count, tiles - first);
  }
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int per = (count + 3) / 4, end = min(count, (q + 1) * per);
  float v = 0.f;
  if (c < m) {
#pragma unroll 8
    for (int t = q * per; t < end; ++t) v += part[(int64_t)(first + t) * m + c];
  }
  sums[q][lane] = v;
  __syncthreads();
  if (q == 0 && c < m) dbias[(int64_t)e * m + c] = sums[0][lane] + sums[1][lane] + sums[2][lane] + sums[3][lane];
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
    hipLaunchKernelGGL(k_linear_dbias, dim3((unsigned)ceil_div(a.m, 64), (unsigned)a.mm.E), dim3(256), 0, s, a.part,
                       a.mm.offsets, a.mm.E, a.mm.R, (int)li_tiles(a.mm.R, a.mm.E), a.m, a.dbias);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return a.mm.R > 0 ? launch_expert_mm_grad(s, a.mm) : hipSuccess;
}

}  // namespace gq

// Products of experts' packed weights, their gradient, and the weight
// gradient from activations kept in 8 bits. All three work on rows that are
// contiguous per expert (route.hip): segment e holds the rows
// p in [offsets[e], offsets[e + 1]), and the counts stay on the device.
//
//   forward   Y[p]  = X[rows[p]] W_hat_e^T,      W_hat = s (q - z)
//   gradient  dX[p] = dY[p] W_hat_e
//   weights   G_e   = sum_{p in segment e} P[p]^T x_hat[rows[p]]
//
// The host knows the number of rows R but not the segments, so a launch has
// ceil(R / BM) + E - 1 row tiles of BM rows, enough for any split of R rows
// into E segments (each segment wastes less than one tile); a workgroup
// finds its segment from the offsets with one wave-wide sum per 64 experts,
// and a tile past the last one ends at once. offsets are clamped to
// [0, R] and rows to [0, T), so wrong ones give wrong values and no access
// out of bounds. Rows from offsets[E] on are neither read nor written.
#include "common.h"
#include "dma.h"

#include <algorithm>
#include <type_traits>

namespace gq {

typedef __bf16 ex_bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 ex_bf16x2_t __attribute__((ext_vector_type(2)));
typedef float ex_f32x16_t __attribute__((ext_vector_type(16)));
typedef float ex_f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int ex_u32x4_t __attribute__((ext_vector_type(4)));
typedef ex_u32x4_t ex_u32x4_any_t __attribute__((aligned(2)));

struct Seg {
  int e;        // expert, -1: no such tile
  int lo, hi;   // its rows
  int row0;     // the tile's first row
};

// Inclusive sum over the wave by lane shifts inside and across its rows of 16
// (no LDS traffic: this stands in front of every product).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast 31 into rows 2, 3
  return v;
}

// The segments of up to 64 experts from e0 on, one per lane, and the
// inclusive sums of their row tiles.
struct SegScan {
  int lo, hi, nt, inc;
};
__device__ __forceinline__ SegScan scan_segments(const int32_t* __restrict__ offsets, int E, int R, int BM, int e0) {
  const int e = e0 + (threadIdx.x & 63);
  SegScan s = {0, 0, 0, 0};
  if (e < E) {
    s.lo = min(max(offsets[e], 0), R);
    s.hi = min(max(offsets[e + 1], s.lo), R);
  }
  s.nt = (s.hi - s.lo + BM - 1) / BM;
  s.inc = wave_scan(s.nt);
  return s;
}

// Row tile rt, if it is among the 64 experts of s (`before` tiles precede them).
__device__ __forceinline__ bool pick_segment(const SegScan& s, int e0, int before, int BM, int rt, Seg& sg) {
  const uint64_t past = __ballot(before + s.inc > rt);
  if (!past) return false;
  const int l = __ffsll((long long)past) - 1;
  const int lo = __builtin_amdgcn_readlane(s.lo, l), hi = __builtin_amdgcn_readlane(s.hi, l);
  const int first = before + __builtin_amdgcn_readlane(s.inc - s.nt, l);
  sg = Seg{e0 + l, lo, hi, lo + (rt - first) * BM};
  return true;
}

// Row tile rt of BM rows (every wave of the workgroup finds it for itself).
__device__ __forceinline__ Seg find_tile(const int32_t* __restrict__ offsets, int E, int R, int BM, int rt) {
  Seg sg = {-1, 0, 0, 0};
  if (offsets == nullptr) {
    if ((int64_t)rt * BM < R) sg = Seg{0, 0, R, rt * BM};
    return sg;
  }
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const SegScan s = scan_segments(offsets, E, R, BM, e0);
    if (pick_segment(s, e0, before, BM, rt, sg)) break;
    before += __builtin_amdgcn_readlane(s.inc, 63);
  }
  return sg;
}

// Source row of sorted row p (rows == nullptr: p itself).
__device__ __forceinline__ int64_t source_row(const int32_t* __restrict__ rows, int p, int T) {
  const int r = rows ? rows[p] : p;
  return min(max(r, 0), T - 1);
}

__device__ __forceinline__ uint32_t ex_pack2(float a, float b) {
  const ex_bf16x2_t p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ void store_out(void* Y, int bf16, int64_t i, float v) {
  if (bf16) static_cast<uint16_t*>(Y)[i] = (uint16_t)ex_pack2(v, 0.f);
  else static_cast<float*>(Y)[i] = v;
}

// The 32 codes of a chunk (BITS words) as integers of a register array.
template <int BITS>
__device__ __forceinline__ void load_chunk(const uint32_t* __restrict__ p, uint32_t (&w)[BITS]) {
  if constexpr (BITS == 4) {
    const ex_u32x4_t v = *reinterpret_cast<const ex_u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) w[i] = p[i];
  }
}

// Codes 8 j .. 8 j + 7 of a chunk of 2- or 3-bit codes, minus z, as floats
// (exact).
template <int BITS>
__device__ __forceinline__ void codes8(const uint32_t (&w)[BITS], int j, float z, float (&f)[8]) {
  static_assert(BITS < 4, "4-bit codes go by mv_codes<4>");
  const int base = 8 * BITS * j, wi = base >> 5, sh = base & 31;
  uint64_t v = w[wi];
  if constexpr (BITS == 3) {
    if (wi + 1 < BITS) v |= (uint64_t)w[wi + 1] << 32;
  }
  v >>= sh;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)(uint32_t)((v >> (BITS * i)) & ((1u << BITS) - 1u)) - z;
}

// Two floats whose low halves are zero (small integers, kept values) as bf16.
__device__ __forceinline__ uint32_t pack_exact(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// ==================================================================== few rows
//
// Matrix-vector products: bound by reading the packed weights once. A
// workgroup of WAVES waves owns 16 OB outputs of one expert and up to 16 of
// its rows (v_mfma_f32_16x16x32_bf16, X as the A operand), and its waves
// split K. K advances in pieces of 128 codes.
//  * Groups that are multiples of 128 (WIDE): lane l (output l % 16,
//    j = l / 16) loads the 32 consecutive codes 32 j .. of its output's piece
//    in one go (16 bytes at 4 bits); MFMA step i then takes codes
//    32 j + 8 i .. + 7 of every lane. The order of K inside a product is
//    free as long as X's fragment follows it.
//  * Other groups: a product must not mix groups, so step i takes chunk i of
//    the piece and lane j its codes 8 j .. + 7, and the sum is scaled after
//    every chunk. At 4 bits a lane still loads a chunk in one go and four lane
//    swaps hand out its words (360 rows over 64 experts, 322 x 4608 in groups
//    of 32: 73 us with a word per load, 36 us so).
//  * 4 bits: a code in bits 3..6 of the bf16 pattern of 16 is the number
//    16 + q, so one shift and one and-or give two codes (pairs i, i + 4: X's
//    fragment is permuted alike), one operation per code against three with
//    conversions. The offset and the zero point leave through
//    sum_k x (q - z) = sum_k x (16 + q) - (16 + z) sum_k x, the last sum
//    formed by one more product with ones, shared by the OB blocks. All of
//    it in fp32: the offset costs up to a factor of about 6 of fp32's
//    rounding. A row with an infinity gives NaN, and so may one whose sum of
//    128 x (16 + q) leaves fp32: 128 31 2^116 is below 2^128.
//
// Measured (median kernel times; two experts of 11008 x 4096 for one token /
// 64 experts of 1408 x 2048 for 256 rows, 4 bits, groups of 128; 48.6 and 99
// MB, 10 and 20 us at the rate of a large copy): 19.9 / 31.8 us. Of it about 2
// are the launch and the look-up, 6 / 10 the unpacking and the products,
// the rest the weights' way from memory. One load per scale and piece instead
// of one per S pieces: 22.9 / 42.5; 8 waves per workgroup 22.0 / 67;
// 16 outputs per wave 19.8 / 40; 64 outputs 23.5 / 32.6; the weights loaded
// past the caches 20.9 / 32.9. In captured calls, which take 20.3 / 32.5: four
// pieces asked for at a time 19.6 / 33.0, one 24.6 / 38.0.
template <int BITS>
__device__ __forceinline__ ex_bf16x8_t mv_window(const uint32_t* __restrict__ chunk, int j, float z) {
  const int base = 8 * BITS * j, wi = base >> 5;
  uint64_t v = chunk[wi];
  if constexpr (BITS == 3) v |= (uint64_t)chunk[min(wi + 1, BITS - 1)] << 32;
  v >>= base & 31;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)(uint32_t)((v >> (BITS * i)) & ((1u << BITS) - 1u)) - z;
  const ex_u32x4_t u = {pack_exact(f[0], f[1]), pack_exact(f[2], f[3]), pack_exact(f[4], f[5]), pack_exact(f[6], f[7])};
  return __builtin_bit_cast(ex_bf16x8_t, u);
}

template <int BITS>
__device__ __forceinline__ ex_bf16x8_t mv_codes(const uint32_t (&w)[BITS], int i, float z) {
  if constexpr (BITS == 4) {
    const uint32_t v = w[i];
    const ex_u32x4_t u = {((v << 3) & 0x00780078u) | 0x41804180u, ((v >> 1) & 0x00780078u) | 0x41804180u,
                          ((v >> 5) & 0x00780078u) | 0x41804180u, ((v >> 9) & 0x00780078u) | 0x41804180u};
    return __builtin_bit_cast(ex_bf16x8_t, u);
  } else {
    float f[8];
    codes8<BITS>(w, i, z, f);
    const ex_u32x4_t u = {pack_exact(f[0], f[1]), pack_exact(f[2], f[3]), pack_exact(f[4], f[5]),
                          pack_exact(f[6], f[7])};
    return __builtin_bit_cast(ex_bf16x8_t, u);
  }
}

// x0..x7 -> x0 x4 x1 x5 x2 x6 x3 x7, the order of mv_codes<4>
__device__ __forceinline__ ex_bf16x8_t mv_order(ex_u32x4_t x) {
  const ex_u32x4_t u = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                        __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
  return __builtin_bit_cast(ex_bf16x8_t, u);
}

// w[i] of lane group j (16 lanes) <-> w[j] of lane group i.
__device__ __forceinline__ void mv_transpose(uint32_t (&w)[4]) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {   // a's upper 32 lanes with b's lower
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {   // a's odd rows of 16 with b's even ones
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
}

template <int BITS, bool WIDE, int WAVES, int OB, int S>
__global__ void __launch_bounds__(64 * WAVES)
k_expert_mv(const uint16_t* __restrict__ X, int T, int64_t n, int64_t ldx, const int32_t* __restrict__ rows,
            const int32_t* __restrict__ offsets, int E, int R, const uint32_t* __restrict__ qw,
            const float* __restrict__ scales, const uint8_t* __restrict__ zeros, int64_t d_out, int group,
            void* __restrict__ Y, int ybf16, int64_t ldy) {
  __shared__ float red[WAVES][OB][4][64];
  const Seg sg = find_tile(offsets, E, R, 16, blockIdx.y);
  if (sg.e < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane >> 4, li = lane & 15;
  const int64_t ngroups = n / group, wpr = n / 32 * BITS;
  const int nchunks = (int)(n / 32), npieces = (nchunks + 3) / 4;
  const int64_t obase = (int64_t)sg.e * d_out;
  const uint32_t* qrow[OB];
  const float* srow[OB];
  const uint8_t* zrow[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) {
    const int64_t o = obase + min((int64_t)blockIdx.x * (16 * OB) + 16 * b + li, d_out - 1);
    qrow[b] = qw + o * wpr;
    srow[b] = scales + o * ngroups;
    zrow[b] = zeros + o * ngroups;
  }
  // lanes of rows past the segment load nothing: rows of the product do not
  // mix, and their results are not stored
  const bool xok = sg.row0 + li < sg.hi;
  const int prow = min(sg.row0 + li, sg.hi - 1);
  int srcrow = rows ? rows[prow] : prow;

  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  const ex_u32x4_t ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const ex_bf16x8_t ones = __builtin_bit_cast(ex_bf16x8_t, ones_bits);

  if constexpr (WIDE) {
    // a wave owns consecutive pieces, four at a time: a row's 64 bytes per
    // piece then share cache lines, and one load brings the scales (zero
    // points) of the four, lane j's for piece j
    const int per = (npieces + WAVES - 1) / WAVES;
    const int pbeg = wave * per, pend = min(npieces, pbeg + per);
    for (int p0 = pbeg; p0 < pend; p0 += S) {
      uint32_t w[S][OB][BITS];
      ex_u32x4_t x[S][4];
      float s[OB];
      uint32_t z[OB];
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int b = 0; b < OB; ++b)
          load_chunk<BITS>(qrow[b] + ((int64_t)min(p0 + u, pend - 1) * 4 + j) * BITS, w[u][b]);
      const int64_t g = (int64_t)min(p0 + (j & (S - 1)), pend - 1) * 128 / group;
#pragma unroll
      for (int b = 0; b < OB; ++b) {
        s[b] = srow[b][g];
        z[b] = zrow[b][g];
      }
      // the weights leave before the row's index is waited for
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" : "+v"(srcrow));
      const uint16_t* __restrict__ xrow = X + (int64_t)min(max(srcrow, 0), T - 1) * ldx;
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("" : "=v"(x[u][i]));   // any value
      if (xok) {
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[u][i] = *reinterpret_cast<const ex_u32x4_t*>(xrow + (int64_t)min(p0 + u, pend - 1) * 128 + 32 * j + 8 * i);
      }
#pragma unroll
      for (int u = 0; u < S; ++u) {
        if (p0 + u >= pend) break;
        ex_f32x4_t acc[OB], xs = {0.f, 0.f, 0.f, 0.f};
        float su[OB], zu[OB];
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          acc[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
          su[b] = __shfl(s[b], 16 * u + li);
          zu[b] = (float)__shfl((int)z[b], 16 * u + li);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ex_bf16x8_t a = BITS == 4 ? mv_order(x[u][i]) : __builtin_bit_cast(ex_bf16x8_t, x[u][i]);
#pragma unroll
          for (int b = 0; b < OB; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, mv_codes<BITS>(w[u][b], i, zu[b]), acc[b], 0, 0, 0);
          if constexpr (BITS == 4) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, xs, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < OB; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = BITS == 4 ? fmaf(-(16.f + zu[b]), xs[r], acc[b][r]) : acc[b][r];
            tot[b][r] = fmaf(su[b], v, tot[b][r]);
          }
      }
    }
  } else if constexpr (BITS == 4) {
    // lane j loads chunk j of a piece (16 bytes) and the four words of each
    // chunk then change lanes, so that step i has chunk i: word j in lane j
    const int per = (npieces + WAVES - 1) / WAVES;
    const int pbeg = wave * per, pend = min(npieces, pbeg + per);
    for (int p0 = pbeg; p0 < pend; p0 += S) {
      uint32_t w[S][OB][4];
      ex_u32x4_t x[S][4];
      float s[S][OB];
      uint32_t z[S][OB];
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int c = min(4 * min(p0 + u, pend - 1) + j, nchunks - 1);
        const int64_t g = (int64_t)c * 32 / group;
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          load_chunk<4>(qrow[b] + (int64_t)c * 4, w[u][b]);
          s[u][b] = srow[b][g];
          z[u][b] = zrow[b][g];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" : "+v"(srcrow));
      const uint16_t* __restrict__ xrow = X + (int64_t)min(max(srcrow, 0), T - 1) * ldx;
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("" : "=v"(x[u][i]));   // any value
      if (xok) {
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = min(4 * min(p0 + u, pend - 1) + i, nchunks - 1);
            x[u][i] = *reinterpret_cast<const ex_u32x4_t*>(xrow + (int64_t)c * 32 + 8 * j);
          }
      }
#pragma unroll
      for (int u = 0; u < S; ++u) {
        if (p0 + u >= pend) break;
#pragma unroll
        for (int b = 0; b < OB; ++b) mv_transpose(w[u][b]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (4 * (p0 + u) + i >= nchunks) break;
          const ex_bf16x8_t a = mv_order(x[u][i]);
          const ex_f32x4_t none = {0.f, 0.f, 0.f, 0.f};
          const ex_f32x4_t xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, none, 0, 0, 0);
#pragma unroll
          for (int b = 0; b < OB; ++b) {
            const ex_f32x4_t acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, mv_codes<4>(w[u][b], i, 0.f), none, 0, 0, 0);
            const float si = __shfl(s[u][b], 16 * i + li), zi = 16.f + (float)__shfl((int)z[u][b], 16 * i + li);
#pragma unroll
            for (int r = 0; r < 4; ++r) tot[b][r] = fmaf(si, fmaf(-zi, xs[r], acc[r]), tot[b][r]);
          }
        }
      }
    }
  } else {
    const uint16_t* __restrict__ xrow = X + (int64_t)min(max(srcrow, 0), T - 1) * ldx;
    for (int p = wave; p < npieces; p += WAVES) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 4 * p + i;
        if (c >= nchunks) break;
        const int64_t g = (int64_t)c * 32 / group;
        const ex_bf16x8_t a = *reinterpret_cast<const ex_bf16x8_t*>(xrow + (int64_t)c * 32 + 8 * j);
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          ex_f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a, mv_window<BITS>(qrow[b] + (int64_t)c * BITS, j, (float)zrow[b][g]), acc, 0, 0, 0);
          const float s = srow[b][g];
#pragma unroll
          for (int r = 0; r < 4; ++r) tot[b][r] = fmaf(s, acc[r], tot[b][r]);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < OB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][b][r][lane] = tot[b][r];
  __syncthreads();
  // the waves' sums in wave order
  for (int i = threadIdx.x; i < OB * 256; i += 64 * WAVES) {
    const int b = i >> 8, r = (i >> 6) & 3, l = i & 63;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += red[w][b][r][l];
    const int64_t o = (int64_t)blockIdx.x * (16 * OB) + 16 * b + (l & 15);
    const int row = sg.row0 + 4 * (l >> 4) + r;
    if (o < d_out && row < sg.hi) store_out(Y, ybf16, (int64_t)row * ldy + o, v);
  }
}

// ==================================================================== many rows
//
// A BM x 128 tile per workgroup (v_mfma_f32_32x32x16_bf16; wave (wm, wn) holds
// MI x NI blocks of 32 x 32). K advances in stages of 64 through two LDS
// buffers. The operands of the next DA and DB stages are on their way into
// registers and those of stage st + 1 are written into the other buffer, the packed one
// expanded to bf16 on its way, in between the products of stage st: one
// barrier per stage, and the expansion (once per workgroup, about three
// operations per code) runs beside the matrix cores. Operand layouts in LDS
// (64 banks: 16 lanes of 16 bytes meet in a
// clock):
//  * K along a row ([row][64], 128 bytes): 16-byte piece c of row r at
//    c ^ ((r / 2) & 7), so sixteen rows' reads of one piece hit all banks;
//  * K down the rows ([64][W]): piece c of row t at c ^ dma_swz(t) ^ x, read
//    with the transposing LDS read; x (a bit of the row or of the column)
//    keeps the writes of wide column runs off each other's banks.
constexpr int kExBK = 64;

// DA, DB: stages of A and B on their way into registers (the loads of stage
// st + D leave at the start of stage st).
template <int MI_, int NI_, int WM_, int WN_, int DA_, int DB_>
struct ExTile {
  static constexpr int DA = DA_, DB = DB_, U = DA_ > 2 || DB_ > 2 ? 4 : 2;   // stages per loop body
  static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = WN_;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NI * WN, THREADS = 64 * WM * WN;
  static constexpr int PA = BM * 8 / THREADS;   // 16-byte pieces of A per thread and stage
  static constexpr int NB = BN * 8 / THREADS;   // 8-code units of B per thread and stage
};
using ExTile128 = ExTile<2, 2, 2, 2, 1, 2>;    // 128 x 128
using ExTile64 = ExTile<2, 1, 1, 4, 4, 4>;     // 64 x 128: little work per stage to hide a load behind
using ExTile32 = ExTile<1, 1, 1, 4, 4, 4>;     // 32 x 128

typedef __attribute__((address_space(3))) ex_u32x4_t lds_piece_t;
typedef __attribute__((address_space(3))) const ex_bf16x8_t lds_frag_t;

__device__ __forceinline__ uint32_t row_piece(int r, int c) { return (uint32_t)r * 128u + 16u * (c ^ ((r >> 1) & 7)); }
// W: columns of the tile
template <int W>
__device__ __forceinline__ uint32_t col_piece(int t, int c) {
  const int x = W == 128 ? (t >> 1) & 1 : (c >> 4) & 1;
  return (uint32_t)t * (2 * W) + 16u * (c ^ dma_swz(t) ^ x);
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void lds_write(uint32_t at, ex_u32x4_t v) { *reinterpret_cast<lds_piece_t*>(at) = v; }
__device__ __forceinline__ ex_bf16x8_t lds_frag(uint32_t at) { return *reinterpret_cast<lds_frag_t*>(at); }

// Address of this lane's fragment of columns c0 .. c0 + 31 in a [64][W] tile
// (K slice kk at + 32 W kk): lane l gets K 8 (l / 32) .. + 7 of column
// c0 + l % 32 by two transposing reads.
template <int W>
__device__ __forceinline__ uint32_t col_frag_at(int c0, int lane) {
  const int t = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int col = c0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  return col_piece<W>(t, col >> 3) + 2 * (col & 7);
}
template <int W>
__device__ __forceinline__ ex_bf16x8_t lds_col_frag(uint32_t at) {
  struct { v4i16_t a, b; } f = {lds_tr16(at), lds_tr16(at + 4 * 2 * W)};
  return __builtin_bit_cast(ex_bf16x8_t, f);
}

// 8 elements of a bf16 row from column c (limit: the row's length). WIDE, at
// least 8 columns: one 16-byte load at any alignment, moved back to end with
// the row (end_piece puts that right); otherwise element by element.
template <bool WIDE>
__device__ __forceinline__ ex_u32x4_t load_piece(const uint16_t* __restrict__ row, int64_t c, int64_t limit) {
  if constexpr (WIDE) {
    return *reinterpret_cast<const ex_u32x4_any_t*>(row + min(c, limit - 8));
  } else {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < limit ? row[c + i] : 0u;
    return (ex_u32x4_t){v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
  }
}

// A piece that was loaded `over` columns early: those columns off, zeros
// behind (over <= 0: as it is).
__device__ __forceinline__ ex_u32x4_t end_piece(ex_u32x4_t v, int64_t over) {
  if (over <= 0) return v;
  if (over >= 8) return (ex_u32x4_t){0u, 0u, 0u, 0u};
  const int o = (int)over;
  if (o & 4) v = (ex_u32x4_t){v[2], v[3], 0u, 0u};
  if (o & 2) v = (ex_u32x4_t){v[1], v[2], v[3], 0u};
  if (o & 1)
    v = (ex_u32x4_t){v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return v;
}

// The 8 codes of w minus z, times f: codes - z + 128 as bytes (one addition
// per four, no borrow from byte to byte), the top bit of each turned to make
// them signed, then one conversion and one product per code. The product is
// finite wherever f (q - z) is.
__device__ __forceinline__ uint32_t xbias(uint32_t z) {
  return __builtin_amdgcn_perm(0u, 0x80u - z, 0u);    // its low byte four times
}
__device__ __forceinline__ ex_u32x4_t xexpand(uint32_t w, uint32_t bias, float f) {
  const uint32_t lo = ((w & 0x0F0F0F0Fu) + bias) ^ 0x80808080u, hi = (((w >> 4) & 0x0F0F0F0Fu) + bias) ^ 0x80808080u;
  ex_u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = ex_pack2((float)(int8_t)(lo >> (8 * i)) * f, (float)(int8_t)(hi >> (8 * i)) * f);
  return o;
}

// The words of 4 units of 8 codes (a chunk), unit u0 (a multiple of 4) of a
// packed row, and unit e of them minus z as floats.
template <int BITS>
struct UnitWords {
  uint32_t w[BITS];
  __device__ __forceinline__ void load(const uint32_t* __restrict__ row, int64_t u0) {
    load_chunk<BITS>(row + (u0 * (8 * BITS) >> 5), w);
  }
  __device__ __forceinline__ void get(int e, float z, float (&f)[8]) const {
    if constexpr (BITS == 4) {
      // byte i of lo / hi holds code 2 i / 2 i + 1: one conversion per code
      const uint32_t lo = w[e] & 0x0F0F0F0Fu, hi = (w[e] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = (float)((lo >> (8 * i)) & 0xFFu) - z;
        f[2 * i + 1] = (float)((hi >> (8 * i)) & 0xFFu) - z;
      }
    } else {
      const int base = 8 * BITS * e, wi = base >> 5;
      uint64_t v = w[wi];
      if (BITS == 3 && wi + 1 < BITS) v |= (uint64_t)w[wi + 1] << 32;
      v >>= base & 31;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = (float)(uint32_t)((v >> (BITS * i)) & ((1u << BITS) - 1u)) - z;
    }
  }
};

// Tile of workgroup b among nr row tiles x nc column tiles: the dispatcher
// deals consecutive workgroups to the 8 XCDs in turn, so each XCD takes a
// consecutive part of the list, in which 8 row tiles share a column tile
// before the next column: what an XCD has in flight then meets in its L2.
__device__ __forceinline__ bool tile_of(int64_t b, int nr, int nc, int& rt, int& ct) {
  const int64_t total = (int64_t)nr * nc, per = ceil_div(total, 8);
  const int64_t i = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || i >= total) return false;
  const int64_t band = i / (8 * (int64_t)nc);
  const int64_t in = i - band * 8 * nc;
  const int h = (int)min((int64_t)8, nr - band * 8);
  ct = (int)(in / h);
  rt = (int)(band * 8 + in % h);
  return true;
}

// The tile of workgroup b. The list holds the tiles that there are, not the
// launch's upper bound, so that the XCDs' parts are equal (with the bound the
// last XCDs' parts were empty: 61 against 51 us for 2036 rows over 32 experts).
__device__ __forceinline__ bool locate(const int32_t* __restrict__ offsets, int E, int R, int BM, int64_t b, int nc,
                                       int& ct, Seg& sg) {
  int rt;
  if (offsets == nullptr) {
    if (!tile_of(b, (int)ceil_div(R, BM), nc, rt, ct)) return false;
    sg = Seg{0, 0, R, rt * BM};
    return true;
  }
  if (E <= 64) {
    const SegScan s = scan_segments(offsets, E, R, BM, 0);
    return tile_of(b, __builtin_amdgcn_readlane(s.inc, 63), nc, rt, ct) && pick_segment(s, 0, 0, BM, rt, sg);
  }
  int total = 0;
  for (int e0 = 0; e0 < E; e0 += 64)
    total += __builtin_amdgcn_readlane(scan_segments(offsets, E, R, BM, e0).inc, 63);
  if (!tile_of(b, total, nc, rt, ct)) return false;
  sg = find_tile(offsets, E, R, BM, rt);
  return sg.e >= 0;
}

struct ExArgs {
  const uint16_t* A; int64_t lda;             // X or dY
  const int32_t* rows; int T;
  const int32_t* offsets; int E, R;
  const uint32_t* qw; const float* scales; const uint8_t* zeros;
  int64_t d_out, n; int group;
  void* Y; int ybf16; int64_t ldy;
  int nrt, nct;
  int per_split;                              // stages of one of the gridDim.y parts of K
  int64_t split_stride;                       // bytes from part to part of Y (fp32 then)
};

template <int B>
using ex_const = std::integral_constant<int, B>;

template <class F>
__device__ __forceinline__ void for_four(F&& f) {
  f(ex_const<0>{});
  f(ex_const<1>{});
  f(ex_const<2>{});
  f(ex_const<3>{});
}

// stage(index modulo U, index) for all stages, U per loop body.
template <int U, class F>
__device__ __forceinline__ void run_stages(int nst, F&& stage) {
  int st = 0;
  for (; st + U <= nst; st += U) {
    stage(ex_const<0>{}, st);
    stage(ex_const<1>{}, st + 1);
    if constexpr (U == 4) {
      stage(ex_const<2>{}, st + 2);
      stage(ex_const<3>{}, st + 3);
    }
  }
  if (st < nst) stage(ex_const<0>{}, st);
  if constexpr (U == 4) {
    if (st + 1 < nst) stage(ex_const<1>{}, st + 1);
    if (st + 2 < nst) stage(ex_const<2>{}, st + 2);
  }
}

// ---- forward: K = n. The codes minus the zero point are exact in bf16, the
// group's sum is scaled once in fp32 (tot += s acc), as in the one-layer
// product. G128: groups of 128, two stages each (the first product of a group
// starts from zero, no test inside a stage); otherwise groups of any number of
// 32-code chunks, tested after every chunk.
template <int BITS, class TL, bool G128>
__global__ void __launch_bounds__(TL::THREADS, 512 / TL::THREADS)
k_expert_mm(ExArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, PA = TL::PA, NB = TL::NB, THREADS = TL::THREADS;
  constexpr uint32_t ASZ = BM * 128, BSZ = TL::BN * 128, BUF = ASZ + BSZ;
  __shared__ __align__(16) uint8_t smem[2 * BUF];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, BM, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t o0 = (int64_t)ct * TL::BN;
  const int64_t ngroups = p.n / p.group;
  const int cpg = p.group / 32, nchunks = (int)(p.n / 32);
  const int s0 = blockIdx.y * p.per_split, nst = min((nchunks + 1) / 2 - s0, p.per_split);   // this part's stages
  const uint32_t lds = lds_addr(smem);

  // staging: piece tid % 8 of rows tid / 8 + (THREADS / 8) i of A; units
  // NB (tid % (8 / NB)) .. of row tid / (8 / NB) of B
  constexpr int AR = THREADS / 8, BU = 8 / NB;
  const int ac = tid & 7, ar = tid >> 3, bu = NB * (tid % BU), br = tid / BU;
  const uint16_t* arow[PA];
#pragma unroll
  for (int i = 0; i < PA; ++i)
    arow[i] = p.A + source_row(p.rows, min(sg.row0 + ar + AR * i, sg.hi - 1), p.T) * p.lda;
  const int64_t bo = (int64_t)sg.e * p.d_out + min(o0 + br, p.d_out - 1);
  const uint32_t* __restrict__ qrow = p.qw + bo * ((int64_t)nchunks * BITS);
  const uint8_t* __restrict__ zrow = p.zeros + bo * ngroups;
  const uint32_t aw = lds + row_piece(ar, ac);            // AR is a multiple of 16: rows apart keep the swizzle
  uint32_t bw[NB];
#pragma unroll
  for (int e = 0; e < NB; ++e) bw[e] = lds + ASZ + row_piece(br, bu + e);

  constexpr int DA = TL::DA, DB = TL::DB, U = TL::U;
  ex_u32x4_t ra[DA][PA];
  static_assert(NB == 4, "a chunk per load");
  UnitWords<BITS> rb[DB];
  uint32_t rz[DB];
  auto aload = [&](auto S, int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) ra[S % DA][i] = load_piece<true>(arow[i], (int64_t)(s0 + st) * kExBK + 8 * ac, p.n);
  };
  auto bload = [&](auto S, int st) {
    const int c = min(2 * (s0 + st) + bu / 4, nchunks - 1);      // a chunk past the end meets zeros of A
    rb[S % DB].load(qrow, 4 * c + bu % 4);
    const int g = G128 ? (s0 + st) >> 1 : c / cpg;
    rz[S % DB] = zrow[g];
  };
  auto awrite = [&](auto S, int st) {
    if ((int64_t)(s0 + st + 1) * kExBK > p.n) {
      const int64_t over = (int64_t)(s0 + st) * kExBK + 8 * ac - (p.n - 8);
#pragma unroll
      for (int i = 0; i < PA; ++i) ra[S % DA][i] = end_piece(ra[S % DA][i], over);
    }
#pragma unroll
    for (int i = 0; i < PA; ++i) lds_write(aw + (S % 2) * BUF + i * (AR * 128), ra[S % DA][i]);
  };
  // part kk of the four that a stage's products interleave with
  auto bwrite = [&](auto S, auto KK) {
    constexpr int kk = decltype(KK)::value, B = decltype(S)::value % DB;
#pragma unroll
    for (int e = 0; e < NB; ++e)
      if (e * 4 / NB == kk) {
        float f[8];
        rb[B].get(e, (float)rz[B], f);
        lds_write(bw[e] + (S % 2) * BUF, (ex_u32x4_t){pack_exact(f[0], f[1]), pack_exact(f[2], f[3]),
                                                       pack_exact(f[4], f[5]), pack_exact(f[6], f[7])});
      }
  };
  const float* srow[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni)
    srow[ni] = p.scales + ((int64_t)sg.e * p.d_out + min(o0 + 32 * (NI * wn + ni) + li, p.d_out - 1)) * ngroups;
  // fragment addresses of K slice kk (both operands have the lane's row at li)
  uint32_t af[4], bf[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    af[kk] = lds + row_piece(32 * MI * wm + li, 2 * kk + h);
    bf[kk] = lds + ASZ + row_piece(32 * NI * wn + li, 2 * kk + h);
  }

  ex_f32x16_t acc[MI][NI] = {}, tot[MI][NI] = {};
  const ex_f32x16_t zero = {};
  float sc[NI];
  int cin = 0;
  int64_t g = (int64_t)s0 * kExBK / p.group;               // a part starts with a group
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) sc[ni] = srow[ni][g];
  auto flush = [&]() {
    ++g;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r) tot[mi][ni][r] = fmaf(sc[ni], acc[mi][ni][r], tot[mi][ni][r]);
      sc[ni] = srow[ni][min(g, ngroups - 1)];
    }
  };
  auto stage = [&](auto S, int st) {
    constexpr int i = decltype(S)::value, b = i % 2;    // i: st modulo U
    const ex_const<i + 1> next{};
    __syncthreads();
    aload(ex_const<i + DA>{}, min(st + DA, nst - 1));
    bload(ex_const<i + DB>{}, min(st + DB, nst - 1));
    __builtin_amdgcn_sched_barrier(0);    // the loads leave before the stage's products
    ex_bf16x8_t fa[2][MI], fb[2][NI];
    auto frags = [&](auto KK) {
      constexpr int kk = decltype(KK)::value;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fa[kk & 1][mi] = lds_frag(af[kk] + b * BUF + mi * 4096);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) fb[kk & 1][ni] = lds_frag(bf[kk] + b * BUF + ni * 4096);
    };
    frags(ex_const<0>{});
    for_four([&](auto KK) {
      constexpr int kk = decltype(KK)::value;
      if constexpr (kk < 3) frags(ex_const<kk + 1>{});
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              fa[kk & 1][mi], fb[kk & 1][ni], G128 && b == 0 && kk == 0 ? zero : acc[mi][ni], 0, 0, 0);
      bwrite(next, KK);
      if (!G128 && (kk & 1) == 1 && ++cin == cpg && g < ngroups) {   // the group is complete
        flush();
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = zero;
        cin = 0;
      }
    });
    awrite(next, st + 1);
    if (G128 && b == 1) flush();
  };
  for_four([&](auto S) {
    if constexpr (S < DA) aload(S, min((int)S, nst - 1));
    if constexpr (S < DB) bload(S, min((int)S, nst - 1));
  });
  awrite(ex_const<0>{}, 0);
  for_four([&](auto KK) { bwrite(ex_const<0>{}, KK); });
  run_stages<U>(nst, stage);
  void* Y = static_cast<char*>(p.Y) + blockIdx.y * p.split_stride;
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t o = o0 + 32 * (NI * wn + ni) + li;
    if (o >= p.d_out) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = sg.row0 + 32 * (MI * wm + mi) + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < sg.hi) store_out(Y, p.ybf16, (int64_t)row * p.ldy + o, tot[mi][ni][r]);
      }
  }
}

// ---- gradient: K = d_out, columns n. The scale changes along K, so it
// cannot leave the sum; the weights s (q - z) are rounded to bf16 on their
// way into LDS (relative 2^-8 at most per weight, independent from weight to
// weight, which adds to the sum's error what the bf16 rounding of the result
// adds again). For results kept in fp32 the weight goes as NP = 3 bf16 pieces
// and three products: 24 bits, what its fp32 value holds.
template <int BITS, int NP, class TL, bool WIDE>
__global__ void __launch_bounds__(TL::THREADS, NP > 1 ? 1 : 512 / TL::THREADS)
k_expert_mm_grad(ExArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, BN = TL::BN, PA = TL::PA, NB = TL::NB, THREADS = TL::THREADS;
  constexpr uint32_t ASZ = BM * 128, BSZ = kExBK * 2 * BN, BUF = ASZ + NP * BSZ;
  __shared__ __align__(16) uint8_t smem[2 * BUF];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, BM, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t c0 = (int64_t)ct * TL::BN;
  const int64_t ngroups = p.n / p.group;
  const int nchunks = (int)(p.n / 32);
  const int s0 = blockIdx.y * p.per_split, nst = min((int)ceil_div(p.d_out, kExBK) - s0, p.per_split);
  const uint32_t lds = lds_addr(smem);

  // staging: A as in the forward product; units NB (tid % BU) .. of output
  // row tid / BU of B
  constexpr int AR = THREADS / 8, BU = BN / 8 / NB;
  const int ac = tid & 7, ar = tid >> 3, bu = NB * (tid % BU), br = tid / BU;
  const uint16_t* arow[PA];
#pragma unroll
  for (int i = 0; i < PA; ++i)
    arow[i] = p.A + source_row(p.rows, min(sg.row0 + ar + AR * i, sg.hi - 1), p.T) * p.lda;
  const int64_t unit = c0 / 8 + bu;
  const bool cok = unit < 4 * (int64_t)nchunks;
  const int64_t uc = cok ? unit : bu % 4;                  // columns past n: weights of 0
  const int64_t ebase = (int64_t)sg.e * p.d_out;
  const int64_t gi = uc * 8 / p.group;
  const uint32_t aw = lds + row_piece(ar, ac);
  uint32_t bw[NB];
#pragma unroll
  for (int e = 0; e < NB; ++e) bw[e] = lds + ASZ + col_piece<BN>(br, bu + e);

  constexpr int DA = TL::DA, DB = TL::DB, U = TL::U;
  ex_u32x4_t ra[DA][PA];
  static_assert(NB == 4, "a chunk per load");
  UnitWords<BITS> rb[DB];
  float rs[DB];
  uint32_t rz[DB];
  bool rv[DB];
  auto aload = [&](auto S, int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) ra[S % DA][i] = load_piece<WIDE>(arow[i], (int64_t)(s0 + st) * kExBK + 8 * ac, p.d_out);
  };
  auto bload = [&](auto S, int st) {
    constexpr int B = decltype(S)::value % DB;
    const int64_t o = (int64_t)(s0 + st) * kExBK + br;
    const int64_t oc = ebase + min(o, p.d_out - 1);
    rb[B].load(p.qw + oc * nchunks * BITS, uc);
    rs[B] = p.scales[oc * ngroups + gi];
    rz[B] = p.zeros[oc * ngroups + gi];
    rv[B] = cok && o < p.d_out;                              // outputs past d_out: weights of 0
  };
  auto awrite = [&](auto S, int st) {
    if (WIDE && (int64_t)(s0 + st + 1) * kExBK > p.d_out) {
      const int64_t over = (int64_t)(s0 + st) * kExBK + 8 * ac - (p.d_out - 8);
#pragma unroll
      for (int i = 0; i < PA; ++i) ra[S % DA][i] = end_piece(ra[S % DA][i], over);
    }
#pragma unroll
    for (int i = 0; i < PA; ++i) lds_write(aw + (S % 2) * BUF + i * (AR * 128), ra[S % DA][i]);
  };
  auto bwrite = [&](auto S, auto KK) {
    constexpr int kk = decltype(KK)::value, B = decltype(S)::value % DB;
    const float scale = rv[B] ? rs[B] : 0.f;
#pragma unroll
    for (int e = 0; e < NB; ++e)
      if (e * 4 / NB == kk) {
        if constexpr (BITS == 4 && NP == 1) {
          lds_write(bw[e] + (S % 2) * BUF, xexpand(rb[B].w[e], xbias(rz[B]), scale));
          continue;
        }
        float f[8];
        rb[B].get(e, (float)rz[B], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          ex_u32x4_t v;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = ex_pack2(f[2 * i], f[2 * i + 1]);
            if (q + 1 < NP) {                                          // what this piece leaves (exact)
              f[2 * i] -= __uint_as_float(v[i] << 16);
              f[2 * i + 1] -= __uint_as_float(v[i] & 0xFFFF0000u);
            }
          }
          lds_write(bw[e] + (S % 2) * BUF + q * BSZ, v);
        }
      }
  };
  uint32_t af[4], bf[NI];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) af[kk] = lds + row_piece(32 * MI * wm + li, 2 * kk + h);
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) bf[ni] = lds + ASZ + col_frag_at<BN>(32 * (NI * wn + ni), lane);

  ex_f32x16_t acc[MI][NI] = {};
  auto stage = [&](auto S, int st) {
    constexpr int i = decltype(S)::value, b = i % 2;    // i: st modulo U
    const ex_const<i + 1> next{};
    __syncthreads();
    aload(ex_const<i + DA>{}, min(st + DA, nst - 1));
    bload(ex_const<i + DB>{}, min(st + DB, nst - 1));
    __builtin_amdgcn_sched_barrier(0);
    ex_bf16x8_t fa[2][MI], fb[2][NP][NI];
    auto frags = [&](auto KK) {
      constexpr int kk = decltype(KK)::value;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fa[kk & 1][mi] = lds_frag(af[kk] + b * BUF + mi * 4096);
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          fb[kk & 1][q][ni] = lds_col_frag<BN>(bf[ni] + b * BUF + q * BSZ + kk * (32 * BN));
    };
    frags(ex_const<0>{});
    for_four([&](auto KK) {
      constexpr int kk = decltype(KK)::value;
      if constexpr (kk < 3) frags(ex_const<kk + 1>{});
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk & 1][mi], fb[kk & 1][q][ni], acc[mi][ni], 0, 0, 0);
      bwrite(next, KK);
    });
    awrite(next, st + 1);
  };
  for_four([&](auto S) {
    if constexpr (S < DA) aload(S, min((int)S, nst - 1));
    if constexpr (S < DB) bload(S, min((int)S, nst - 1));
  });
  awrite(ex_const<0>{}, 0);
  for_four([&](auto KK) { bwrite(ex_const<0>{}, KK); });
  run_stages<U>(nst, stage);
  void* Y = static_cast<char*>(p.Y) + blockIdx.y * p.split_stride;
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t c = c0 + 32 * (NI * wn + ni) + li;
    if (c >= p.n) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = sg.row0 + 32 * (MI * wm + mi) + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < sg.hi) store_out(Y, p.ybf16, (int64_t)row * p.ldy + c, acc[mi][ni][r]);
      }
  }
}

// ---- many rows per expert, 4 bits: the DMA ring
//
// 256 x 256 x 32 stages, 8 waves of 128 x 64 (128 accumulators per lane). The
// tiles above spend their time on the way of A through registers: without its
// loads the forward product took 27% less, although they hit the L1. Here
// everything comes by LDS-DMA and is counted by hand, so the compiler waits
// for none of it:
//  * A's slots are a ring of four, its DMA three stages ahead; packed codes,
//    zero points and scales land in buffers of their own, the codes of st + 2
//    before stage st;
//  * every wave issues a number of DMA instructions per stage that is known at
//    compile time, and the barrier that opens a stage leaves exactly the stage
//    before's in flight, so everything older has landed;
//  * during stage st the codes of st + 2 are expanded into B's ring, in between
//    the products, and the first K slice of st + 1 is read before its barrier,
//    so products never wait for LDS behind one.
// A group's scale leaves the forward sum without a second set of
// accumulators: the sum is kept in units of the current group's scale, and at
// a group's end all of it is multiplied by s_g / s_(g+1). That is one rounded
// multiplication per group and element, as the other tiles' one fused
// addition is. Groups whose scale is outside 2^-40 .. 2^40 (zero among them)
// use the unit 1 and have their weights s (q - z) rounded to bf16 instead. A
// sum below 2^88 is in fp32's range in any of these units, and fp32's smallest
// step in the largest unit is 2^-149 2^40.
// Measured: 8192 rows over 8 experts of 11008 x 4096 880 to 950 us (0.78 to 0.84
// PFLOP/s; 1030 in 128 x 128 tiles, a library product of expanded weights
// 530), gradient of 4096 x 4096 344 to 376 us (0.73 to 0.80 PFLOP/s; 391, 197).
// The products keep the matrix cores busy half of the time and the expansion
// the vector units the other half; the two waves of a SIMD meet at the
// barriers too often to fill each other's gaps. Waves whose half of the tile
// has no rows only expand (939 -> 925 us, gradient 370 -> 364).
// DMA of 16 bytes, a dword or a byte (widened to a dword) per lane from
// base + voff to lds + (16 or 4) lane.
__device__ __forceinline__ void xdma16(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory");
}
__device__ __forceinline__ void xdma4(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory");
}
__device__ __forceinline__ void xdma1(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "memory");
}
template <int VM>
__device__ __forceinline__ void xbarrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

typedef __attribute__((address_space(3))) const uint32_t lds_word_t;
typedef __attribute__((address_space(3))) const uint64_t lds_dword_t;
__device__ __forceinline__ uint32_t lds_u32(uint32_t at) { return *reinterpret_cast<lds_word_t*>(at); }
__device__ __forceinline__ uint64_t lds_u64(uint32_t at) { return *reinterpret_cast<lds_dword_t*>(at); }

// Piece c of row r of a [row][32] tile (64 bytes a row).
__device__ __forceinline__ uint32_t xrow_piece(int r, int c) { return (uint32_t)r * 64u + 16u * (c ^ ((r >> 2) & 3)); }

// 16 codes of one output row on their way from LDS to LDS. They are read half
// a stage before they are expanded, so that the expansion does not hold up the
// products it stands between.
struct XCodes {
  uint64_t w;
  uint32_t z, s;
};

// One MFMA, then VALU operations and LDS reads of its share, N times.
template <int N, int READS, int VALUS, int I = 0>
__device__ __forceinline__ void xinterleave() {
  if constexpr (I < N) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int r = (I + 1) * READS / N - I * READS / N;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    if constexpr (VALUS > 0) __builtin_amdgcn_sched_group_barrier(0x002, VALUS, 0);
    xinterleave<N, READS, VALUS, I + 1>();
  }
}

// Forward, groups that are multiples of 128. A block is four stages (128
// codes, 64 bytes of a row): its codes, zero points and scales come as whole
// blocks, two buffers of each, so that a row's 64 bytes are fetched at once (a
// stage's 16 bytes per row and fetch made 166 instead of 50 million requests to
// the L2). B's slots are a ring of three, addressed at run time.
constexpr uint32_t kFA = 0, kFB = 4 * 16384, kFRaw = kFB + 3 * 16384, kFScale = kFRaw + 2 * 16384,
                   kFZero = kFScale + 2 * 1024, kFLds = kFZero + 2 * 1024;
__global__ void __launch_bounds__(512, 2)
k_expert_ring(ExArgs p) {
  constexpr int MI = 4, NI = 2;
  __shared__ __align__(16) uint8_t smem[kFLds];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, 256, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, h = lane >> 5, li = lane & 31;
  const int64_t o0 = (int64_t)ct * 256;
  const int64_t ngroups = p.n / p.group;
  const int nblk = (int)(p.n / 128), bpg = p.group / 128;     // blocks, blocks per group
  const int nst = 4 * nblk;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // A: instruction 2 wave + i moves rows 16 (2 wave + i) + lane / 4 of a
  // stage; codes: the same rows of B, 64 bytes of a block
  uint32_t va[2], vq[2];
  const int64_t ebase = (int64_t)sg.e * p.d_out;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 16 * (2 * wave + i) + (lane >> 2);
    const uint32_t c = 16 * ((lane & 3) ^ ((r >> 2) & 3));
    va[i] = (uint32_t)(source_row(p.rows, min(sg.row0 + r, sg.hi - 1), p.T) * p.lda * 2 + c);
    vq[i] = (uint32_t)(min(o0 + r, p.d_out - 1) * (p.n / 2) + c);
  }
  // scales (waves 0..3) and zero points (4..7) of a block: one row per lane
  const int w4 = wave & 3;
  const uint32_t vs = (uint32_t)(min(o0 + 64 * w4 + lane, p.d_out - 1) * ngroups);
  const char* abase = reinterpret_cast<const char*>(p.A);
  const char* qbase = reinterpret_cast<const char*>(p.qw) + ebase * (p.n / 2);
  const char* sbase = reinterpret_cast<const char*>(p.scales + ebase * ngroups);
  const char* zbase = reinterpret_cast<const char*>(p.zeros + ebase * ngroups);
  auto issue_a = [&](int st, int slot) {
    const int c = min(st, nst - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      xdma16(va[i], abase + (int64_t)c * 64,
             __builtin_amdgcn_readfirstlane(lds + kFA + slot * 16384 + (2 * wave + i) * 1024));
  };
  auto issue_q = [&](int b, int i) {
    xdma16(vq[i], qbase + (int64_t)min(b, nblk - 1) * 64,
           __builtin_amdgcn_readfirstlane(lds + kFRaw + (b & 1) * 16384 + (2 * wave + i) * 1024));
  };
  auto issue_g = [&](int b) {
    const int g = min(b, nblk - 1) / bpg;
    if (wave < 4) xdma4(vs * 4u, sbase + (int64_t)g * 4, __builtin_amdgcn_readfirstlane(lds + kFScale + (b & 1) * 1024 + w4 * 256));
    else xdma1(vs, zbase + g, __builtin_amdgcn_readfirstlane(lds + kFZero + (b & 1) * 1024 + w4 * 256));
  };
  // expansion of a stage's codes: half tid % 2 (16 codes) of output row tid / 2
  const int xr = tid >> 1, xh = tid & 1;
  const uint32_t xq = lds + kFRaw + xr * 64 + xh * 8;
  const uint32_t xd0 = lds + kFB + xrow_piece(xr, 2 * xh), xd1 = lds + kFB + xrow_piece(xr, 2 * xh + 1);
  const uint32_t xz = lds + kFZero + 4 * xr, xs = lds + kFScale + 4 * xr;
  auto unit_ok = [](float s) { return fabsf(s) >= 0x1p-40f && fabsf(s) <= 0x1p40f; };
  XCodes xw;
  auto fetch = [&](int b, int i) {
    xw.w = lds_u64(xq + (b & 1) * 16384 + 16 * (i ^ ((xr >> 2) & 3)));
    xw.z = lds_u32(xz + (b & 1) * 1024);
    xw.s = lds_u32(xs + (b & 1) * 1024);
  };
  auto factor = [&]() { return unit_ok(__uint_as_float(xw.s)) ? 1.f : __uint_as_float(xw.s); };
  auto expand0 = [&](uint32_t slot) { lds_write(xd0 + slot, xexpand((uint32_t)xw.w, xbias(xw.z), factor())); };
  auto expand1 = [&](uint32_t slot) { lds_write(xd1 + slot, xexpand((uint32_t)(xw.w >> 32), xbias(xw.z), factor())); };
  uint32_t af[2], bf[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    af[k] = lds + kFA + xrow_piece(128 * wm + li, 2 * k + h);
    bf[k] = lds + kFB + xrow_piece(64 * wn + li, 2 * k + h);
  }
  ex_bf16x8_t fa[2][MI], fb[2][NI];
  auto read = [&](auto SL, auto KK, uint32_t bslot) {
    constexpr int sl = decltype(SL)::value, kk = decltype(KK)::value;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) fa[kk][mi] = lds_frag(af[kk] + sl * 16384 + mi * 2048);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) fb[kk][ni] = lds_frag(bf[kk] + bslot + ni * 2048);
  };
  ex_f32x16_t acc[MI][NI] = {};
  auto multiply = [&](auto KK) {
    constexpr int kk = decltype(KK)::value;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk][mi], fb[kk][ni], acc[mi][ni], 0, 0, 0);
  };

  for (int st = 0; st < 3; ++st) issue_a(st, st);
  for (int b = 0; b < 2; ++b) {
    issue_q(b, 0);
    issue_q(b, 1);
    issue_g(b);
  }
  xbarrier<0>();
  uint32_t b0 = 0, b1 = 16384, b2 = 2 * 16384;        // B's slots of stages st, st + 1, st + 2
  fetch(0, 0);
  expand0(b0);
  expand1(b0);
  fetch(0, 1);
  expand0(b1);
  expand1(b1);
  fetch(0, 2);
  const uint32_t su = lds + kFScale + 4 * (64 * wn + li);
  float unit[NI];                                      // the current unit of each of the lane's columns
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const float s = __uint_as_float(lds_u32(su + 128 * ni));
    unit[ni] = unit_ok(s) ? s : 1.f;
  }
  xbarrier<0>();
  read(ex_const<0>{}, ex_const<0>{}, b0);
  // DMA instructions of a wave in stage i of a block: A 2; codes of the next
  // block but one in stages 2 and 3, scales or zero points in stage 3 (their
  // buffers' last readers were stages 0 and, for the units, the end of the
  // block before)
  int left = bpg;                                      // blocks left of the group
  auto stage = [&](auto ON, auto I, int blk) {
    constexpr int i = decltype(I)::value;
    xbarrier<i == 0 ? 4 : (i == 3 ? 3 : 2)>();         // what stage i - 1 issued may still fly
    issue_a(4 * blk + i + 3, (i + 3) & 3);
    if constexpr (i == 2) issue_q(blk + 2, 0);
    if constexpr (i == 3) {
      issue_q(blk + 2, 1);
      issue_g(blk + 2);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ON) read(I, ex_const<1>{}, b0);
    expand0(b2);
    if constexpr (ON) {
      multiply(ex_const<0>{});
      xinterleave<8, 6, 4>();
      __builtin_amdgcn_sched_barrier(0);
      read(ex_const<(i + 1) & 3>{}, ex_const<0>{}, b1);
    }
    expand1(b2);
    fetch(i == 0 ? blk : blk + 1, (i + 3) & 3);
    if constexpr (ON) {
      multiply(ex_const<1>{});
      xinterleave<8, 9, 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
    const uint32_t t = b0;
    b0 = b1;
    b1 = b2;
    b2 = t;
  };
  if (__builtin_amdgcn_readfirstlane(sg.row0 + 128 * wm < sg.hi)) {
    for (int blk = 0; blk < nblk; ++blk) {
      for_four([&](auto I) { stage(std::true_type{}, I, blk); });
      if (--left == 0 && blk + 1 < nblk) {             // the group is complete: into the next one's unit
        left = bpg;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const float s = __uint_as_float(lds_u32(su + ((blk + 1) & 1) * 1024 + 128 * ni));
          const float next = unit_ok(s) ? s : 1.f;
          const float r = unit[ni] / next;
          unit[ni] = next;
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[mi][ni][q] *= r;
        }
      }
    }
  } else {
    // no row of these waves' half exists: they expand codes for the others
    for (int blk = 0; blk < nblk; ++blk) for_four([&](auto I) { stage(std::false_type{}, I, blk); });
  }
  // no DMA may land in LDS that this workgroup no longer owns
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t o = o0 + 64 * wn + 32 * ni + li;
    if (o >= p.d_out) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = sg.row0 + 128 * wm + 32 * mi + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < sg.hi) store_out(p.Y, p.ybf16, (int64_t)row * p.ldy + o, unit[ni] * acc[mi][ni][r]);
      }
  }
}

// Gradient: the rows of a stage's 32 outputs hold 128 contiguous bytes of
// codes each, so codes, scales and zero points (one of each per row and
// 32-column chunk, whatever the group) come stage by stage, five ahead.
constexpr int kGPer = 4;                               // DMA instructions per wave and stage
constexpr uint32_t kGSlot = 32768, kGRaw = 4 * kGSlot, kGScale = kGRaw + 4 * 4096, kGZero = kGScale + 4 * 1024,
                   kGDump = kGZero + 4 * 1024, kGLds = kGDump + 256;   // kGDump: never read
__global__ void __launch_bounds__(512, 2)
k_expert_ring_grad(ExArgs p) {
  constexpr int MI = 4, NI = 2;
  __shared__ __align__(16) uint8_t smem[kGLds];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, 256, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, h = lane >> 5, li = lane & 31;
  const int64_t c0 = (int64_t)ct * 256;
  const int64_t ngroups = p.n / p.group;
  const int nchunks = (int)(p.n / 32), cpg = p.group / 32;
  const int nst = (int)(p.d_out / 32);
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  uint32_t va[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 16 * (2 * wave + i) + (lane >> 2);
    const int64_t src = source_row(p.rows, min(sg.row0 + r, sg.hi - 1), p.T);
    va[i] = (uint32_t)(src * p.lda * 2 + 16 * ((lane & 3) ^ ((r >> 2) & 3)));
  }
  // output row 32 st + 8 w + lane / 8, chunk lane % 8 of the tile's 256
  // columns (chunks past n: the last one; their columns are not stored)
  const int w4 = wave & 3;
  const int row = 8 * w4 + (lane >> 3);
  const int chunk = min((int)(c0 / 32) + (lane & 7), nchunks - 1);
  const uint32_t vq = (uint32_t)(((int64_t)row * nchunks + chunk) * 16);
  const uint32_t vs = (uint32_t)((int64_t)row * ngroups + chunk / cpg);
  const int64_t ebase = (int64_t)sg.e * p.d_out;
  const char* qbase = reinterpret_cast<const char*>(p.qw + ebase * nchunks * 4);
  const char* sbase = reinterpret_cast<const char*>(p.scales + ebase * ngroups);
  const char* zbase = reinterpret_cast<const char*>(p.zeros + ebase * ngroups);
  const char* abase = reinterpret_cast<const char*>(p.A);
  const int64_t qstep = (int64_t)32 * nchunks * 16, gstep = 32 * ngroups;

  auto issue_a = [&](int st, int slot) {
    const int c = min(st, nst - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      xdma16(va[i], abase + (int64_t)c * 64, __builtin_amdgcn_readfirstlane(lds + slot * kGSlot + (2 * wave + i) * 1024));
  };
  // two instructions per wave: codes and scales, or zero points and a dummy
  auto issue_b = [&](int st) {
    const int64_t c = min(st, nst - 1);
    if (wave < 4) {
      xdma16(vq, qbase + c * qstep, __builtin_amdgcn_readfirstlane(lds + kGRaw + (st & 3) * 4096 + w4 * 1024));
      xdma4(vs * 4u, sbase + c * gstep * 4, __builtin_amdgcn_readfirstlane(lds + kGScale + (st & 3) * 1024 + w4 * 256));
    } else {
      xdma1(vs, zbase + c * gstep, __builtin_amdgcn_readfirstlane(lds + kGZero + (st & 3) * 1024 + w4 * 256));
      xdma4(0u, kZeroChunk, __builtin_amdgcn_readfirstlane(lds + kGDump));
    }
  };
  // expansion: columns 16 (tid % 16) .. of output row tid / 16
  const int xr = tid >> 4, xc = tid & 15;
  const uint32_t xq = lds + kGRaw + xr * 128 + xc * 8;
  const uint32_t xz = lds + kGZero + 4 * (xr * 8 + (xc >> 1)), xs = lds + kGScale + 4 * (xr * 8 + (xc >> 1));
  const uint32_t xd0 = lds + 16384 + col_piece<256>(xr, 2 * xc), xd1 = lds + 16384 + col_piece<256>(xr, 2 * xc + 1);
  XCodes xw;
  auto fetch = [&](int st) {
    xw.w = lds_u64(xq + (st & 3) * 4096);
    xw.z = lds_u32(xz + (st & 3) * 1024);
    xw.s = lds_u32(xs + (st & 3) * 1024);
  };
  auto expand0 = [&](int slot) {
    lds_write(xd0 + slot * kGSlot, xexpand((uint32_t)xw.w, xbias(xw.z), __uint_as_float(xw.s)));
  };
  auto expand1 = [&](int slot) {
    lds_write(xd1 + slot * kGSlot, xexpand((uint32_t)(xw.w >> 32), xbias(xw.z), __uint_as_float(xw.s)));
  };
  // fragment addresses (slots 2 and 3 are past the offset field of 0)
  uint32_t af[2][2], bf[2][2];                        // [slot / 2][kk], [slot / 2][ni]
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      af[q][k] = lds + q * 2 * kGSlot + xrow_piece(128 * wm + li, 2 * k + h);
      bf[q][k] = lds + q * 2 * kGSlot + 16384 + col_frag_at<256>(64 * wn + 32 * k, lane);
    }
  ex_bf16x8_t fa[2][MI], fb[2][NI];
  auto read = [&](auto SL, auto KK) {
    constexpr int sl = decltype(SL)::value, kk = decltype(KK)::value;
    constexpr uint32_t so = (sl & 1) * kGSlot;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) fa[kk][mi] = lds_frag(af[sl >> 1][kk] + so + mi * 2048);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) fb[kk][ni] = lds_col_frag<256>(bf[sl >> 1][ni] + so + kk * 8192);
  };
  ex_f32x16_t acc[MI][NI] = {};
  auto multiply = [&](auto KK) {
    constexpr int kk = decltype(KK)::value;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk][mi], fb[kk][ni], acc[mi][ni], 0, 0, 0);
  };

  for (int st = 0; st < 3; ++st) issue_a(st, st);
  for (int st = 0; st < 4; ++st) issue_b(st);
  xbarrier<0>();
  for (int st = 0; st < 2; ++st) {
    fetch(st);
    expand0(st);
    expand1(st);
  }
  fetch(2);
  xbarrier<0>();
  issue_b(4);                                          // into the codes of stage 0, read above
  read(ex_const<0>{}, ex_const<0>{});
  auto stage = [&](auto ON, auto SL, int st) {
    constexpr int sl = decltype(SL)::value;
    xbarrier<kGPer>();
    issue_a(st + 3, (sl + 3) & 3);
    issue_b(st + 5);                                   // over the codes of st + 1, read in stage st - 2
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ON) read(SL, ex_const<1>{});
    expand0((sl + 2) & 3);
    if constexpr (ON) {
      multiply(ex_const<0>{});
      xinterleave<8, 8, 4>();
      __builtin_amdgcn_sched_barrier(0);
      read(ex_const<(sl + 1) & 3>{}, ex_const<0>{});
    }
    expand1((sl + 2) & 3);
    fetch(st + 3);
    if constexpr (ON) {
      multiply(ex_const<1>{});
      xinterleave<8, 11, 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (__builtin_amdgcn_readfirstlane(sg.row0 + 128 * wm < sg.hi))
    run_stages<4>(nst, [&](auto SL, int st) { stage(std::true_type{}, SL, st); });
  else                                                 // no row of these waves' half exists
    run_stages<4>(nst, [&](auto SL, int st) { stage(std::false_type{}, SL, st); });
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // no DMA into LDS that is no longer owned
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t c = c0 + 64 * wn + 32 * ni + li;
    if (c >= p.n) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int orow = sg.row0 + 128 * wm + 32 * mi + 8 * (r >> 2) + 4 * h + (r & 3);
        if (orow < sg.hi) store_out(p.Y, p.ybf16, (int64_t)orow * p.ldy + c, acc[mi][ni][r]);
      }
  }
}

// Y[row][c] = the parts' sum, in order, for the rows of the segments.
__global__ void __launch_bounds__(256)
k_expert_sum(const float* __restrict__ part, int splits, int R, uint32_t cols, const int32_t* __restrict__ offsets, int E,
             void* __restrict__ Y, int ybf16, int64_t ldy) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, count = (int64_t)R * cols;
  if (i >= count) return;
  const int64_t row = i / cols;
  if (offsets && (row < offsets[0] || row >= offsets[E])) return;
  float v = part[i];
  for (int s = 1; s < splits; ++s) v += part[s * count + i];
  store_out(Y, ybf16, row * ldy + (i - row * cols), v);
}

// ---- weight gradient: K = a segment's rows. Both operands have K down their
// rows. The kept values have at most 7 significant bits, so they are exact in
// bf16, products are exact and the sums fp32. A segment's rows are split over
// `splits` workgroups (equal parts, whole stages, from the segment's own
// length) when there are few tiles; their partial sums are added in order by
// a second kernel.
struct KgArgs {
  const uint16_t* P; int64_t ldp; int64_t m;
  const int8_t* codes; const uint8_t* exps; int T; int64_t n, pitch;   // pitch: codes per row
  const int32_t* rows; const int32_t* offsets; int E, R;
  int nmt, nnt, splits;
  float* out; int64_t split_stride;   // out[split][e][m][n]
};

template <class TL, bool WIDE>
__global__ void __launch_bounds__(TL::THREADS, 512 / TL::THREADS)
k_keep_grad(KgArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, BN = TL::BN, PA = TL::PA, NB = TL::NB, THREADS = TL::THREADS;
  constexpr int AW = BM < 128 ? 128 : BM;                 // columns of P's tile in LDS
  constexpr uint32_t ASZ = kExBK * 2 * AW, BUF = ASZ + kExBK * 2 * BN;
  __shared__ __align__(16) uint8_t smem[2 * BUF];
  int rt, ct;
  if (!tile_of(blockIdx.x, p.nmt, p.nnt, rt, ct)) return;
  const int e = blockIdx.y, sp = blockIdx.z;
  int lo = 0, hi = p.R;
  if (p.offsets) {
    lo = min(max(p.offsets[e], 0), p.R);
    hi = min(max(p.offsets[e + 1], lo), p.R);
  }
  const int per = (int)(ceil_div(ceil_div(hi - lo, p.splits), kExBK) * kExBK);
  const int k0 = (int)min((int64_t)hi, lo + (int64_t)sp * per), k1 = (int)min((int64_t)hi, k0 + (int64_t)per);
  const int nst = (int)ceil_div(k1 - k0, kExBK);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM;
  const int64_t m0 = (int64_t)rt * BM, c0 = (int64_t)ct * TL::BN;
  const uint32_t lds = lds_addr(smem);

  // staging: A piece tid % AP of rows tid / AP + AR i; B units NB (tid % BU)
  // .. of row tid / BU
  constexpr int AP = BM / 8, AR = THREADS / AP, BU = BN / 8 / NB;
  const int ap = tid % AP, ar = tid / AP, bu = NB * (tid % BU), br = tid / BU;
  const int64_t bcol = c0 + 8 * bu;
  const bool bok = bcol < p.pitch;
  static_assert(AR % 4 == 0, "rows apart keep the swizzle");
  const uint32_t aw = lds + col_piece<AW>(ar, ap);
  uint32_t bw[NB];
#pragma unroll
  for (int u = 0; u < NB; ++u) bw[u] = lds + ASZ + col_piece<BN>(br, bu + u);
  constexpr int DA = TL::DA, DB = TL::DB, U = TL::U;
  ex_u32x4_t ra[DA][PA], rb[DB][NB / 2];
  uint32_t rx[DB];
  bool rv[DB];
  const int64_t bc = bok ? bcol : 0;
  // the source row of a stage is looked up U stages before its loads: loads
  // return in order, so waiting for a recent one would wait for all of them
  // (one stage ahead: 34 against 30 us for 16384 rows, 64 x 4096)
  auto lookup = [&](int st) { return (int)source_row(p.rows, min(k0 + min(st, nst) * kExBK + br, k1 - 1), p.T); };
  int src[U];
  // Columns past m are read along with a row where they are in bounds (their
  // results are not stored); at the end of P the piece is moved back.
  const int64_t pend = (int64_t)(p.R - 1) * p.ldp + p.m - 8;
  auto aload = [&](auto S, int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = k0 + st * kExBK + ar + AR * i;        // rows past the part: zeros on both sides
      if constexpr (WIDE) {
        const int64_t at = min((int64_t)r * p.ldp + m0 + 8 * ap, pend);
        const void* src = r < k1 ? static_cast<const void*>(p.P + at) : kZeroChunk;
        ra[S % DA][i] = *static_cast<const ex_u32x4_any_t*>(src);
      } else {
        ra[S % DA][i] = load_piece<false>(p.P + (int64_t)min(r, k1 - 1) * p.ldp, m0 + 8 * ap, r < k1 ? p.m : 0);
      }
    }
  };
  auto bload = [&](auto S, int st) {
    constexpr int B = decltype(S)::value % DB, Q = decltype(S)::value % U;
    const int64_t row = src[Q];
    src[Q] = lookup(st + U);
    const ex_u32x4_t* c = reinterpret_cast<const ex_u32x4_t*>(p.codes + row * p.pitch + bc);
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) rb[B][i] = c[i];
    rx[B] = p.exps[row * (p.pitch / 32) + bc / 32];
    rv[B] = k0 + st * kExBK + br < k1 && bok;
  };
  auto awrite = [&](auto S, int st) {
    if (WIDE && k0 + (st + 1) * kExBK >= p.R) {           // the stage may hold the last row
#pragma unroll
      for (int i = 0; i < PA; ++i) {
        const int r = k0 + st * kExBK + ar + AR * i;
        if (r < k1) ra[S % DA][i] = end_piece(ra[S % DA][i], (int64_t)r * p.ldp + m0 + 8 * ap - pend);
      }
    }
#pragma unroll
    for (int i = 0; i < PA; ++i) lds_write(aw + (S % 2) * BUF + i * (AR * 2 * AW), ra[S % DA][i]);
  };
  auto bwrite = [&](auto S, auto KK) {
    constexpr int kk = decltype(KK)::value, B = decltype(S)::value % DB;
    const float step = rv[B] ? __uint_as_float(rx[B] == 255u ? 0x7FC00000u : rx[B] << 23) : 0.f;
#pragma unroll
    for (int q = 0; q < NB; ++q)
      if (q * 4 / NB == kk) {
        ex_u32x4_t o;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // codes + 128 as unsigned bytes: one conversion per code
          const uint32_t u = rb[B][q >> 1][2 * (q & 1) + w] ^ 0x80808080u;
          float f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = ((float)((u >> (8 * i)) & 0xFFu) - 128.f) * step;
          o[2 * w] = pack_exact(f[0], f[1]);
          o[2 * w + 1] = pack_exact(f[2], f[3]);
        }
        lds_write(bw[q] + (S % 2) * BUF, o);
      }
  };
  uint32_t af[MI], bf[NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) af[mi] = lds + col_frag_at<AW>(32 * (MI * wm + mi), lane);
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) bf[ni] = lds + ASZ + col_frag_at<BN>(32 * (NI * wn + ni), lane);

  ex_f32x16_t acc[MI][NI] = {};
  auto stage = [&](auto S, int st) {
    constexpr int i = decltype(S)::value, b = i % 2;    // i: st modulo U
    const ex_const<i + 1> next{};
    __syncthreads();
    aload(ex_const<i + DA>{}, min(st + DA, nst - 1));
    bload(ex_const<i + DB>{}, min(st + DB, nst - 1));
    __builtin_amdgcn_sched_barrier(0);
    ex_bf16x8_t fa[2][MI], fb[2][NI];
    auto frags = [&](auto KK) {
      constexpr int kk = decltype(KK)::value;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fa[kk & 1][mi] = lds_col_frag<AW>(af[mi] + b * BUF + kk * (32 * AW));
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) fb[kk & 1][ni] = lds_col_frag<BN>(bf[ni] + b * BUF + kk * (32 * BN));
    };
    frags(ex_const<0>{});
    for_four([&](auto KK) {
      constexpr int kk = decltype(KK)::value;
      if constexpr (kk < 3) frags(ex_const<kk + 1>{});
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk & 1][mi], fb[kk & 1][ni], acc[mi][ni], 0, 0, 0);
      bwrite(next, KK);
    });
    awrite(next, st + 1);
  };
  if (nst > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i) src[i] = lookup(i);
    for_four([&](auto S) {
      if constexpr (S < DA) aload(S, min((int)S, nst - 1));
      if constexpr (S < DB) bload(S, min((int)S, nst - 1));
    });
    awrite(ex_const<0>{}, 0);
    for_four([&](auto KK) { bwrite(ex_const<0>{}, KK); });
  }
  run_stages<U>(nst, stage);
  const int h = lane >> 5, li = lane & 31;
  float* __restrict__ out = p.out + (int64_t)sp * p.split_stride + (int64_t)e * p.m * p.n;
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t c = c0 + 32 * (NI * wn + ni) + li;
    if (c >= p.n) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + 32 * (MI * wm + mi) + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < p.m) out[row * p.n + c] = acc[mi][ni][r];
      }
  }
}

// Wide gradients (m > 128): the ring of the expert products. 256 x 256 x 32
// stages, 8 waves of 128 x 64; P, the kept codes and their steps come by
// LDS-DMA (P three stages ahead, the others five), four instructions per wave
// and stage. A wave fetches the codes of the four rows it expands, so their
// source rows are the same for 16 lanes each and are read as scalars.
constexpr int kKPer = 4;
constexpr uint32_t kKB = 4 * 16384, kKRaw = kKB + 3 * 16384, kKExp = kKRaw + 4 * 8192, kKLds = kKExp + 4 * 2048;
__global__ void __launch_bounds__(512, 2)
k_keep_ring(KgArgs p) {
  constexpr int MI = 4, NI = 2;
  __shared__ __align__(16) uint8_t smem[kKLds];
  int rt, ct;
  if (!tile_of(blockIdx.x, p.nmt, p.nnt, rt, ct)) return;
  const int e = blockIdx.y, sp = blockIdx.z;
  int lo = 0, hi = p.R;
  if (p.offsets) {
    lo = min(max(p.offsets[e], 0), p.R);
    hi = min(max(p.offsets[e + 1], lo), p.R);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int per = (int)(ceil_div(ceil_div(hi - lo, p.splits), kExBK) * kExBK);
  const int k0 = (int)min((int64_t)hi, lo + (int64_t)sp * per), k1 = (int)min((int64_t)hi, k0 + (int64_t)per);
  const int nst = (k1 - k0 + 31) / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, h = lane >> 5, li = lane & 31;
  const int64_t m0 = (int64_t)rt * 256, c0 = (int64_t)ct * 256;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // P: instruction 2 wave + i moves rows 2 (2 wave + i) + lane / 32 of a stage
  int ta[2];
  const uint16_t* pa[2];
  bool pok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ta[i] = 2 * (2 * wave + i) + (lane >> 5);
    const int pos = lane & 31, c = pos ^ dma_swz(ta[i]) ^ (pos >> 4);
    pok[i] = m0 + 8 * c < p.m;
    pa[i] = p.P + (int64_t)(k0 + ta[i]) * p.ldp + m0 + 8 * c;
  }
  auto issue_a = [&](int st, int slot) {
    const int c = min(st, nst - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // rows past the part and columns past m: zeros
      const bool ok = pok[i] && k0 + 32 * c + ta[i] < k1;
      const void* src = ok ? static_cast<const void*>(pa[i] + (int64_t)c * 32 * p.ldp) : kZeroChunk;
      dma16(src, __builtin_amdgcn_readfirstlane(lds + slot * 16384 + (2 * wave + i) * 1024));
    }
  };
  // codes: 16 columns lane % 16 of row 4 wave + lane / 16; their steps
  typedef __attribute__((address_space(4))) const int32_t const_i32;
  const const_i32* rows = (const const_i32*)(uintptr_t)p.rows;
  const uint32_t vcol = (uint32_t)min(c0 + 16 * (lane & 15), p.pitch - 16);
  const uint32_t vgrp = (uint32_t)min(c0 / 32 + (lane & 7), p.pitch / 32 - 1);
  auto issue_b = [&](int st) {
    const int r = k0 + 32 * min(st, nst - 1) + 4 * wave;
    int src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = min(r + i, k1 - 1);
      src[i] = min(max(p.rows ? rows[q] : q, 0), p.T - 1);
    }
    const int a = lane & 16 ? src[1] : src[0], b = lane & 16 ? src[3] : src[2];
    const uint32_t row = (uint32_t)(lane & 32 ? b : a);
    xdma16(row * (uint32_t)p.pitch + vcol, p.codes, __builtin_amdgcn_readfirstlane(lds + kKRaw + (st & 3) * 8192 + wave * 1024));
    xdma1(row * (uint32_t)(p.pitch / 32) + vgrp, p.exps,
          __builtin_amdgcn_readfirstlane(lds + kKExp + (st & 3) * 2048 + wave * 256));
  };
  // expansion: columns 16 (tid % 16) .. of the stage's row tid / 16
  const int xr = tid >> 4, xc = tid & 15;
  const uint32_t xq = lds + kKRaw + tid * 16;
  const uint32_t xe = lds + kKExp + wave * 256 + 4 * (16 * (xr & 3) + (xc >> 1));
  const uint32_t xd0 = lds + kKB + col_piece<256>(xr, 2 * xc), xd1 = lds + kKB + col_piece<256>(xr, 2 * xc + 1);
  typedef __attribute__((address_space(3))) const ex_u32x4_t lds_quad_t;
  ex_u32x4_t xw;
  uint32_t xx = 0;
  auto fetch = [&](int st) {
    xw = *reinterpret_cast<lds_quad_t*>(xq + (st & 3) * 8192);
    xx = lds_u32(xe + (st & 3) * 2048);
  };
  auto step_of = [&](int st) {
    return k0 + 32 * st + xr < k1 ? __uint_as_float(xx == 255u ? 0x7FC00000u : xx << 23) : 0.f;
  };
  auto convert = [&](uint32_t w0, uint32_t w1, float step) {
    ex_u32x4_t o;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t u = (w ? w1 : w0) ^ 0x80808080u;
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = ((float)((u >> (8 * i)) & 0xFFu) - 128.f) * step;
      o[2 * w] = pack_exact(f[0], f[1]);
      o[2 * w + 1] = pack_exact(f[2], f[3]);
    }
    return o;
  };
  uint32_t af[MI], bf[NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) af[mi] = lds + col_frag_at<256>(128 * wm + 32 * mi, lane);
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) bf[ni] = lds + kKB + col_frag_at<256>(64 * wn + 32 * ni, lane);
  ex_bf16x8_t fa[2][MI], fb[2][NI];
  auto read = [&](uint32_t aslot, uint32_t bslot, auto KK) {
    constexpr int kk = decltype(KK)::value;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) fa[kk][mi] = lds_col_frag<256>(af[mi] + aslot + kk * 8192);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) fb[kk][ni] = lds_col_frag<256>(bf[ni] + bslot + kk * 8192);
  };
  ex_f32x16_t acc[MI][NI] = {};
  auto multiply = [&](auto KK) {
    constexpr int kk = decltype(KK)::value;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk][mi], fb[kk][ni], acc[mi][ni], 0, 0, 0);
  };
  if (nst > 0) {
    for (int st = 0; st < 3; ++st) issue_a(st, st);
    for (int st = 0; st < 4; ++st) issue_b(st);
    xbarrier<0>();
    uint32_t b0 = 0, b1 = 16384, b2 = 2 * 16384;       // B's slots of stages st, st + 1, st + 2
    for (int st = 0; st < 2; ++st) {
      fetch(st);
      const float f = step_of(st);
      lds_write(xd0 + st * 16384, convert(xw[0], xw[1], f));
      lds_write(xd1 + st * 16384, convert(xw[2], xw[3], f));
    }
    fetch(2);
    xbarrier<0>();
    issue_b(4);                                         // over the codes of stage 0, read above
    read(0, b0, ex_const<0>{});
    auto stage = [&](auto SL, int st) {
      constexpr int sl = decltype(SL)::value;
      xbarrier<kKPer>();
      issue_a(st + 3, (sl + 3) & 3);
      issue_b(st + 5);                                  // over the codes of st + 1, read in stage st - 2
      __builtin_amdgcn_sched_barrier(0);
      const float f = step_of(st + 2);
      read(sl * 16384, b0, ex_const<1>{});
      lds_write(xd0 + b2, convert(xw[0], xw[1], f));
      multiply(ex_const<0>{});
      xinterleave<8, 12, 5>();
      __builtin_amdgcn_sched_barrier(0);
      read(((sl + 1) & 3) * 16384, b1, ex_const<0>{});
      lds_write(xd1 + b2, convert(xw[2], xw[3], f));
      fetch(st + 3);
      multiply(ex_const<1>{});
      xinterleave<8, 14, 5>();
      __builtin_amdgcn_sched_barrier(0);
      const uint32_t t = b0;
      b0 = b1;
      b1 = b2;
      b2 = t;
    };
    run_stages<4>(nst, stage);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no DMA into LDS that is no longer owned
  }
  float* __restrict__ out = p.out + (int64_t)sp * p.split_stride + (int64_t)e * p.m * p.n;
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t c = c0 + 64 * wn + 32 * ni + li;
    if (c >= p.n) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + 128 * wm + 32 * mi + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < p.m) out[row * p.n + c] = acc[mi][ni][r];
      }
  }
}

__global__ void __launch_bounds__(256)
k_keep_grad_sum(const float* __restrict__ part, int splits, int64_t count, float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float v = part[i];
  for (int s = 1; s < splits; ++s) v += part[(int64_t)s * count + i];
  out[i] = v;
}

// ---------------------------------------------------------------- host
static int64_t row_tiles(int64_t R, int E, int BM) { return std::min<int64_t>(R, ceil_div(R, BM) + E - 1); }

static bool bf16_rows_vec(const void* p, int64_t ld, int64_t cols) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && cols % 8 == 0;
}

// The ring kernels: 4 bits, whole blocks (forward) or stages and a bf16 result
// (gradient), offsets from the bases that fit 32 bits, tiles for half of the
// chip at least (fewer are better split along K), and more columns than the
// smaller tile has (65536 rows, 128 outputs of 4096: 157 us here, 105 us in
// 128 x 128 tiles; gradient 173 and 134 us). One expert, K 4096, ring and
// smaller tiles: 64 tiles (2048 x 2048) 122 and 69 us, gradient 107 and 66; 128
// tiles (1024 x 8192) 121 and 95, 106 and 96; 172 tiles (1024 x 11008) 122 and
// 136, 112 and 137; 256 tiles (2048 x 8192) 144 and 183, 131 and 180. Between
// 128 and about 160 tiles the smaller ones are still ahead.
static bool ring_fits(const ExpertArgs& a, int grad) {
  const int64_t lim = (int64_t)1 << 32;
  if (a.bits != 4 || a.d_out * (a.n / 2) >= lim || a.lda >= lim / 2 / std::max(a.T, 1)) return false;
  if (!(grad ? a.y_bf16 && a.d_out % 32 == 0 : a.group % 128 == 0)) return false;
  const int64_t cols = grad ? a.n : a.d_out;
  return cols > 128 && ceil_div(a.R, 256) * ceil_div(cols, 256) >= 128;
}

// 64 or 128 rows of a tile: the small ones while all of them run at once, two
// (gradient: nearly three) workgroups per CU, or while most segments fit one;
// beyond, the large ones expand each weight for twice the rows. 64 against 128
// rows, 4 bits, groups of 64: 96 rows for each of 8 experts of 4096 x 4096 (512 tiles) 89 and
// 111 us, gradient 74 and 88; 96 for each of 32 of 1408 x 2048 (704 tiles) 82
// and 72, gradient 55 and 53; 29 for each of 64 of 1272 x 5120 154 and 184.
// Three pieces (fp32 gradient) fill a CU's LDS with one workgroup, small or
// large: 100 rows for each of 4 experts of 2048 x 2048 40 and 49 us, 450 rows
// 99 and 69.
static int small_bm(int64_t R, int E, int64_t cols, int grad, bool pieces) {
  if (pieces) return ceil_div(R, E) <= 128 ? 64 : 128;
  const int64_t tiles = std::min<int64_t>(R, ceil_div(R, 64) + (E - 1) / 2) * ceil_div(cols, 128);
  return ceil_div(R, E) <= 48 || tiles <= (grad ? 640 : 512) ? 64 : 128;
}

// Rows of a tile: 16 is the matrix-vector form, 256 the ring kernel.
//  * Matrix-vector form and 64-row tiles, 4 bits: 8 experts of 4096 x 4096 with
//    4, 16, 20 and 32 rows each 26, 45, 54, 71 and 42, 46, 44, 49 us; 64 of
//    1408 x 2048 with 4, 16, 20 and 24 rows 29, 57, 65, 74 and 53, 58, 59, 63;
//    groups of 64 with 16 rows 58 and 57, 77 and 74. (3 bits stay ahead longer:
//    24 rows 58 and 74, 74 and 108.)
//  * Ring and 128-row tiles: 8 experts of 4096 x 4096 with 512, 640 and 1024
//    rows each 247, 251, 381 and 219, 258, 392 us, gradient 222, 228, 348 and
//    219, 257, 391; 8 of 11008 x 4096 506, 562, 901 and 568, 661, 1030. Fewer
//    rows go either way with how full the last tiles are (256 rows: 125 and 136,
//    but 372 and 343).
static int expert_bm(const ExpertArgs& a, int grad) {
  const int64_t avg = ceil_div(a.R, a.E);
  const bool vec = bf16_rows_vec(a.A, a.lda, grad ? a.d_out : a.n);
  if (!grad && avg <= 16 && vec) return 16;
  if (grad && a.d_out < 8) return 64;
  if (vec && avg > 512 && ring_fits(a, grad)) return 256;
  return small_bm(a.R, a.E, grad ? a.n : a.d_out, grad, grad && !a.y_bf16);
}

// Parts of K. Few tiles leave most of the chip idle and make every workgroup
// walk all of K: then K is split until there are two workgroups per CU (one
// with three pieces; 150 rows of 4096 outputs, K 2048, in 320 workgroups 43 us,
// in 256 31 us), at least four stages each (24 rows of 5612 outputs, gradient of 512 columns:
// 185 us in one part, 38 us in parts). The parts meet in fp32 in the workspace.
// From the sizes alone, so that the workspace's size is known before the call.
ExpertSplit expert_split(int64_t R, int E, int64_t n, int64_t d_out, int group, int grad, bool pieces) {
  ExpertSplit sp = {1, 0, 0};
  const int64_t K = grad ? d_out : n, cols = grad ? n : d_out;
  const int64_t nst = ceil_div(K, kExBK);
  sp.per = (int)nst;
  const int64_t avg = ceil_div(R, E);
  if (R <= 0 || (!grad && avg <= 16)) return sp;           // the matrix-vector form splits inside
  const int bm = small_bm(R, E, cols, grad, pieces);
  const int64_t tiles = std::min<int64_t>(R, ceil_div(R, bm) + (E - 1) / 2) * ceil_div(cols, 128);
  int64_t unit = 1;                                        // stages between starts of a group
  if (!grad)
    while (unit * kExBK % group != 0) ++unit;
  int64_t s = std::min<int64_t>((pieces ? 256 : 512) / std::max<int64_t>(tiles, 1), nst / 4);
  if (s <= 1) return sp;
  const int64_t per = ceil_div(ceil_div(nst, s), unit) * unit;
  sp.per = (int)per;
  sp.splits = (int)ceil_div(nst, per);
  sp.part_bytes = sp.splits > 1 ? (size_t)sp.splits * R * cols * sizeof(float) : 0;
  return sp;
}

int64_t expert_threads(const ExpertArgs& a, int grad) {
  const int bm = expert_bm(a, grad);
  const int64_t cols = grad ? a.n : a.d_out;
  if (bm == 16) return ceil_div(cols, 32) * 256;           // the row tiles are the second dimension
  return bm == 256 ? (row_tiles(a.R, a.E, 256) * ceil_div(cols, 256) + 8) * 512
                   : (row_tiles(a.R, a.E, bm) * ceil_div(cols, 128) + 8) * 256;
}

template <int BITS>
static void mv_go(hipStream_t s, const ExpertArgs& a) {
  constexpr int WAVES = 4, OB = 2, S = 2;
  const dim3 grid((unsigned)ceil_div(a.d_out, 16 * OB), (unsigned)row_tiles(a.R, a.E, 16));
  const uint16_t* X = static_cast<const uint16_t*>(a.A);
  if (a.group % 128 == 0)
    hipLaunchKernelGGL((k_expert_mv<BITS, true, WAVES, OB, S>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
  else
    hipLaunchKernelGGL((k_expert_mv<BITS, false, WAVES, OB, S>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
}

static dim3 tile_grid(int nr, int nc) { return dim3((unsigned)(8 * ceil_div((int64_t)nr * nc, 8))); }

static ExArgs ex_args(const ExpertArgs& a, int BM, int BN, int64_t cols) {
  ExArgs p;
  p.A = static_cast<const uint16_t*>(a.A);
  p.lda = a.lda;
  p.rows = a.rows;
  p.T = a.T;
  p.offsets = a.offsets;
  p.E = a.E;
  p.R = a.R;
  p.qw = a.qw;
  p.scales = a.scales;
  p.zeros = a.zeros;
  p.d_out = a.d_out;
  p.n = a.n;
  p.group = a.group;
  p.Y = a.Y;
  p.ybf16 = a.y_bf16;
  p.ldy = a.ldy;
  p.nrt = (int)row_tiles(a.R, a.E, BM);
  p.nct = (int)ceil_div(cols, BN);
  p.per_split = 0;
  p.split_stride = 0;
  return p;
}

// The tile kernels write their parts of K into the workspace when there are several.
template <class F>
static void split_go(hipStream_t s, const ExpertArgs& a, ExArgs p, int64_t cols, int grad, F&& launch) {
  const ExpertSplit sp = expert_split(a.R, a.E, a.n, a.d_out, a.group, grad, grad && !a.y_bf16);
  p.per_split = sp.per;
  dim3 grid = tile_grid(p.nrt, p.nct);
  grid.y = (unsigned)sp.splits;
  if (sp.splits > 1) {
    p.Y = a.part;
    p.ybf16 = 0;
    p.ldy = cols;
    p.split_stride = (int64_t)a.R * cols * (int64_t)sizeof(float);
  }
  launch(grid, p);
  if (sp.splits > 1)
    hipLaunchKernelGGL(k_expert_sum, dim3((unsigned)ceil_div((int64_t)a.R * cols, 256)), dim3(256), 0, s,
                       static_cast<const float*>(a.part), sp.splits, a.R, (uint32_t)cols, a.offsets, a.E, a.Y, a.y_bf16,
                       a.ldy);
}

template <int BITS, class TL, bool G128>
static void mm_go(hipStream_t s, const ExpertArgs& a) {
  split_go(s, a, ex_args(a, TL::BM, TL::BN, a.d_out), a.d_out, 0, [&](dim3 grid, const ExArgs& p) {
    hipLaunchKernelGGL((k_expert_mm<BITS, TL, G128>), grid, dim3(TL::THREADS), 0, s, p);
  });
}

// Groups of 128 are worth their own code at 4 bits, the common layer: 8 experts
// of 4096 x 4096 with 32, 96, 200 and 400 rows each 51, 71, 121 and 183 us, in
// the code for any group 56, 77, 135 and 196.
template <int BITS, class TL>
static void mm_group(hipStream_t s, const ExpertArgs& a) {
  if constexpr (BITS == 4) {
    if (a.group == 128) return mm_go<4, TL, true>(s, a);
  }
  mm_go<BITS, TL, false>(s, a);
}

template <int BITS, int NP, class TL, bool WIDE>
static void grad_go(hipStream_t s, const ExpertArgs& a) {
  split_go(s, a, ex_args(a, TL::BM, TL::BN, a.n), a.n, 1, [&](dim3 grid, const ExArgs& p) {
    hipLaunchKernelGGL((k_expert_mm_grad<BITS, NP, TL, WIDE>), grid, dim3(TL::THREADS), 0, s, p);
  });
}

static void ring_go(hipStream_t s, const ExpertArgs& a, int grad) {
  const ExArgs p = ex_args(a, 256, 256, grad ? a.n : a.d_out);
  hipLaunchKernelGGL(grad ? k_expert_ring_grad : k_expert_ring, tile_grid(p.nrt, p.nct), dim3(512), 0, s, p);
}

template <int BITS>
static void fwd_bits(hipStream_t s, const ExpertArgs& a) {
  const int bm = expert_bm(a, 0);
  if (bm == 16) mv_go<BITS>(s, a);
  else if (bm == 256) ring_go(s, a, 0);
  else if (bm == 64) mm_group<BITS, ExTile64>(s, a);
  else mm_group<BITS, ExTile128>(s, a);
}

template <int BITS>
static void grad_bits(hipStream_t s, const ExpertArgs& a) {
  const int bm = expert_bm(a, 1);
  if (a.d_out < 8) {
    if (a.y_bf16) grad_go<BITS, 1, ExTile64, false>(s, a);
    else grad_go<BITS, 3, ExTile64, false>(s, a);
  } else if (a.y_bf16) {
    if (bm == 64) grad_go<BITS, 1, ExTile64, true>(s, a);
    else if (bm == 128) grad_go<BITS, 1, ExTile128, true>(s, a);
    else ring_go(s, a, 1);
  } else {
    if (bm == 64) grad_go<BITS, 3, ExTile64, true>(s, a);
    else grad_go<BITS, 3, ExTile128, true>(s, a);
  }
}

hipError_t launch_expert_mm(hipStream_t s, const ExpertArgs& a) {
  if (a.R <= 0 || a.d_out <= 0 || a.n <= 0 || a.E <= 0) return hipSuccess;
  if (a.bits == 2) fwd_bits<2>(s, a);
  else if (a.bits == 3) fwd_bits<3>(s, a);
  else fwd_bits<4>(s, a);
  return hipGetLastError();
}

hipError_t launch_expert_mm_grad(hipStream_t s, const ExpertArgs& a) {
  if (a.R <= 0 || a.d_out <= 0 || a.n <= 0 || a.E <= 0) return hipSuccess;
  if (a.bits == 2) grad_bits<2>(s, a);
  else if (a.bits == 3) grad_bits<3>(s, a);
  else grad_bits<4>(s, a);
  return hipGetLastError();
}

// Tiles of 32 and 64 rows where m is no more: 16 x 4096 from 16384 rows 29 us, in
// 64-row tiles 32, in 128-row ones 36; 64 x 4096 36 and 40. The ring for m > 128
// and 128-row tiles: 2048 x 4096, 8 experts of 1024 rows 213 and 249 us; from 16384
// rows 136 x 4096 60 and 65, 256 x 4096 66 and 66; but 8 experts of 256 x 4096 63
// and 45, which the ring's fewer tiles leave half of the chip without.
KeepGradPlan keep_grad_plan(int64_t R, int E, int64_t m, int64_t n) {
  KeepGradPlan p{};
  p.bm = m <= 32 ? 32 : (m <= 64 ? 64 : (m <= 128 ? 128 : 256));
  const int64_t tiles = ceil_div(m, p.bm) * ceil_div(n, p.bm == 256 ? 256 : 128) * E;
  const int64_t seg = ceil_div(R, E);                 // rows of an average segment
  // two workgroups per CU, of the ring's one (16384 rows, 256 x 4096: 92 us with
  // two, 70 with one; 64 x 4096 with one instead of two: 43 against 38)
  int64_t s = tiles > 0 ? (p.bm == 256 ? 256 : 512) / tiles : 1;
  s = std::min<int64_t>(s, seg / 256);                // at least four stages each
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, 64));
  p.part_bytes = p.splits > 1 ? (size_t)p.splits * E * m * n * sizeof(float) : 0;
  return p;
}

// Of the smallest tiles that m may get (256 threads each); the 256 x 256 ones,
// of 512, have no more for the same G. G's parts are at most 2^24 values
// (fewer tiles than workgroups fit the chip), so their sum is never larger.
int64_t keep_grad_threads(int64_t m, int64_t n) {
  const int bm = m <= 32 ? 32 : (m <= 64 ? 64 : 128);
  return (ceil_div(m, bm) * ceil_div(n, 128) + 8) * 256;
}

template <class TL>
static void kg_go(hipStream_t s, const KgArgs& p) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)p.nmt * p.nnt, 8)), (unsigned)p.E, (unsigned)p.splits);
  if (p.m >= 8) hipLaunchKernelGGL((k_keep_grad<TL, true>), grid, dim3(TL::THREADS), 0, s, p);
  else hipLaunchKernelGGL((k_keep_grad<TL, false>), grid, dim3(TL::THREADS), 0, s, p);
}

hipError_t launch_keep_grad(hipStream_t s, const KeepGradPlan& pl, const uint16_t* P, int64_t ldp, int64_t R, int64_t m,
                            const int8_t* codes, const uint8_t* exps, int64_t T, int64_t n, const int32_t* rows,
                            const int32_t* offsets, int E, float* G, float* part) {
  if (m <= 0 || n <= 0 || E <= 0) return hipSuccess;
  KgArgs p;
  p.P = P;
  p.ldp = ldp;
  p.m = m;
  p.codes = codes;
  p.exps = exps;
  p.T = (int)T;
  p.n = n;
  p.pitch = 32 * ceil_div(n, 32);
  p.rows = rows;
  p.offsets = offsets;
  p.E = E;
  p.R = (int)R;
  p.splits = pl.splits;
  p.out = pl.splits > 1 ? part : G;
  p.split_stride = (int64_t)E * m * n;
  const bool vec = bf16_rows_vec(P, ldp, m);
  // the ring's offsets into the codes are 32 bits
  const int bm = pl.bm == 256 && !(vec && T * p.pitch < ((int64_t)1 << 32)) ? 128 : pl.bm;
  p.nmt = (int)ceil_div(m, bm);
  p.nnt = (int)ceil_div(n, bm == 256 ? 256 : 128);
  if (bm == 32) kg_go<ExTile32>(s, p);
  else if (bm == 64) kg_go<ExTile64>(s, p);
  else if (bm == 128) kg_go<ExTile128>(s, p);
  else
    hipLaunchKernelGGL(k_keep_ring, dim3((unsigned)(8 * ceil_div((int64_t)p.nmt * p.nnt, 8)), (unsigned)E,
                                         (unsigned)pl.splits), dim3(512), 0, s, p);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || pl.splits <= 1) return err;
  const int64_t count = (int64_t)E * m * n;
  hipLaunchKernelGGL(k_keep_grad_sum, dim3((unsigned)ceil_div(count, 256)), dim3(256), 0, s, part, pl.splits, count, G);
  return hipGetLastError();
}

}  // namespace gq

// Building blocks of the products with packed weights: segments of rows, packed
// codes, and the matrix-vector product of one wave.
#pragma once
#include "common.h"

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

// The packed rows of a lane's outputs, one per block of 16.
template <int OB>
struct MvRows {
  const uint32_t* q[OB];
  const float* s[OB];
  const uint8_t* z[OB];
  __device__ __forceinline__ MvRows(const uint32_t* qw, const float* scales, const uint8_t* zeros,
                                    const int64_t (&row)[OB], int64_t n, int group, int bits) {
#pragma unroll
    for (int b = 0; b < OB; ++b) {
      q[b] = qw + row[b] * (n / 32 * bits);
      s[b] = scales + row[b] * (n / group);
      z[b] = zeros + row[b] * (n / group);
    }
  }
};

// tot[b] += the share of part `part` of `parts` of K in the product of up to
// 16 rows of X (lane l: row l % 16; xrow() gives its address, called after the
// first weights have been asked for) and 16 OB packed rows. X in NP pieces,
// xplane elements apart, whose sum it is. WIDE: groups are multiples of 128.
template <int BITS, bool WIDE, int OB, int S, int NP, class XR>
__device__ __forceinline__ void mv_sum(const MvRows<OB>& rows, int64_t n, int group, int part, int parts, bool xok,
                                       int64_t xplane, XR&& xrow_of, ex_f32x4_t (&tot)[OB]) {
  const int lane = threadIdx.x & 63, j = lane >> 4, li = lane & 15;
  const int nchunks = (int)(n / 32), npieces = (nchunks + 3) / 4;
  const ex_u32x4_t ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const ex_bf16x8_t ones = __builtin_bit_cast(ex_bf16x8_t, ones_bits);
  const int per = (npieces + parts - 1) / parts;
  const int pbeg = part * per, pend = min(npieces, pbeg + per);

  if constexpr (WIDE) {
    // a wave owns consecutive pieces, S at a time: a row's 64 bytes per
    // piece then share cache lines, and one load brings the scales (zero
    // points) of the S, lane j's for piece j
    for (int p0 = pbeg; p0 < pend; p0 += S) {
      uint32_t w[S][OB][BITS];
      ex_u32x4_t x[S][NP][4];
      float s[OB];
      uint32_t z[OB];
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int b = 0; b < OB; ++b)
          load_chunk<BITS>(rows.q[b] + ((int64_t)min(p0 + u, pend - 1) * 4 + j) * BITS, w[u][b]);
      const int64_t g = (int64_t)min(p0 + (j & (S - 1)), pend - 1) * 128 / group;
#pragma unroll
      for (int b = 0; b < OB; ++b) {
        s[b] = rows.s[b][g];
        z[b] = rows.z[b][g];
      }
      const uint16_t* __restrict__ xrow = xrow_of();
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) asm("" : "=v"(x[u][q][i]));   // any value
      if (xok) {
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[u][q][i] = *reinterpret_cast<const ex_u32x4_t*>(xrow + q * xplane + (int64_t)min(p0 + u, pend - 1) * 128 +
                                                                32 * j + 8 * i);
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
          ex_bf16x8_t c[OB];
#pragma unroll
          for (int b = 0; b < OB; ++b) c[b] = mv_codes<BITS>(w[u][b], i, zu[b]);
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            const ex_bf16x8_t a = BITS == 4 ? mv_order(x[u][q][i]) : __builtin_bit_cast(ex_bf16x8_t, x[u][q][i]);
#pragma unroll
            for (int b = 0; b < OB; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, c[b], acc[b], 0, 0, 0);
            if constexpr (BITS == 4) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, xs, 0, 0, 0);
          }
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
    for (int p0 = pbeg; p0 < pend; p0 += S) {
      uint32_t w[S][OB][4];
      ex_u32x4_t x[S][NP][4];
      float s[S][OB];
      uint32_t z[S][OB];
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int c = min(4 * min(p0 + u, pend - 1) + j, nchunks - 1);
        const int64_t g = (int64_t)c * 32 / group;
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          load_chunk<4>(rows.q[b] + (int64_t)c * 4, w[u][b]);
          s[u][b] = rows.s[b][g];
          z[u][b] = rows.z[b][g];
        }
      }
      const uint16_t* __restrict__ xrow = xrow_of();
#pragma unroll
      for (int u = 0; u < S; ++u)
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) asm("" : "=v"(x[u][q][i]));   // any value
      if (xok) {
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = min(4 * min(p0 + u, pend - 1) + i, nchunks - 1);
#pragma unroll
            for (int q = 0; q < NP; ++q)
              x[u][q][i] = *reinterpret_cast<const ex_u32x4_t*>(xrow + q * xplane + (int64_t)c * 32 + 8 * j);
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
          ex_f32x4_t xs = {0.f, 0.f, 0.f, 0.f}, acc[OB];
#pragma unroll
          for (int b = 0; b < OB; ++b) acc[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            const ex_bf16x8_t a = mv_order(x[u][q][i]);
            xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, xs, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < OB; ++b)
              acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, mv_codes<4>(w[u][b], i, 0.f), acc[b], 0, 0, 0);
          }
#pragma unroll
          for (int b = 0; b < OB; ++b) {
            const float si = __shfl(s[u][b], 16 * i + li), zi = 16.f + (float)__shfl((int)z[u][b], 16 * i + li);
#pragma unroll
            for (int r = 0; r < 4; ++r) tot[b][r] = fmaf(si, fmaf(-zi, xs[r], acc[b][r]), tot[b][r]);
          }
        }
      }
    }
  } else {
    const uint16_t* __restrict__ xrow = xrow_of();
    for (int p = part; p < npieces; p += parts) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 4 * p + i;
        if (c >= nchunks) break;
        const int64_t g = (int64_t)c * 32 / group;
        ex_bf16x8_t a[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q) a[q] = *reinterpret_cast<const ex_bf16x8_t*>(xrow + q * xplane + (int64_t)c * 32 + 8 * j);
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          const ex_bf16x8_t w = mv_window<BITS>(rows.q[b] + (int64_t)c * BITS, j, (float)rows.z[b][g]);
          ex_f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < NP; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], w, acc, 0, 0, 0);
          const float s = rows.s[b][g];
#pragma unroll
          for (int r = 0; r < 4; ++r) tot[b][r] = fmaf(s, acc[r], tot[b][r]);
        }
      }
    }
  }
}

}  // namespace gq

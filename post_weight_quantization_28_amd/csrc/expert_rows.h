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
typedef unsigned int ex_u32x2_t __attribute__((ext_vector_type(2)));
typedef ex_u32x4_t ex_u32x4_any_t __attribute__((aligned(2)));

typedef __attribute__((address_space(3))) ex_u32x4_t lds_piece_t;
typedef __attribute__((address_space(3))) const ex_bf16x8_t lds_frag_t;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void lds_write(uint32_t at, ex_u32x4_t v) { *reinterpret_cast<lds_piece_t*>(at) = v; }
__device__ __forceinline__ ex_bf16x8_t lds_frag(uint32_t at) { return *reinterpret_cast<lds_frag_t*>(at); }

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

// The bits of a code in each half of a word, and the patterns of 16.0 around
// them: one from a scalar and one from a vector register, so that masking and
// setting them is one instruction (v_and_or_b32).
struct MvMask {
  uint32_t code = 0x00780078u, base = 0x41804180u;
  __device__ __forceinline__ MvMask() { asm("" : "+s"(code), "+v"(base)); }
};

template <int BITS>
__device__ __forceinline__ ex_bf16x8_t mv_codes(const uint32_t (&w)[BITS], int i, float z, const MvMask& m) {
  if constexpr (BITS == 4) {
    const uint32_t v = w[i];
    const ex_u32x4_t u = {((v << 3) & m.code) | m.base, ((v >> 1) & m.code) | m.base, ((v >> 5) & m.code) | m.base,
                          ((v >> 9) & m.code) | m.base};
    return __builtin_bit_cast(ex_bf16x8_t, u);
  } else {
    float f[8];
    codes8<BITS>(w, i, z, f);
    const ex_u32x4_t u = {pack_exact(f[0], f[1]), pack_exact(f[2], f[3]), pack_exact(f[4], f[5]),
                          pack_exact(f[6], f[7])};
    return __builtin_bit_cast(ex_bf16x8_t, u);
  }
}

// The four quarters (8 codes each) of a chunk, and a quarter's codes as operands.
template <int BITS>
__device__ __forceinline__ void mv_quarters(const uint32_t (&w)[BITS], uint32_t (&part)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int base = 8 * BITS * i, wi = base >> 5, sh = base & 31;
    uint64_t v = w[wi];
    if (sh + 8 * BITS > 32) v |= (uint64_t)w[(wi + 1) % BITS] << 32;     // (never past the last word)
    part[i] = (uint32_t)(v >> sh);
  }
}
template <int BITS>
__device__ __forceinline__ ex_bf16x8_t mv_quarter(uint32_t v, float z, const MvMask& m) {
  if constexpr (BITS == 4) {
    const uint32_t w[4] = {v, 0u, 0u, 0u};
    return mv_codes<4>(w, 0, z, m);
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)((v >> (BITS * i)) & ((1u << BITS) - 1u)) - z;
    const ex_u32x4_t u = {pack_exact(f[0], f[1]), pack_exact(f[2], f[3]), pack_exact(f[4], f[5]), pack_exact(f[6], f[7])};
    return __builtin_bit_cast(ex_bf16x8_t, u);
  }
}

// x0..x7 -> x0 x4 x1 x5 x2 x6 x3 x7, the order of mv_codes<4>
__device__ __forceinline__ ex_bf16x8_t mv_order(ex_u32x4_t x) {
  const ex_u32x4_t u = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                        __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
  return __builtin_bit_cast(ex_bf16x8_t, u);
}

__device__ __forceinline__ void mv_swap32(uint32_t& a, uint32_t& b) {   // a's upper 32 lanes with b's lower
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void mv_swap16(uint32_t& a, uint32_t& b) {   // a's odd rows of 16 with b's even ones
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// w[i] of lane group j (16 lanes) <-> w[j] of lane group i.
__device__ __forceinline__ void mv_transpose(uint32_t (&w)[4]) {
  mv_swap32(w[0], w[2]);
  mv_swap32(w[1], w[3]);
  mv_swap16(w[0], w[1]);
  mv_swap16(w[2], w[3]);
}

// c / d for the same d again and again (d and c d below 2^32 or a division).
struct MvDiv {
  uint32_t d, m;       // m = ceil(2^32 / d): exact while c d < 2^32
  __device__ __forceinline__ MvDiv(uint32_t div, uint32_t most)
      : d(div), m(div > 1 && (uint64_t)div * most < (1ull << 32) ? 0xFFFFFFFFu / div + 1 : 0) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t c) const { return m ? __umulhi(c, m) : (d == 1 ? c : c / d); }
};

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

// What the product of a wave knows of K: chunks, pieces, and the group of a
// piece (WIDE) or chunk.
template <bool WIDE>
struct MvK {
  int nchunks, npieces;
  MvDiv div;
  __device__ __forceinline__ MvK(int64_t n, int group)
      : nchunks((int)(n / 32)), npieces((int)((n / 32 + 3) / 4)),
        div((uint32_t)group / (WIDE ? 128 : 32), (uint32_t)(n / 32)) {}
};

// The product of one wave. What makes such products slow is the number of cache
// lines that their loads touch, not their bytes: a load of one scale per output
// touches a line for each of them, and one of a fragment of X a line per row. (A
// layer of two experts of 3 x 11008 x 4096 for one token took 60 us so, 40 with
// neither of them.) So both go through LDS of the wave's own: rows of X as whole
// lines, in the order in which the fragments want them, SX pieces at a time, and
// the scales and zero points of GB groups at a time, four to a load. These loads
// leave first, then those of the packed codes of SW pieces, which are on their
// way while the others are written to LDS. (Loading a piece's codes again as soon
// as it is multiplied: two pieces share cache lines, which are gone by then, 111
// to 130 us for 32 tokens over 64 experts of 3 x 1408 x 2048; two pieces' 113; a
// second set of registers 125.)
// X: NP pieces of its own, xplane elements apart, whose sum it is. TILE: rows
// that there may be (fragments of the others read some of these: rows of a
// product do not mix).
template <int BITS, bool WIDE, int OB, int NP, int TILE>
struct MvWave {
  static constexpr int SX = 2, SW = OB == 1 ? 4 : 2;     // pieces of X, of codes
  static constexpr int XB = NP * TILE * SX * 256;        // bytes of X
  static constexpr int GB = 128 / (16 * OB) * 2;         // groups at a time (8 or 16): 64 lanes of four
  static constexpr int BYTES = XB + GB * 16 * OB * 8;
  static constexpr int LPR = 16 * SX, RPL = 64 / LPR;    // lanes per row of X, rows per load
  static constexpr int XL = TILE / RPL;                  // loads of X
  const MvRows<OB>& rows;
  const MvK<WIDE> k;
  const MvMask mask;
  const uint16_t* xp[XL];                                // this lane's address of each load, K = 0
  uint32_t lds;
  int nrows, ngroups, n, last, g0;                       // last piece; first of the groups in LDS
  int64_t xplane;
  bool vec;                                              // scales by four
  ex_u32x4_t x[NP][XL];
  uint32_t w[SW][OB][BITS];

  // xrow_of(r): address of row r of the tile (r < nrows)
  template <class XR>
  __device__ __forceinline__ MvWave(const MvRows<OB>& rw, int64_t n_, int group, int nrows_, int64_t plane, uint32_t at,
                                    bool vec_, XR&& xrow_of)
      : rows(rw), k(n_, group), lds(__builtin_amdgcn_readfirstlane(at)), nrows(__builtin_amdgcn_readfirstlane(nrows_)),
        ngroups((int)(n_ / group)), n((int)n_), g0(-GB), xplane(plane), vec(vec_) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if (i * RPL < nrows) xp[i] = xrow_of(min(i * RPL + lane / LPR, nrows - 1)) + 8 * (lane % LPR);
  }

  // where unit u (16 bytes) of row r lies: sixteen rows' same unit in all banks
  static __device__ __forceinline__ uint32_t x_at(int q, int r, int u) {
    return (uint32_t)(((q * TILE + r) * (16 * SX) + (u ^ (r & 15))) * 16);
  }
  __device__ __forceinline__ int group_of(int chunk) const { return (int)k.div((uint32_t)(WIDE ? chunk >> 2 : chunk)); }

  __device__ __forceinline__ void load_x(int p) {
    const int at = min(128 * p, n - 8 - 8 * (int)(threadIdx.x % LPR));   // K may end inside
#pragma unroll
    for (int q = 0; q < NP; ++q)
#pragma unroll
      for (int i = 0; i < XL; ++i)
        if (i * RPL < nrows) x[q][i] = *reinterpret_cast<const ex_u32x4_t*>(xp[i] + q * xplane + at);
  }
  __device__ __forceinline__ void load_w(int u, int p) {
    const int j = (threadIdx.x & 63) >> 4;
    const int64_t at = (int64_t)min(4 * min(p, last) + j, k.nchunks - 1) * BITS;
#pragma unroll
    for (int b = 0; b < OB; ++b) load_chunk<BITS>(rows.q[b] + at, w[u][b]);
  }

  // The scales of the groups from chunk c on, and their way into LDS.
  __device__ __forceinline__ void load_scales(int c, float (&sv)[4], uint32_t (&zv)[4]) {
    const int lane = threadIdx.x & 63;
    g0 = group_of(c) & ~3;
    const int b = OB == 2 ? (lane >> 4) & 1 : 0, t0 = 4 * (lane / (16 * OB));
    const float* sp = b ? rows.s[OB - 1] : rows.s[0];
    const uint8_t* zp = b ? rows.z[OB - 1] : rows.z[0];
    if (vec) {
      const int gc = min(g0 + t0, ngroups - 4);
      const ex_u32x4_t v = *reinterpret_cast<const ex_u32x4_t*>(sp + gc);
      const uint32_t zw = *reinterpret_cast<const uint32_t*>(zp + gc);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        sv[t] = __uint_as_float(v[t]);
        zv[t] = (zw >> (8 * t)) & 255u;
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int gc = min(g0 + t0 + t, ngroups - 1);
        sv[t] = sp[gc];
        zv[t] = zp[gc];
      }
    }
  }
  __device__ __forceinline__ void write_scales(const float (&sv)[4], const uint32_t (&zv)[4]) {
    const int lane = threadIdx.x & 63, t0 = 4 * (lane / (16 * OB));
    const uint32_t at = lds + XB + (t0 * (16 * OB) + lane % (16 * OB)) * 8;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const ex_u32x2_t v = {__float_as_uint(sv[t]), __float_as_uint((float)zv[t] + (BITS == 4 ? 16.f : 0.f))};
      *reinterpret_cast<__attribute__((address_space(3))) ex_u32x2_t*>(at + t * (16 * OB) * 8) = v;
    }
  }
  __device__ __forceinline__ ex_u32x2_t scale(int b, int chunk) const {
    return *reinterpret_cast<__attribute__((address_space(3))) const ex_u32x2_t*>(
        lds + XB + ((group_of(chunk) - g0) * (16 * OB) + 16 * b + (threadIdx.x & 15)) * 8);
  }
  // units of step i: 4 j + i (WIDE), 4 i + j
  __device__ __forceinline__ ex_bf16x8_t frag(int q, int v, int i) const {
    const int j = (threadIdx.x & 63) >> 4;
    return lds_frag(lds + x_at(q, threadIdx.x & (TILE - 1), 16 * v + (WIDE ? 4 * j + i : 4 * i + j)));
  }

  // tot += piece p, whose codes are w[u] and whose X is the v-th of LDS
  __device__ __forceinline__ void add(int u, int v, int p, ex_f32x4_t (&tot)[OB]) {
    const ex_u32x4_t ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const ex_bf16x8_t ones = __builtin_bit_cast(ex_bf16x8_t, ones_bits);
    ex_f32x4_t acc[OB], xs;
    ex_bf16x8_t c[OB];
    ex_u32x2_t sz[OB];
    auto clear = [&]() {
      xs = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < OB; ++b) acc[b] = xs;
    };
    auto multiply = [&](int i) {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const ex_bf16x8_t a = frag(q, v, i);
#pragma unroll
        for (int b = 0; b < OB; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, c[b], acc[b], 0, 0, 0);
        if constexpr (BITS == 4) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, xs, 0, 0, 0);
      }
    };
    auto flush = [&]() {
#pragma unroll
      for (int b = 0; b < OB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float t = BITS == 4 ? fmaf(-__uint_as_float(sz[b][1]), xs[r], acc[b][r]) : acc[b][r];
          tot[b][r] = fmaf(__uint_as_float(sz[b][0]), t, tot[b][r]);
        }
    };
    if constexpr (WIDE) {
      clear();
#pragma unroll
      for (int b = 0; b < OB; ++b) sz[b] = scale(b, 4 * p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int b = 0; b < OB; ++b) c[b] = mv_codes<BITS>(w[u][b], i, __uint_as_float(sz[b][1]), mask);
        multiply(i);
      }
      flush();
    } else {
      // the four quarters of each lane's chunk change lanes: step i has chunk i, quarter j in lane j
      uint32_t quarter[OB][4];
#pragma unroll
      for (int b = 0; b < OB; ++b) {
        mv_quarters<BITS>(w[u][b], quarter[b]);
        mv_transpose(quarter[b]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * p + i >= k.nchunks) break;
        clear();
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          sz[b] = scale(b, 4 * p + i);
          c[b] = mv_quarter<BITS>(quarter[b][i], __uint_as_float(sz[b][1]), mask);
        }
        multiply(i);
        flush();
      }
    }
  }

  // tot += pieces beg .. end - 1
  __device__ __forceinline__ void run(int beg, int end, ex_f32x4_t (&tot)[OB]) {
    const int lane = threadIdx.x & 63;
    last = end - 1;
    for (int p = beg; p < end; p += SW) {
#pragma unroll
      for (int h = 0; h < SW / SX; ++h) {
        const int ph = p + SX * h;
        if (h > 0 && ph >= end) break;
        const bool fresh =
            __builtin_amdgcn_readfirstlane(group_of(min(4 * min(ph + SX - 1, last) + 3, k.nchunks - 1)) >= g0 + GB);
        float sv[4];
        uint32_t zv[4];
        if (fresh) load_scales(4 * ph, sv, zv);
        load_x(ph);
        if (h == 0) {
#pragma unroll
          for (int u = 0; u < SW; ++u) load_w(u, p + u);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (fresh) write_scales(sv, zv);
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int i = 0; i < XL; ++i)
            if (i * RPL < nrows) {
              const ex_u32x4_t v = BITS == 4 ? __builtin_bit_cast(ex_u32x4_t, mv_order(x[q][i])) : x[q][i];
              lds_write(lds + x_at(q, i * RPL + lane / LPR, lane % LPR), v);
            }
        asm volatile("" ::: "memory");                   // (a wave's own LDS operations keep their order)
#pragma unroll
        for (int v = 0; v < SX; ++v) {
          if (ph + v > last) break;
          add(SX * h + v, v, ph + v, tot);
        }
      }
    }
  }
};

// Scales and zero points of four groups can be loaded at once.
__device__ __forceinline__ bool mv_vec(const float* scales, const uint8_t* zeros, int64_t n, int group) {
  return (((uintptr_t)scales & 15) | ((uintptr_t)zeros & 3)) == 0 && n / group % 4 == 0;
}

// tot += the share of part `part` of `parts` of K in the product of up to TILE
// (nrows) rows of X, xrow_of(r) their addresses, and 16 OB packed rows: lane l's
// results are rows 4 (l / 16) .. + 3, output l % 16 of each block. lds:
// MvWave::BYTES of the wave's own, 16-byte aligned. A wave owns consecutive
// pieces.
template <int BITS, bool WIDE, int OB, int NP, int TILE, class XR>
__device__ __forceinline__ void mv_sum(const MvRows<OB>& rows, int64_t n, int group, int part, int parts, int nrows,
                                       int64_t xplane, uint32_t lds, bool vec, XR&& xrow_of, ex_f32x4_t (&tot)[OB]) {
  MvWave<BITS, WIDE, OB, NP, TILE> w(rows, n, group, nrows, xplane, lds, vec, xrow_of);
  const int per = (w.k.npieces + parts - 1) / parts, beg = __builtin_amdgcn_readfirstlane(part) * per;
  w.run(beg, min(w.k.npieces, beg + per), tot);
}

}  // namespace gq

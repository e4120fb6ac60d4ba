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

namespace gq {

typedef __bf16 ex_bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 ex_bf16x2_t __attribute__((ext_vector_type(2)));
typedef float ex_f32x16_t __attribute__((ext_vector_type(16)));
typedef float ex_f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int ex_u32x4_t __attribute__((ext_vector_type(4)));

struct Seg {
  int e;        // expert, -1: no such tile
  int lo, hi;   // its rows
  int row0;     // the tile's first row
};

// Row tile rt of BM rows (every wave of the workgroup finds it for itself).
__device__ __forceinline__ Seg find_tile(const int32_t* __restrict__ offsets, int E, int R, int BM, int rt) {
  const int lane = threadIdx.x & 63;
  if (offsets == nullptr) {
    const bool in = (int64_t)rt * BM < R;
    return Seg{in ? 0 : -1, 0, R, rt * BM};
  }
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = min(max(offsets[e], 0), R);
      hi = min(max(offsets[e + 1], lo), R);
    }
    const int nt = (hi - lo + BM - 1) / BM;
    int inc = nt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    const uint64_t past = __ballot(before + inc > rt);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      const int slo = __shfl(lo, l), shi = __shfl(hi, l);
      const int first = before + __shfl(inc - nt, l);
      return Seg{__builtin_amdgcn_readfirstlane(e0 + l), __builtin_amdgcn_readfirstlane(slo),
                 __builtin_amdgcn_readfirstlane(shi), __builtin_amdgcn_readfirstlane(slo + (rt - first) * BM)};
    }
    before += __shfl(inc, 63);
  }
  return Seg{-1, 0, 0, 0};
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

// Codes 8 j .. 8 j + 7 of a chunk, minus z, as floats (exact).
template <int BITS>
__device__ __forceinline__ void codes8(const uint32_t (&w)[BITS], int j, float z, float (&f)[8]) {
  if constexpr (BITS == 4) {
    // byte i of lo / hi holds code 2 i / 2 i + 1: one conversion per code
    const uint32_t lo = w[j] & 0x0F0F0F0Fu, hi = (w[j] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (float)((lo >> (8 * i)) & 0xFFu) - z;
      f[2 * i + 1] = (float)((hi >> (8 * i)) & 0xFFu) - z;
    }
  } else {
    const int base = 8 * BITS * j, wi = base >> 5, sh = base & 31;
    uint64_t v = w[wi];
    if constexpr (BITS == 3) {
      if (wi + 1 < BITS) v |= (uint64_t)w[wi + 1] << 32;
    }
    v >>= sh;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)(uint32_t)((v >> (BITS * i)) & ((1u << BITS) - 1u)) - z;
  }
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
//    the piece and lane j its codes 8 j .. + 7 (one word at 4 bits), and the
//    sum is scaled after every chunk.
//  * 4 bits: a code in bits 3..6 of the bf16 pattern of 16 is the number
//    16 + q, so one shift and one and-or give two codes (pairs i, i + 4: X's
//    fragment is permuted alike), one operation per code against three with
//    conversions. The offset and the zero point leave through
//    sum_k x (q - z) = sum_k x (16 + q) - (16 + z) sum_k x, the last sum
//    formed by one more product with ones, shared by the OB blocks. All of
//    it in fp32: the offset costs up to a factor of about 6 of fp32's
//    rounding. A row with an infinity gives NaN.
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

template <int BITS, bool WIDE, int WAVES, int OB>
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
  // rows past the segment read its last row; their results are not stored
  const uint16_t* __restrict__ xrow = X + source_row(rows, min(sg.row0 + li, sg.hi - 1), T) * ldx;

  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  const ex_u32x4_t ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const ex_bf16x8_t ones = __builtin_bit_cast(ex_bf16x8_t, ones_bits);

  if constexpr (WIDE) {
    // U pieces' loads are issued before the first product
    constexpr int U = 2;
    for (int p0 = wave; p0 < npieces; p0 += U * WAVES) {
      uint32_t w[U][OB][BITS];
      ex_u32x4_t x[U][4];
      float s[U][OB], z[U][OB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = min(p0 + u * WAVES, npieces - 1);
        const int64_t g = (int64_t)p * 128 / group;
#pragma unroll
        for (int b = 0; b < OB; ++b) {
          load_chunk<BITS>(qrow[b] + ((int64_t)p * 4 + j) * BITS, w[u][b]);
          s[u][b] = srow[b][g];
          z[u][b] = (float)zrow[b][g];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[u][i] = *reinterpret_cast<const ex_u32x4_t*>(xrow + (int64_t)p * 128 + 32 * j + 8 * i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p0 + u * WAVES >= npieces) break;
        ex_f32x4_t acc[OB], xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < OB; ++b) acc[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ex_bf16x8_t a = BITS == 4 ? mv_order(x[u][i]) : __builtin_bit_cast(ex_bf16x8_t, x[u][i]);
#pragma unroll
          for (int b = 0; b < OB; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, mv_codes<BITS>(w[u][b], i, z[u][b]), acc[b], 0, 0, 0);
          if constexpr (BITS == 4) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, xs, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < OB; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = BITS == 4 ? fmaf(-(16.f + z[u][b]), xs[r], acc[b][r]) : acc[b][r];
            tot[b][r] = fmaf(s[u][b], v, tot[b][r]);
          }
      }
    }
  } else {
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
// 256 threads, four waves, a BM x 128 tile with BM = 32 MI WM
// (v_mfma_f32_32x32x16_bf16; wave (wm, wn) holds MI x NI blocks). K advances
// in stages of 64 through two LDS buffers: a stage's operands come from
// registers that were loaded one stage ahead, the packed one is expanded to
// bf16 on its way into LDS, once per workgroup, and one barrier per stage
// separates the buffers. Operand layouts in LDS:
//  * K along a row ([row][64], 128 bytes): 16-byte piece c of row r at
//    c ^ (r & 7), so eight rows' reads of one piece hit all banks;
//  * K down the rows ([64][128], 256 bytes): piece c of row t at
//    c ^ dma_swz(t), read with the transposing LDS read.
constexpr int kExBK = 64;
constexpr int kExBN = 128;

template <int MI_, int NI_, int WM_>
struct ExTile {
  static constexpr int MI = MI_, NI = NI_, WM = WM_, WN = 4 / WM_;
  static constexpr int BM = 32 * MI * WM;
  static_assert(32 * NI * WN == kExBN, "four waves cover 128 columns");
};
using ExTile128 = ExTile<2, 2, 2>;
using ExTile64 = ExTile<2, 1, 1>;
using ExTile32 = ExTile<1, 1, 1>;

__device__ __forceinline__ uint32_t row_piece(int r, int c) { return (uint32_t)r * 128u + 16u * (c ^ (r & 7)); }
__device__ __forceinline__ uint32_t col_piece(int t, int c) { return (uint32_t)t * 256u + 16u * (c ^ dma_swz(t)); }

__device__ __forceinline__ ex_bf16x8_t frag_row(const uint8_t* buf, int row, int kk, int h) {
  return *reinterpret_cast<const ex_bf16x8_t*>(buf + row_piece(row, 2 * kk + h));
}

// Columns c0 .. c0 + 31, K slice kk of 16, from a [64][128] tile: lane l
// gets K 16 kk + 8 (l / 32) .. + 7 of column c0 + l % 32.
__device__ __forceinline__ ex_bf16x8_t frag_col(uint32_t buf, int c0, int kk, int lane) {
  const int t = 16 * kk + 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int col = c0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const uint32_t o0 = col_piece(t, col >> 3) + 2 * (col & 7);
  const uint32_t o1 = col_piece(t + 4, col >> 3) + 2 * (col & 7);
  struct { v4i16_t a, b; } f = {lds_tr16(buf + o0), lds_tr16(buf + o1)};
  return __builtin_bit_cast(ex_bf16x8_t, f);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// 8 elements of a bf16 row from column c (limit: the row's length); vec:
// 16-byte aligned rows and limit % 8 == 0.
__device__ __forceinline__ ex_u32x4_t load_piece(const uint16_t* __restrict__ row, int64_t c, int64_t limit, bool vec) {
  if (c >= limit) return (ex_u32x4_t){0u, 0u, 0u, 0u};
  if (vec) return *reinterpret_cast<const ex_u32x4_t*>(row + c);
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c + i < limit ? row[c + i] : 0u;
  return (ex_u32x4_t){v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

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

struct ExArgs {
  const uint16_t* A; int64_t lda; int avec;   // X or dY
  const int32_t* rows; int T;
  const int32_t* offsets; int E, R;
  const uint32_t* qw; const float* scales; const uint8_t* zeros;
  int64_t d_out, n; int group;
  void* Y; int ybf16; int64_t ldy;
  int nrt, nct;
};

// ---- forward: K = n. The codes minus the zero point are exact in bf16, the
// group's sum is scaled once in fp32 (tot += s acc), as in the one-layer
// product.
template <int BITS, class TL>
__global__ void __launch_bounds__(256, 2)
k_expert_mm(ExArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, PA = BM / 32;
  __shared__ __align__(16) uint8_t As[2][BM * 128];
  __shared__ __align__(16) uint8_t Bs[2][kExBN * 128];
  int rt, ct;
  if (!tile_of(blockIdx.x, p.nrt, p.nct, rt, ct)) return;
  const Seg sg = find_tile(p.offsets, p.E, p.R, BM, rt);
  if (sg.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t o0 = (int64_t)ct * kExBN;
  const int64_t ngroups = p.n / p.group;
  const int cpg = p.group / 32, nchunks = (int)(p.n / 32), nst = (nchunks + 1) / 2;

  // staging: piece tid & 7 of rows tid / 8 + 32 i of A, chunk tid & 1 of row tid / 2 of B
  const uint16_t* arow[PA];
#pragma unroll
  for (int i = 0; i < PA; ++i)
    arow[i] = p.A + source_row(p.rows, min(sg.row0 + (tid >> 3) + 32 * i, sg.hi - 1), p.T) * p.lda;
  const int br = tid >> 1, bc = tid & 1;
  const int64_t bo = (int64_t)sg.e * p.d_out + min(o0 + br, p.d_out - 1);
  const uint32_t* __restrict__ qrow = p.qw + bo * ((int64_t)nchunks * BITS);
  const uint8_t* __restrict__ zrow = p.zeros + bo * ngroups;

  ex_u32x4_t ra[PA];
  uint32_t rb[BITS];
  float rz = 0.f;
  auto gload = [&](int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) ra[i] = load_piece(arow[i], (int64_t)st * kExBK + 8 * (tid & 7), p.n, p.avec);
    const int c = min(2 * st + bc, nchunks - 1);      // a chunk past the end meets zeros of A
    load_chunk<BITS>(qrow + (int64_t)c * BITS, rb);
    rz = (float)zrow[c / cpg];
  };
  auto lwrite = [&](int b) {
#pragma unroll
    for (int i = 0; i < PA; ++i)
      *reinterpret_cast<ex_u32x4_t*>(As[b] + row_piece((tid >> 3) + 32 * i, tid & 7)) = ra[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float f[8];
      codes8<BITS>(rb, e, rz, f);
      *reinterpret_cast<ex_u32x4_t*>(Bs[b] + row_piece(br, 4 * bc + e)) =
          (ex_u32x4_t){pack_exact(f[0], f[1]), pack_exact(f[2], f[3]), pack_exact(f[4], f[5]), pack_exact(f[6], f[7])};
    }
  };
  const float* srow[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni)
    srow[ni] = p.scales + ((int64_t)sg.e * p.d_out + min(o0 + 32 * (NI * wn + ni) + li, p.d_out - 1)) * ngroups;

  ex_f32x16_t acc[MI][NI] = {}, tot[MI][NI] = {};
  float sc[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) sc[ni] = srow[ni][0];
  int cin = 0;
  int64_t g = 0;
  gload(0);
  for (int st = 0; st < nst; ++st) {
    const int b = st & 1;
    lwrite(b);
    __syncthreads();
    if (st + 1 < nst) gload(st + 1);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        const int kk = 2 * hf + k2;
        ex_bf16x8_t fa[MI], fb[NI];
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) fa[mi] = frag_row(As[b], 32 * (MI * wm + mi) + li, kk, h);
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) fb[ni] = frag_row(Bs[b], 32 * (NI * wn + ni) + li, kk, h);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[mi], fb[ni], acc[mi][ni], 0, 0, 0);
      }
      if (++cin == cpg && g < ngroups) {          // the group is complete
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              tot[mi][ni][r] = fmaf(sc[ni], acc[mi][ni][r], tot[mi][ni][r]);
              acc[mi][ni][r] = 0.f;
            }
        cin = 0;
        ++g;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) sc[ni] = srow[ni][min(g, ngroups - 1)];
      }
    }
  }
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t o = o0 + 32 * (NI * wn + ni) + li;
    if (o >= p.d_out) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = sg.row0 + 32 * (MI * wm + mi) + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < sg.hi) store_out(p.Y, p.ybf16, (int64_t)row * p.ldy + o, tot[mi][ni][r]);
      }
  }
}

// ---- gradient: K = d_out, columns n. The scale changes along K, so it
// cannot leave the sum; the weights s (q - z) are rounded to bf16 on their
// way into LDS (relative 2^-8 at most per weight, independent from weight to
// weight, which adds to the sum's error what the bf16 rounding of the result
// adds again). For results kept in fp32 the weight goes as NP = 3 bf16 pieces
// and three products: 24 bits, what its fp32 value holds.
template <int BITS, int NP, class TL>
__global__ void __launch_bounds__(256, NP > 1 ? 1 : 2)
k_expert_mm_grad(ExArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, PA = BM / 32;
  __shared__ __align__(16) uint8_t As[2][BM * 128];
  __shared__ __align__(16) uint8_t Bs[2][NP][kExBK * 256];
  int rt, ct;
  if (!tile_of(blockIdx.x, p.nrt, p.nct, rt, ct)) return;
  const Seg sg = find_tile(p.offsets, p.E, p.R, BM, rt);
  if (sg.e < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t c0 = (int64_t)ct * kExBN;
  const int64_t ngroups = p.n / p.group;
  const int nchunks = (int)(p.n / 32);
  const int nst = (int)ceil_div(p.d_out, kExBK);

  const uint16_t* arow[PA];
#pragma unroll
  for (int i = 0; i < PA; ++i)
    arow[i] = p.A + source_row(p.rows, min(sg.row0 + (tid >> 3) + 32 * i, sg.hi - 1), p.T) * p.lda;
  // B staging: chunk tid & 3 (32 columns) of output row tid / 4
  const int br = tid >> 2, bc = tid & 3;
  const int chunk = (int)(c0 / 32) + bc;
  const bool cok = chunk < nchunks;
  const int cc = min(chunk, nchunks - 1);
  const int64_t ebase = (int64_t)sg.e * p.d_out;
  const int64_t gi = (int64_t)cc * 32 / p.group;

  ex_u32x4_t ra[PA];
  uint32_t rb[BITS];
  float rs = 0.f, rz = 0.f;
  auto gload = [&](int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) ra[i] = load_piece(arow[i], (int64_t)st * kExBK + 8 * (tid & 7), p.d_out, p.avec);
    const int64_t o = (int64_t)st * kExBK + br;
    const int64_t oc = ebase + min(o, p.d_out - 1);
    load_chunk<BITS>(p.qw + (oc * nchunks + cc) * BITS, rb);
    rs = cok && o < p.d_out ? p.scales[oc * ngroups + gi] : 0.f;   // outputs past d_out: weights of 0
    rz = (float)p.zeros[oc * ngroups + gi];
  };
  auto lwrite = [&](int b) {
#pragma unroll
    for (int i = 0; i < PA; ++i)
      *reinterpret_cast<ex_u32x4_t*>(As[b] + row_piece((tid >> 3) + 32 * i, tid & 7)) = ra[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float f[8];
      codes8<BITS>(rb, e, rz, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= rs;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        ex_u32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = ex_pack2(f[2 * i], f[2 * i + 1]);
          f[2 * i] -= __uint_as_float(v[i] << 16);                 // what this piece leaves (exact)
          f[2 * i + 1] -= __uint_as_float(v[i] & 0xFFFF0000u);
        }
        *reinterpret_cast<ex_u32x4_t*>(Bs[b][q] + col_piece(br, 4 * bc + e)) = v;
      }
    }
  };

  ex_f32x16_t acc[MI][NI] = {};
  gload(0);
  for (int st = 0; st < nst; ++st) {
    const int b = st & 1;
    lwrite(b);
    __syncthreads();
    if (st + 1 < nst) gload(st + 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      ex_bf16x8_t fa[MI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fa[mi] = frag_row(As[b], 32 * (MI * wm + mi) + li, kk, h);
#pragma unroll
      for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const ex_bf16x8_t fb = frag_col(lds_addr(Bs[b][q]), 32 * (NI * wn + ni), kk, lane);
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[mi], fb, acc[mi][ni], 0, 0, 0);
        }
    }
  }
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) {
    const int64_t c = c0 + 32 * (NI * wn + ni) + li;
    if (c >= p.n) continue;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = sg.row0 + 32 * (MI * wm + mi) + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row < sg.hi) store_out(p.Y, p.ybf16, (int64_t)row * p.ldy + c, acc[mi][ni][r]);
      }
  }
}

// ---- weight gradient: K = a segment's rows. Both operands have K down their
// rows. The kept values have at most 7 significant bits, so they are exact in
// bf16, products are exact and the sums fp32. A segment's rows are split over
// `splits` workgroups (equal parts, whole stages, from the segment's own
// length) when there are few tiles; their partial sums are added in order by
// a second kernel.
struct KgArgs {
  const uint16_t* P; int64_t ldp; int pvec; int64_t m;
  const int8_t* codes; const uint8_t* exps; int T; int64_t n, pitch;   // pitch: codes per row
  const int32_t* rows; const int32_t* offsets; int E, R;
  int nmt, nnt, splits;
  float* out; int64_t split_stride;   // out[split][e][m][n]
};

template <class TL>
__global__ void __launch_bounds__(256, 2)
k_keep_grad(KgArgs p) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM;
  constexpr int AP = BM / 8;              // 16-byte pieces per row of P's tile
  constexpr int PA = BM / 32;             // pieces per thread
  __shared__ __align__(16) uint8_t As[2][kExBK * 256];
  __shared__ __align__(16) uint8_t Bs[2][kExBK * 256];
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
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t m0 = (int64_t)rt * BM, c0 = (int64_t)ct * kExBN;

  // staging: A piece tid % AP of rows tid / AP + (256 / AP) i; B 32 columns
  // tid & 3 of row tid / 4
  const int ap = tid % AP, ar = tid / AP;
  const int br = tid >> 2, bc = tid & 3;
  const int64_t bcol = c0 + 32 * bc;
  const bool bok = bcol < p.pitch;
  ex_u32x4_t ra[PA], rb[2];
  float rs = 0.f;
  auto gload = [&](int st) {
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = k0 + st * kExBK + ar + (256 / AP) * i;
      ra[i] = r < k1 ? load_piece(p.P + (int64_t)r * p.ldp, m0 + 8 * ap, p.m, p.pvec) : (ex_u32x4_t){0u, 0u, 0u, 0u};
    }
    const int r = k0 + st * kExBK + br;
    if (r < k1 && bok) {
      const int64_t src = source_row(p.rows, r, p.T);
      const ex_u32x4_t* c = reinterpret_cast<const ex_u32x4_t*>(p.codes + src * p.pitch + bcol);
      rb[0] = c[0];
      rb[1] = c[1];
      const uint32_t x = p.exps[src * (p.pitch / 32) + bcol / 32];
      rs = __uint_as_float(x == 255u ? 0x7FC00000u : x << 23);
    } else {                               // rows past the part: zeros on both sides
      rb[0] = rb[1] = (ex_u32x4_t){0u, 0u, 0u, 0u};
      rs = 0.f;
    }
  };
  auto lwrite = [&](int b) {
#pragma unroll
    for (int i = 0; i < PA; ++i)
      *reinterpret_cast<ex_u32x4_t*>(As[b] + col_piece(ar + (256 / AP) * i, ap)) = ra[i];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ex_u32x4_t o;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        // codes + 128 as unsigned bytes: one conversion per code
        const uint32_t u = rb[q >> 1][2 * (q & 1) + w] ^ 0x80808080u;
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = ((float)((u >> (8 * i)) & 0xFFu) - 128.f) * rs;
        o[2 * w] = pack_exact(f[0], f[1]);
        o[2 * w + 1] = pack_exact(f[2], f[3]);
      }
      *reinterpret_cast<ex_u32x4_t*>(Bs[b] + col_piece(br, 4 * bc + q)) = o;
    }
  };

  ex_f32x16_t acc[MI][NI] = {};
  if (nst > 0) gload(0);
  for (int st = 0; st < nst; ++st) {
    const int b = st & 1;
    lwrite(b);
    __syncthreads();
    if (st + 1 < nst) gload(st + 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      ex_bf16x8_t fa[MI], fb[NI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fa[mi] = frag_col(lds_addr(As[b]), 32 * (MI * wm + mi), kk, lane);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) fb[ni] = frag_col(lds_addr(Bs[b]), 32 * (NI * wn + ni), kk, lane);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[mi], fb[ni], acc[mi][ni], 0, 0, 0);
    }
  }
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

// Rows of a tile: 16 is the matrix-vector form.
static int expert_bm(const ExpertArgs& a, int grad) {
  const int64_t avg = ceil_div(a.R, a.E);
  if (!grad && avg <= 16 && ((uintptr_t)a.A & 15) == 0 && a.lda % 8 == 0) return 16;
  return avg <= 64 ? 64 : 128;
}

int64_t expert_grid(const ExpertArgs& a, int grad) {
  const int bm = expert_bm(a, grad);
  const int64_t cols = grad ? a.n : a.d_out;
  return row_tiles(a.R, a.E, bm) * ceil_div(cols, bm == 16 ? 32 : kExBN) + 8;
}

template <int BITS>
static void mv_go(hipStream_t s, const ExpertArgs& a) {
  constexpr int WAVES = 4, OB = 2;
  const dim3 grid((unsigned)ceil_div(a.d_out, 16 * OB), (unsigned)row_tiles(a.R, a.E, 16));
  const uint16_t* X = static_cast<const uint16_t*>(a.A);
  if (a.group % 128 == 0)
    hipLaunchKernelGGL((k_expert_mv<BITS, true, WAVES, OB>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
  else
    hipLaunchKernelGGL((k_expert_mv<BITS, false, WAVES, OB>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
}

static ExArgs ex_args(const ExpertArgs& a, int BM, int64_t kdim, int64_t cols) {
  ExArgs p;
  p.A = static_cast<const uint16_t*>(a.A);
  p.lda = a.lda;
  p.avec = bf16_rows_vec(a.A, a.lda, kdim) ? 1 : 0;
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
  p.nct = (int)ceil_div(cols, kExBN);
  return p;
}

static dim3 tile_grid(int nr, int nc) { return dim3((unsigned)(8 * ceil_div((int64_t)nr * nc, 8))); }

template <int BITS, class TL>
static void mm_go(hipStream_t s, const ExpertArgs& a) {
  const ExArgs p = ex_args(a, TL::BM, a.n, a.d_out);
  hipLaunchKernelGGL((k_expert_mm<BITS, TL>), tile_grid(p.nrt, p.nct), dim3(256), 0, s, p);
}

template <int BITS, int NP, class TL>
static void grad_go(hipStream_t s, const ExpertArgs& a) {
  const ExArgs p = ex_args(a, TL::BM, a.d_out, a.n);
  hipLaunchKernelGGL((k_expert_mm_grad<BITS, NP, TL>), tile_grid(p.nrt, p.nct), dim3(256), 0, s, p);
}

template <int BITS>
static void fwd_bits(hipStream_t s, const ExpertArgs& a) {
  const int bm = expert_bm(a, 0);
  if (bm == 16) mv_go<BITS>(s, a);
  else if (bm == 64) mm_go<BITS, ExTile64>(s, a);
  else mm_go<BITS, ExTile128>(s, a);
}

template <int BITS>
static void grad_bits(hipStream_t s, const ExpertArgs& a) {
  const bool small = expert_bm(a, 1) == 64;
  if (a.y_bf16) {
    if (small) grad_go<BITS, 1, ExTile64>(s, a);
    else grad_go<BITS, 1, ExTile128>(s, a);
  } else {
    if (small) grad_go<BITS, 3, ExTile64>(s, a);
    else grad_go<BITS, 3, ExTile128>(s, a);
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

KeepGradPlan keep_grad_plan(int64_t R, int E, int64_t m, int64_t n) {
  KeepGradPlan p{};
  p.bm = m <= 32 ? 32 : (m <= 64 ? 64 : 128);
  const int64_t tiles = ceil_div(m, p.bm) * ceil_div(n, kExBN) * E;
  const int64_t seg = ceil_div(R, E);                 // rows of an average segment
  int64_t s = tiles > 0 ? 512 / tiles : 1;            // two workgroups per CU
  s = std::min<int64_t>(s, seg / 256);                // at least four stages each
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, 64));
  p.part_bytes = p.splits > 1 ? (size_t)p.splits * E * m * n * sizeof(float) : 0;
  return p;
}

template <class TL>
static void kg_go(hipStream_t s, const KgArgs& p) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)p.nmt * p.nnt, 8)), (unsigned)p.E, (unsigned)p.splits);
  hipLaunchKernelGGL((k_keep_grad<TL>), grid, dim3(256), 0, s, p);
}

hipError_t launch_keep_grad(hipStream_t s, const KeepGradPlan& pl, const uint16_t* P, int64_t ldp, int64_t R, int64_t m,
                            const int8_t* codes, const uint8_t* exps, int64_t T, int64_t n, const int32_t* rows,
                            const int32_t* offsets, int E, float* G, float* part) {
  if (m <= 0 || n <= 0 || E <= 0) return hipSuccess;
  KgArgs p;
  p.P = P;
  p.ldp = ldp;
  p.pvec = bf16_rows_vec(P, ldp, m) ? 1 : 0;
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
  p.nmt = (int)ceil_div(m, pl.bm);
  p.nnt = (int)ceil_div(n, kExBN);
  p.splits = pl.splits;
  p.out = pl.splits > 1 ? part : G;
  p.split_stride = (int64_t)E * m * n;
  if (pl.bm == 32) kg_go<ExTile32>(s, p);
  else if (pl.bm == 64) kg_go<ExTile64>(s, p);
  else kg_go<ExTile128>(s, p);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || pl.splits <= 1) return err;
  const int64_t count = (int64_t)E * m * n;
  hipLaunchKernelGGL(k_keep_grad_sum, dim3((unsigned)ceil_div(count, 256)), dim3(256), 0, s, part, pl.splits, count, G);
  return hipGetLastError();
}

}  // namespace gq

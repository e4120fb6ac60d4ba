// The products of many rows with packed weights: tiles of 32 to 128 rows by
// register prefetch, 256 x 256 tiles by DMA rings; and what the gradients share
// with them.
#pragma once
#include "common.h"
#include "dma.h"
#include "expert_rows.h"

#include <algorithm>
#include <type_traits>

namespace gq {

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

__device__ __forceinline__ uint32_t row_piece(int r, int c) { return (uint32_t)r * 128u + 16u * (c ^ ((r >> 1) & 7)); }
// W: columns of the tile
template <int W>
__device__ __forceinline__ uint32_t col_piece(int t, int c) {
  const int x = W == 128 ? (t >> 1) & 1 : (c >> 4) & 1;
  return (uint32_t)t * (2 * W) + 16u * (c ^ dma_swz(t) ^ x);
}

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

// What follows a product: nothing, or what stands behind it in a model (linear.hip).
// A gated one computes the columns of the gate and of the other factor side by
// side: 32 of the one, 32 of the other, in turn, so that a lane has both.
struct NoEnd {
  static constexpr bool GATED = false, STORES = false;
};

// Packed row (of an expert's d_out) of column c of the tile whose first output
// is o0, past the last one: some row.
template <class END>
__device__ __forceinline__ int64_t tile_row(int64_t o0, int c, int64_t d_out) {
  if constexpr (END::GATED) {
    const int64_t d = d_out / 2;
    return min(o0 + 32 * (c >> 6) + (c & 31), d - 1) + ((c >> 5) & 1) * d;
  }
  return min(o0 + c, d_out - 1);
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
// product. GS: stages of a group where groups are whole stages, 1 (64 codes) or 2
// (the first product of a group starts from zero, no test inside a stage);
// 0: groups of any number of 32-code chunks, tested after every chunk.
template <int BITS, class TL, int GS, class END>
__global__ void __launch_bounds__(TL::THREADS, 512 / TL::THREADS)
k_expert_mm(ExArgs p, END finish) {
  constexpr int MI = TL::MI, NI = TL::NI, BM = TL::BM, PA = TL::PA, NB = TL::NB, THREADS = TL::THREADS;
  constexpr uint32_t ASZ = BM * 128, BSZ = TL::BN * 128, BUF = ASZ + BSZ;
  __shared__ __align__(16) uint8_t smem[2 * BUF];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, BM, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % TL::WM, wn = wave / TL::WM, h = lane >> 5, li = lane & 31;
  const int64_t o0 = (int64_t)ct * (END::GATED ? TL::BN / 2 : TL::BN);
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
  const int64_t bo = (int64_t)sg.e * p.d_out + tile_row<END>(o0, br, p.d_out);
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
    const int g = GS == 2 ? (s0 + st) >> 1 : (GS == 1 ? min(s0 + st, (int)ngroups - 1) : c / cpg);
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
    srow[ni] = p.scales + ((int64_t)sg.e * p.d_out + tile_row<END>(o0, 32 * (NI * wn + ni) + li, p.d_out)) * ngroups;
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
              fa[kk & 1][mi], fb[kk & 1][ni], GS > 0 && kk == 0 && (GS == 1 || b == 0) ? zero : acc[mi][ni], 0, 0, 0);
      bwrite(next, KK);
      if (GS == 0 && (kk & 1) == 1 && ++cin == cpg && g < ngroups) {   // the group is complete
        flush();
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = zero;
        cin = 0;
      }
    });
    awrite(next, st + 1);
    if (GS == 1 || (GS == 2 && b == 1)) flush();
  };
  for_four([&](auto S) {
    if constexpr (S < DA) aload(S, min((int)S, nst - 1));
    if constexpr (S < DB) bload(S, min((int)S, nst - 1));
  });
  awrite(ex_const<0>{}, 0);
  for_four([&](auto KK) { bwrite(ex_const<0>{}, KK); });
  run_stages<U>(nst, stage);
  if constexpr (END::STORES) {
    __syncthreads();                                       // the tiles in LDS are done with
    finish.template store<MI, NI>(sg.e, sg.row0 + 32 * MI * wm, sg.hi, o0, NI * wn, lds + wave * END::LDS,
                                  [&](auto M, auto N, int r) { return tot[M][N][r]; });
    return;
  }
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
template <class END>
__global__ void __launch_bounds__(512, 2)
k_expert_ring(ExArgs p, END finish) {
  constexpr int MI = 4, NI = 2;
  __shared__ __align__(16) uint8_t smem[kFLds];
  int ct;
  Seg sg;
  if (!locate(p.offsets, p.E, p.R, 256, blockIdx.x, p.nct, ct, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3, h = lane >> 5, li = lane & 31;
  const int64_t o0 = (int64_t)ct * (END::GATED ? 128 : 256);
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
    vq[i] = (uint32_t)(tile_row<END>(o0, r, p.d_out) * (p.n / 2) + c);
  }
  // scales (waves 0..3) and zero points (4..7) of a block: one row per lane
  const int w4 = wave & 3;
  const uint32_t vs = (uint32_t)(tile_row<END>(o0, 64 * w4 + lane, p.d_out) * ngroups);
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
  if constexpr (END::STORES) {
    __syncthreads();                                   // or that holds results
    finish.template store<MI, NI>(sg.e, sg.row0 + 128 * wm, sg.hi, o0, NI * wn, lds + wave * END::LDS,
                                  [&](auto M, auto N, int r) { return unit[N] * acc[M][N][r]; });
    return;
  }
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

// ---------------------------------------------------------------- host
inline int64_t row_tiles(int64_t R, int E, int BM) { return std::min<int64_t>(R, ceil_div(R, BM) + E - 1); }

inline bool bf16_rows_vec(const void* p, int64_t ld, int64_t cols) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && cols % 8 == 0;
}

inline dim3 tile_grid(int nr, int nc) { return dim3((unsigned)(8 * ceil_div((int64_t)nr * nc, 8))); }

inline ExArgs ex_args(const ExpertArgs& a, int BM, int BN, int64_t cols) {
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

}  // namespace gq

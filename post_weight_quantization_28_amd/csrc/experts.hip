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
#include "expert_tiles.h"

#include <algorithm>
#include <type_traits>

namespace gq {

// ==================================================================== few rows
//
// Matrix-vector products: bound by reading the packed weights once. A
// workgroup of WAVES waves owns 16 OB outputs of one expert and up to TILE of
// its rows (v_mfma_f32_16x16x32_bf16, X as the A operand), and its waves
// split K (MvWave in expert_rows.h). K advances in pieces of 128 codes.
//  * Groups that are multiples of 128 (WIDE): lane l (output l % 16,
//    j = l / 16) loads the 32 consecutive codes 32 j .. of its output's piece
//    in one go (16 bytes at 4 bits); MFMA step i then takes codes
//    32 j + 8 i .. + 7 of every lane. The order of K inside a product is
//    free as long as X's fragment follows it.
//  * Other groups: a product must not mix groups, so step i takes chunk i of
//    the piece and lane j its codes 8 j .. + 7, and the sum is scaled after
//    every chunk. A lane still loads a chunk in one go and four lane swaps hand
//    out its quarters (360 rows over 64 experts, 322 x 4608 in groups of 32: 30
//    us at 4 bits; at 3 and 2 bits, whose words were loaded chunk by chunk
//    before, 97 and 73 to 33 and 31; two of 11008 x 4096 for one token each, groups
//    of 64, 94 and 73 to 26 and 25).
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
// Measured in captured calls (two experts of 11008 x 4096 for one token / 64
// experts of 1408 x 2048 for 256 rows, 4 bits, groups of 128; 48.6 and 99 MB,
// which are read in 9.4 and 17.6 us in the same pattern): 17.6 / 31 us, with
// scales and rows of X loaded to where they are used 23.6 / 34.6. With tiles of
// 8 rows up to 8 rows an expert; of 16: 20.6 / 33.5, and with 16 rows each 64 in
// tiles of 8, 55 of 16.
template <int BITS, bool WIDE, int WAVES, int OB, int TILE>
__global__ void __launch_bounds__(64 * WAVES, 4)
k_expert_mv(const uint16_t* __restrict__ X, int T, int64_t n, int64_t ldx, const int32_t* __restrict__ rows,
            const int32_t* __restrict__ offsets, int E, int R, const uint32_t* __restrict__ qw,
            const float* __restrict__ scales, const uint8_t* __restrict__ zeros, int64_t d_out, int group,
            void* __restrict__ Y, int ybf16, int64_t ldy) {
  __shared__ __align__(16) uint8_t smem[WAVES][MvWave<BITS, WIDE, OB, 1, TILE>::BYTES];
  __shared__ float red[WAVES][OB][4][64];
  const Seg sg = find_tile(offsets, E, R, TILE, blockIdx.y);
  if (sg.e < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int64_t obase = (int64_t)sg.e * d_out;
  int64_t orow[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) orow[b] = obase + min((int64_t)blockIdx.x * (16 * OB) + 16 * b + li, d_out - 1);
  const MvRows<OB> w(qw, scales, zeros, orow, n, group, BITS);
  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  const int nrows = min(sg.hi - sg.row0, TILE);
  auto xrow = [&](int r) { return X + source_row(rows, sg.row0 + r, T) * ldx; };
  mv_sum<BITS, WIDE, OB, 1, TILE>(w, n, group, wave, WAVES, nrows, 0, lds_addr(smem[wave]),
                                  mv_vec(scales, zeros, n, group), xrow, tot);
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
    if (o < d_out && row < min(sg.hi, sg.row0 + TILE)) store_out(Y, ybf16, (int64_t)row * ldy + o, v);
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
//  * Matrix-vector form and 64-row tiles, 4 bits, captured: 8 experts of 4096 x
//    4096 with 1, 8, 16, 20 and 32 rows each 20, 22, 26, 38, 39 and 46, 46, 47, 44,
//    46 us; 64 of 1408 x 2048 with 1, 8, 16, 20 and 32 30, 33, 41, 64, 70 and 60, 58,
//    59, 59, 61; groups of 64 with 16 and 24 rows 37, 50 and 51, 51, 48, 81 and 64,
//    65. 3 bits with 16 and 24 rows 30, 46 and 87, 79, 41, 71 and 112, 114; 2 bits
//    29, 44 and 52, 48, 39, 67 and 65, 65. So from 17 rows on either may be ahead,
//    by what a second tile costs and whether the tiles have K in parts (two of
//    11008 x 4096 with 32 rows 31 and 41, at 3 bits 37 and 71): here the border is 16
//    for all of them; linear, in linear.hip, goes by that.
//  * Ring and 128-row tiles: 8 experts of 4096 x 4096 with 512, 640 and 1024
//    rows each 247, 251, 381 and 219, 258, 392 us, gradient 222, 228, 348 and
//    219, 257, 391; 8 of 11008 x 4096 506, 562, 901 and 568, 661, 1030. Fewer
//    rows go either way with how full the last tiles are (256 rows: 125 and 136,
//    but 372 and 343).
int expert_bm(const ExpertArgs& a, int grad) {
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

template <int BITS, int TILE>
static void mv_go(hipStream_t s, const ExpertArgs& a) {
  constexpr int WAVES = 4, OB = 2;
  const dim3 grid((unsigned)ceil_div(a.d_out, 16 * OB), (unsigned)row_tiles(a.R, a.E, TILE));
  const uint16_t* X = static_cast<const uint16_t*>(a.A);
  if (a.group % 128 == 0)
    hipLaunchKernelGGL((k_expert_mv<BITS, true, WAVES, OB, TILE>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
  else
    hipLaunchKernelGGL((k_expert_mv<BITS, false, WAVES, OB, TILE>), grid, dim3(64 * WAVES), 0, s, X, a.T, a.n, a.lda, a.rows,
                       a.offsets, a.E, a.R, a.qw, a.scales, a.zeros, a.d_out, a.group, a.Y, a.y_bf16, a.ldy);
}

// The tile kernels write their parts of K into the workspace when there are
// several; a.parts_only: they stay there.
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
  if (sp.splits > 1 && !a.parts_only)
    hipLaunchKernelGGL(k_expert_sum, dim3((unsigned)ceil_div((int64_t)a.R * cols, 256)), dim3(256), 0, s,
                       static_cast<const float*>(a.part), sp.splits, a.R, (uint32_t)cols, a.offsets, a.E, a.Y, a.y_bf16,
                       a.ldy);
}

template <int BITS, class TL, int GS>
static void mm_go(hipStream_t s, const ExpertArgs& a) {
  split_go(s, a, ex_args(a, TL::BM, TL::BN, a.d_out), a.d_out, 0, [&](dim3 grid, const ExArgs& p) {
    hipLaunchKernelGGL((k_expert_mm<BITS, TL, GS, NoEnd>), grid, dim3(TL::THREADS), 0, s, p, NoEnd{});
  });
}

// Groups of 128 are worth their own code at 4 bits, the common layer: 8 experts
// of 4096 x 4096 with 32, 96, 200 and 400 rows each 51, 71, 121 and 183 us, in
// the code for any group 56, 77, 135 and 196. Groups of 64 in 64-row tiles: 96
// rows each 75 and 86; in 128-row tiles their code spills (119 to 195 us for 4096
// rows over 64 experts of 1408 x 2048).
template <int BITS, class TL>
static void mm_group(hipStream_t s, const ExpertArgs& a) {
  if constexpr (BITS == 4) {
    if (a.group == 128) return mm_go<4, TL, 2>(s, a);
    if constexpr (TL::BM == 64) {
      if (a.group == 64) return mm_go<4, TL, 1>(s, a);
    }
  }
  mm_go<BITS, TL, 0>(s, a);
}

template <int BITS, int NP, class TL, bool WIDE>
static void grad_go(hipStream_t s, const ExpertArgs& a) {
  split_go(s, a, ex_args(a, TL::BM, TL::BN, a.n), a.n, 1, [&](dim3 grid, const ExArgs& p) {
    hipLaunchKernelGGL((k_expert_mm_grad<BITS, NP, TL, WIDE>), grid, dim3(TL::THREADS), 0, s, p);
  });
}

static void ring_go(hipStream_t s, const ExpertArgs& a, int grad) {
  const ExArgs p = ex_args(a, 256, 256, grad ? a.n : a.d_out);
  const dim3 grid = tile_grid(p.nrt, p.nct);
  if (grad) hipLaunchKernelGGL(k_expert_ring_grad, grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL(k_expert_ring<NoEnd>, grid, dim3(512), 0, s, p, NoEnd{});
}

template <int BITS>
static void fwd_bits(hipStream_t s, const ExpertArgs& a) {
  const int bm = expert_bm(a, 0);
  if (bm == 16 && a.R > 8 * a.E) mv_go<BITS, 16>(s, a);
  else if (bm == 16) mv_go<BITS, 8>(s, a);
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

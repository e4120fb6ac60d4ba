// A whole layer of experts for a few tokens, in two launches:
//
//   h[t, j] = end(U_e x_t + b1_e),          e = ids[t, j]
//   Y[t] = residual[t] + sum_j w[t, j] (D_e h[t, j] + b2_e)
//
// Bound by reading the packed weights of the experts in use once. The slots
// (t, j) of one expert go through the matrix-vector product together, up to 16
// to a tile (v_mfma_f32_16x16x32_bf16). Every workgroup sorts the slots by
// expert for itself: that costs it about a microsecond and spares the launches
// that would order rows, move them, and add them up again.
//  * k_layer_up: a workgroup owns 16 columns of h (32 without a gate) of one
//    tile, gate and other factor side by side, and its waves split K. h goes to
//    the workspace as bf16 pieces.
//  * k_layer_down: a workgroup owns 16 columns of Y for all tokens. Its waves
//    share the tiles (and K, when the tiles are fewer than the waves), leave
//    their results by slot in LDS, and the slots of a token are added in their
//    order: no result depends on timing.
#include "act.h"
#include "common.h"
#include "expert_rows.h"

#include <algorithm>

namespace gq {

constexpr int kLyMax = kLayerMaxSlots;

// Slots by expert: `sorted` lists them expert by expert (in slot order), tile i
// holds the slots sorted[start[i]] .. of expert e[i], up to TILE of them.
struct LySort {
  uint16_t sorted[kLyMax], start[kLyMax], end[kLyMax], expert[kLyMax];
  uint16_t tiles, places;                // places: slots with an expert
};
struct LyScratch {
  int32_t id[kLyMax];                    // -1: no expert
  uint16_t place[kLyMax];                // of a slot with an expert, in `sorted`
  int32_t count[kRouteMaxExperts];       // then the expert's first place (low half) and first tile (high half)
};

// Called by whole workgroups of THREADS threads.
template <int THREADS, int TILE>
__device__ __forceinline__ void ly_sort(const int32_t* __restrict__ ids, int64_t ldi, int slots, int k, int E, LySort& so,
                                        LyScratch& sc) {
  const int tid = threadIdx.x;
  for (int i = tid; i < E; i += THREADS) sc.count[i] = 0;
  for (int i = tid; i < slots; i += THREADS) {
    const int t = i / k, id = ids[t * ldi + (i - t * k)];
    sc.id[i] = id >= 0 && id < E ? id : -1;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS)
    if (sc.id[i] >= 0) atomicAdd(&sc.count[sc.id[i]], 1);
  __syncthreads();
  if (tid < 64) {
    int places = 0, tiles = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int c = e0 + tid < E ? sc.count[e0 + tid] : 0, nt = (c + TILE - 1) / TILE;
      const int pc = wave_scan(c), pt = wave_scan(nt);
      if (e0 + tid < E) sc.count[e0 + tid] = (places + pc - c) | (tiles + pt - nt) << 16;
      places += __builtin_amdgcn_readlane(pc, 63);
      tiles += __builtin_amdgcn_readlane(pt, 63);
    }
    if (tid == 0) {
      so.tiles = (uint16_t)tiles;
      so.places = (uint16_t)places;
    }
  }
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const int id = sc.id[i];
    if (id < 0) continue;
    int rank = 0, all = 0;                               // equal ids before this slot, and at all
    for (int s = 0; s < slots; ++s) {
      const bool same = sc.id[s] == id;
      all += same;
      rank += same && s < i;
    }
    const int place = (sc.count[id] & 0xFFFF) + rank, tile = (sc.count[id] >> 16) + rank / TILE;
    so.sorted[place] = (uint16_t)i;
    sc.place[i] = (uint16_t)place;
    if (rank % TILE == 0) {
      so.start[tile] = (uint16_t)place;
      so.end[tile] = (uint16_t)(place + min(TILE, all - rank));
      so.expert[tile] = (uint16_t)id;
    }
  }
  __syncthreads();
}

template <int BITS, bool WIDE, bool GATED>
__global__ void __launch_bounds__(256)
k_layer_up(LayerArgs a) {
  constexpr int WAVES = 4, OB = 2, S = 2;
  __shared__ LySort so;
  __shared__ union {
    LyScratch sort;
    float red[WAVES][OB][4][64];
  } sh;
  ly_sort<256, 16>(a.ids, a.ldi, a.slots, a.k, a.E, so, sh.sort);
  const int tile = blockIdx.y;
  if (tile >= so.tiles) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15;
  const int e = so.expert[tile], first = so.start[tile], rows = so.end[tile] - first;
  const int64_t m = GATED ? 2 * a.d : a.d, o0 = (int64_t)blockIdx.x * (GATED ? 16 : 32);
  // column of h and packed row of output b, li
  auto column = [&](int b, int l) { return o0 + (GATED ? 0 : 16 * b) + l; };
  int64_t orow[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) orow[b] = e * m + min(column(b, li), a.d - 1) + (GATED ? b * a.d : 0);
  const MvRows<OB> w(a.up.qw, a.up.scales, a.up.zeros, orow, a.n, a.group, BITS);
  const uint16_t* x = a.X + (int64_t)(so.sorted[first + min(li, rows - 1)] / a.k) * a.ldx;
  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  mv_sum<BITS, WIDE, OB, S, 1>(w, a.n, a.group, wave, WAVES, li < rows, 0, [&]() { return x; }, tot);
#pragma unroll
  for (int b = 0; b < OB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh.red[wave][b][r][lane] = tot[b][r];
  __syncthreads();
  for (int i = threadIdx.x; i < (GATED ? 1 : OB) * 256; i += 256) {
    const int b0 = i >> 8, r = (i >> 6) & 3, l = i & 63;
    const int64_t c = column(b0, l & 15);
    const int row = 4 * (l >> 4) + r;
    if (c >= a.d || row >= rows) continue;
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
#pragma unroll
      for (int v = 0; v < WAVES; ++v) z[h] += sh.red[v][GATED ? h : b0][r][l];
      if (a.b1) z[h] += a.b1[e * m + h * a.d + c];
    }
    float h = act_value(a.act, z[0]);
    if constexpr (GATED) h *= z[1];
    uint16_t* out = a.H + (int64_t)so.sorted[first + row] * a.d + c;
    for (int q = 0; q < a.pieces; ++q) {                 // what a piece leaves is exact
      const uint32_t p = ex_pack2(h, 0.f);
      out[q * a.plane] = (uint16_t)p;
      h -= __uint_as_float(p << 16);
    }
  }
}

template <int BITS, bool WIDE, int NP>
__global__ void __launch_bounds__(64 * kLayerDownWaves)
k_layer_down(LayerArgs a) {
  constexpr int WAVES = kLayerDownWaves, S = 2;
  __shared__ LySort so;
  __shared__ LyScratch scratch;
  extern __shared__ float part[];                        // [part of K][place][column]
  ly_sort<64 * WAVES, 16>(a.ids, a.ldi, a.slots, a.k, a.E, so, scratch);
  const int tiles = so.tiles, places = so.places;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  const int kp = tiles >= WAVES || tiles == 0 ? 1 : WAVES / tiles;
  for (int i = wave; i < tiles * kp; i += WAVES) {
    const int tile = i / kp, p = i - tile * kp;
    const int e = so.expert[tile], first = so.start[tile], rows = so.end[tile] - first;
    const int64_t orow[1] = {(int64_t)e * a.n + min(o0 + li, a.n - 1)};
    const MvRows<1> w(a.down.qw, a.down.scales, a.down.zeros, orow, a.d, a.group, BITS);
    const uint16_t* h = a.H + (int64_t)so.sorted[first + min(li, rows - 1)] * a.d;
    ex_f32x4_t tot[1] = {{0.f, 0.f, 0.f, 0.f}};
    mv_sum<BITS, WIDE, 1, S, NP>(w, a.d, a.group, p, kp, li < rows, a.plane, [&]() { return h; }, tot);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * (lane >> 4) + r;
      if (row < rows) part[(p * places + first + row) * 16 + li] = tot[0][r];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 64 * WAVES) {
    const int t = i >> 4, c = i & 15;
    const int64_t o = o0 + c;
    if (o >= a.n) continue;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int s = t * a.k + j, id = scratch.id[s];
      if (id < 0) continue;
      float v = 0.f;
      for (int p = 0; p < kp; ++p) v += part[(p * places + scratch.place[s]) * 16 + c];
      if (a.b2) v += a.b2[id * a.n + o];
      y = fmaf(a.w ? a.w[s] : 1.f, v, y);
    }
    if (a.res) {
      const int64_t at = t * a.ldr + o;
      y += a.res_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.res)[at] << 16)
                      : static_cast<const float*>(a.res)[at];
    }
    store_out(a.Y, a.y_bf16, t * a.ldy + o, y);
  }
}

// ---------------------------------------------------------------- host
int layer_pieces(int y_bf16) { return y_bf16 ? 1 : 3; }

template <int BITS, bool WIDE>
static void ly_go(hipStream_t s, const LayerArgs& a) {
  const int64_t tiles = std::min<int64_t>(a.slots, ceil_div(a.slots, 16) + a.E - 1);
  const dim3 up((unsigned)ceil_div(a.d, a.gated ? 16 : 32), (unsigned)tiles), down((unsigned)ceil_div(a.n, 16));
  if (a.gated) hipLaunchKernelGGL((k_layer_up<BITS, WIDE, true>), up, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_layer_up<BITS, WIDE, false>), up, dim3(256), 0, s, a);
  // K is in waves / tiles parts while the tiles are fewer than the waves: 16 slots a tile, 16 waves times 16 places
  const size_t lds = std::max<size_t>(a.slots, (size_t)std::min(a.slots, 16) * kLayerDownWaves) * 64;
  const dim3 block(64 * kLayerDownWaves);
  if (a.pieces == 1) hipLaunchKernelGGL((k_layer_down<BITS, WIDE, 1>), down, block, lds, s, a);
  else hipLaunchKernelGGL((k_layer_down<BITS, WIDE, 3>), down, block, lds, s, a);
}

template <int BITS>
static void ly_bits(hipStream_t s, const LayerArgs& a) {
  if (a.group % 128 == 0) ly_go<BITS, true>(s, a);
  else ly_go<BITS, false>(s, a);
}

hipError_t launch_layer(hipStream_t s, const LayerArgs& a) {
  if (a.bits == 2) ly_bits<2>(s, a);
  else if (a.bits == 3) ly_bits<3>(s, a);
  else ly_bits<4>(s, a);
  return hipGetLastError();
}

}  // namespace gq

// A whole layer of experts for a few tokens, in two launches:
//
//   h[t, j] = end(U_e x_t + b1_e),          e = ids[t, j]
//   Y[t] = residual[t] + sum_j w[t, j] (D_e h[t, j] + b2_e)
//
// Bound by reading the packed weights of the experts in use once. The slots
// (t, j) of one expert go through the matrix-vector product together, up to 8
// to a tile (v_mfma_f32_16x16x32_bf16). Every workgroup of the first launch finds
// the slots of its tile for itself, which spares the launches that would order
// rows, move them, and add them up again.
//  * k_layer_up: a workgroup owns 16 columns of h (32 without a gate) of one
//    tile, gate and other factor side by side, and its waves split K. h goes to
//    the workspace as bf16 pieces.
//  * k_layer_down: a workgroup owns 16 columns of Y for all tokens. Its waves
//    share the tiles (and K, when the tiles are fewer than the waves), leave
//    their results by slot in LDS, and the slots of a token are added in their
//    order: no result depends on timing.
// Tiles are of 4 slots for up to 4 tokens and where Y is fp32 (h then has three
// pieces), of 8 beyond (16 take LDS from the second launch's 16 waves). Measured at 4 bits, groups of 128 (both launches of
// a call among others): one token through 2 of 8 experts of 3 x 11008 x 4096, 146
// MB, 43 us (25 + 18); one through 8 of 64 of 3 x 1408 x 2048, 37 MB, 19 us (10 +
// 11); 32 tokens through these 64, 294 MB, 107 us (55 + 47). Every workgroup
// sorting all slots by comparing them pairwise took 175 us of the last.
// Half as many columns a workgroup in the second launch, K in two halves beside
// each other in the product's columns: 11 to 14 and 51 to 58 us.
#include "act.h"
#include "common.h"
#include "expert_rows.h"

#include <algorithm>

namespace gq {

constexpr int kLyMax = kLayerMaxSlots, kLyMost = 8;

// A tile: up to TILE slots of one expert, in slot order. The places of all tiles'
// slots follow each other.
struct LyTile {
  int e, rows, first;                    // first: place of its first slot
  uint16_t slot[kLyMost];
};
// What the first launch leaves for the second, in front of h.
struct LyTable {
  int tiles, places;
  LyTile tile[1];
};

// The up to TILE slots of tile number `tile` (rows = 0: no such tile) by one
// histogram of the slots' experts in LDS, which every wave of the workgroup
// scans for itself.
template <int THREADS, int TILE>
__device__ __forceinline__ LyTile ly_find(const LayerArgs& a, int tile, int16_t* id, int32_t* count, uint16_t* list,
                                          int& tiles, int& places) {
  const int tid = threadIdx.x, lane = tid & 63;
  for (int i = tid; i < a.E; i += THREADS) count[i] = 0;
  __syncthreads();
  for (int i = tid; i < a.slots; i += THREADS) {
    const int t = i / a.k, v = a.ids[t * a.ldi + (i - t * a.k)];
    const bool ok = v >= 0 && v < a.E;
    id[i] = (int16_t)(ok ? v : -1);
    if (ok) atomicAdd(&count[v], 1);
  }
  __syncthreads();
  LyTile r;
  r.e = -1;
  r.rows = r.first = tiles = places = 0;
  int skip = 0;                          // slots of the expert in its tiles before this one
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int c = e0 + lane < a.E ? count[e0 + lane] : 0, nt = (c + TILE - 1) / TILE;
    const int pc = wave_scan(c), pt = wave_scan(nt);
    const uint64_t past = __ballot(tiles + pt > tile);
    if (r.e < 0 && past) {
      const int l = __ffsll((long long)past) - 1;
      skip = TILE * (tile - tiles - __builtin_amdgcn_readlane(pt - nt, l));
      r.e = e0 + l;
      r.rows = min(TILE, __builtin_amdgcn_readlane(c, l) - skip);
      r.first = places + __builtin_amdgcn_readlane(pc - c, l) + skip;
    }
    places += __builtin_amdgcn_readlane(pc, 63);
    tiles += __builtin_amdgcn_readlane(pt, 63);
  }
  int rank = -skip;
  for (int s0 = 0; s0 < a.slots && rank < r.rows; s0 += 64) {
    const bool mine = s0 + lane < a.slots && id[s0 + lane] == r.e;
    const uint64_t all = __ballot(mine);
    const int at = rank + __popcll(all & ((1ull << lane) - 1));
    if (mine && at >= 0 && at < r.rows) list[at] = (uint16_t)(s0 + lane);   // every wave writes the same
    rank += __popcll(all);
  }
  return r;
}

template <int BITS, bool WIDE, bool GATED, int TILE>
__global__ void __launch_bounds__(256, 4)
k_layer_up(LayerArgs a) {
  constexpr int WAVES = 4, OB = 2;
  __shared__ union {
    struct {
      int16_t id[kLyMax];
      int32_t count[kRouteMaxExperts];
    } find;
    float red[WAVES][OB][4][64];
  } sh;
  __shared__ __align__(16) uint8_t smem[WAVES][MvWave<BITS, WIDE, OB, 1, TILE>::BYTES];
  __shared__ uint16_t list[TILE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15;
  const int tile = blockIdx.y;
  LyTile t;
  if (a.T == 1) {                                        // a tile per slot
    t.e = a.ids[tile];
    t.rows = t.e >= 0 && t.e < a.E;
    if (threadIdx.x == 0) list[0] = (uint16_t)tile;
  } else {
    int tiles, places;
    t = ly_find<256, TILE>(a, tile, sh.find.id, sh.find.count, list, tiles, places);
    if (blockIdx.x == 0 && threadIdx.x < TILE) {
      LyTable* table = static_cast<LyTable*>(a.table);
      if (tile == 0 && threadIdx.x == 0) {
        table->tiles = tiles;
        table->places = places;
      }
      if ((int)threadIdx.x < t.rows) table->tile[tile].slot[threadIdx.x] = list[threadIdx.x];
      if (threadIdx.x == 0 && t.rows > 0) {
        table->tile[tile].e = t.e;
        table->tile[tile].rows = t.rows;
        table->tile[tile].first = t.first;
      }
    }
  }
  if (t.rows == 0) return;
  __syncthreads();                                       // the lists are read, or written: red takes their place
  const int e = t.e, rows = t.rows;
  const int64_t m = GATED ? 2 * a.d : a.d, o0 = (int64_t)blockIdx.x * (GATED ? 16 : 32);
  // column of h and packed row of output b, li
  auto column = [&](int b, int l) { return o0 + (GATED ? 0 : 16 * b) + l; };
  int64_t orow[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) orow[b] = e * m + min(column(b, li), a.d - 1) + (GATED ? b * a.d : 0);
  const MvRows<OB> w(a.up.qw, a.up.scales, a.up.zeros, orow, a.n, a.group, BITS);
  ex_f32x4_t tot[OB];
#pragma unroll
  for (int b = 0; b < OB; ++b) tot[b] = (ex_f32x4_t){0.f, 0.f, 0.f, 0.f};
  mv_sum<BITS, WIDE, OB, 1, TILE>(w, a.n, a.group, wave, WAVES, rows, 0, lds_addr(smem[wave]),
                                  mv_vec(a.up.scales, a.up.zeros, a.n, a.group),
                                  [&](int r) { return a.X + (int64_t)(list[r] / a.k) * a.ldx; }, tot);
#pragma unroll
  for (int b = 0; b < OB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh.red[wave][b][r][lane] = tot[b][r];
  __syncthreads();
  for (int i = threadIdx.x; i < (GATED ? 1 : OB) * 256; i += 64 * WAVES) {
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
    uint16_t* out = a.H + (int64_t)list[row] * a.d + c;
    for (int q = 0; q < a.pieces; ++q) {                 // what a piece leaves is exact
      const uint32_t p = ex_pack2(h, 0.f);
      out[q * a.plane] = (uint16_t)p;
      h -= __uint_as_float(p << 16);
    }
  }
}

template <int BITS, bool WIDE, int NP, int TILE, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 4)
k_layer_down(LayerArgs a) {
  // the tiles, and the slots' places (0xFFFF: none) and back
  __shared__ uint16_t te[kLyMax], trows[kLyMax], tfirst[kLyMax], slot[kLyMax], place[kLyMax];
  __shared__ __align__(16) uint8_t smem[WAVES][MvWave<BITS, WIDE, 1, NP, TILE>::BYTES];
  extern __shared__ float part[];                        // [part of K][place][column]
  __shared__ float weight[kLyMax];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  int tiles, places;
  // what the end needs of memory: asked for now
  for (int i = tid; i < a.slots; i += 64 * WAVES) weight[i] = a.w ? a.w[i] : 1.f;
  auto residual = [&](int i) {
    const int64_t at = (int64_t)(i >> 4) * a.ldr + o0 + (i & 15);
    if (!a.res || i >= a.T * 16 || o0 + (i & 15) >= a.n) return 0.f;
    return a.res_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.res)[at] << 16)
                      : static_cast<const float*>(a.res)[at];
  };
  const float first_res = residual(tid);
  if (a.T == 1) {
    tiles = places = a.k;
    for (int i = tid; i < a.k; i += 64 * WAVES) {
      const int id = a.ids[i];
      const bool ok = id >= 0 && id < a.E;
      te[i] = (uint16_t)(ok ? id : 0);
      trows[i] = ok;
      tfirst[i] = slot[i] = (uint16_t)i;
      place[i] = (uint16_t)(ok ? i : 0xFFFF);
    }
  } else {
    const LyTable* table = static_cast<const LyTable*>(a.table);
    tiles = table->tiles;
    places = table->places;
    for (int i = tid; i < a.slots; i += 64 * WAVES) place[i] = 0xFFFF;
    __syncthreads();
    for (int i = tid; i < tiles * TILE; i += 64 * WAVES) {
      const LyTile& t = table->tile[i / TILE];
      const int r = i % TILE;
      if (r == 0) {
        te[i / TILE] = (uint16_t)t.e;
        trows[i / TILE] = (uint16_t)t.rows;
        tfirst[i / TILE] = (uint16_t)t.first;
      }
      if (r < t.rows) {
        slot[t.first + r] = t.slot[r];
        place[t.slot[r]] = (uint16_t)(t.first + r);
      }
    }
  }
  __syncthreads();
  const int kp = tiles >= WAVES || tiles == 0 ? 1 : WAVES / tiles;
  const bool vec = mv_vec(a.down.scales, a.down.zeros, a.d, a.group);
  for (int i = wave; i < tiles * kp; i += WAVES) {
    const int tile = i / kp, p = i - tile * kp;
    const int e = te[tile], first = tfirst[tile], rows = trows[tile];
    if (rows == 0) continue;
    const int64_t orow[1] = {(int64_t)e * a.n + min(o0 + li, a.n - 1)};
    const MvRows<1> w(a.down.qw, a.down.scales, a.down.zeros, orow, a.d, a.group, BITS);
    ex_f32x4_t tot[1] = {{0.f, 0.f, 0.f, 0.f}};
    mv_sum<BITS, WIDE, 1, NP, TILE>(w, a.d, a.group, p, kp, rows, a.plane, lds_addr(smem[wave]), vec,
                                    [&](int r) { return a.H + (int64_t)slot[first + r] * a.d; }, tot);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * (lane >> 4) + r;
      if (row < rows) part[(p * places + first + row) * 16 + li] = tot[0][r];
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += 64 * WAVES) {
    const int t = i >> 4, c = i & 15;
    const int64_t o = o0 + c;
    if (o >= a.n) continue;
    float y = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int s = t * a.k + j, at = place[s];
      if (at == 0xFFFF) continue;
      float v = 0.f;
      for (int p = 0; p < kp; ++p) v += part[(p * places + at) * 16 + c];
      if (a.b2) v += a.b2[a.ids[t * a.ldi + j] * a.n + o];
      y = fmaf(weight[s], v, y);
    }
    y += i == tid ? first_res : residual(i);
    store_out(a.Y, a.y_bf16, t * a.ldy + o, y);
  }
}

// ---------------------------------------------------------------- host
// Slots of a tile. Three pieces of h take three times the LDS.
static int layer_tile(int64_t T, int y_bf16) { return !y_bf16 || T <= 4 ? 4 : 8; }
static int layer_pieces(int y_bf16) { return y_bf16 ? 1 : 3; }
static int64_t layer_tiles(int64_t T, int64_t slots, int64_t E, int y_bf16) {
  return T == 1 ? slots : std::min(slots, ceil_div(slots, layer_tile(T, y_bf16)) + E - 1);
}
static size_t table_bytes(int64_t T, int64_t slots, int64_t E, int y_bf16) {
  return T == 1 ? 0 : (offsetof(LyTable, tile) + layer_tiles(T, slots, E, y_bf16) * sizeof(LyTile) + 255) / 256 * 256;
}
size_t layer_workspace(int64_t T, int64_t k, int64_t E, int64_t d, int y_bf16) {
  return table_bytes(T, T * k, E, y_bf16) + ((size_t)layer_pieces(y_bf16) * T * k * d * sizeof(uint16_t) + 255) / 256 * 256;
}

template <int BITS, bool WIDE, int NP, int TILE, int WAVES>
static void down_go(hipStream_t s, const LayerArgs& a) {
  // K is in WAVES / tiles parts while the tiles are fewer than the waves: up to WAVES times TILE places
  const size_t lds = std::max<size_t>(a.slots, (size_t)std::min(a.slots, TILE) * WAVES) * 64;
  hipLaunchKernelGGL((k_layer_down<BITS, WIDE, NP, TILE, WAVES>), dim3((unsigned)ceil_div(a.n, 16)),
                     dim3(64 * WAVES), lds, s, a);
}
template <int BITS, bool WIDE, int NP, int TILE>
static void down_waves(hipStream_t s, const LayerArgs& a) {
  // LDS holds 16 waves' share beside the results of 512 slots
  constexpr bool BIG = MvWave<BITS, WIDE, 1, NP, TILE>::BYTES <= 6144;
  if constexpr (BIG) {
    if (a.slots <= 512) return down_go<BITS, WIDE, NP, TILE, 16>(s, a);
  }
  down_go<BITS, WIDE, NP, TILE, 8>(s, a);
}

template <int BITS, bool WIDE>
static void ly_go(hipStream_t s, const LayerArgs& a) {
  const dim3 up((unsigned)ceil_div(a.d, a.gated ? 16 : 32), (unsigned)layer_tiles(a.T, a.slots, a.E, a.y_bf16)), block(256);
  const bool four = layer_tile(a.T, a.y_bf16) == 4;
  if (a.gated && four) hipLaunchKernelGGL((k_layer_up<BITS, WIDE, true, 4>), up, block, 0, s, a);
  else if (a.gated) hipLaunchKernelGGL((k_layer_up<BITS, WIDE, true, 8>), up, block, 0, s, a);
  else if (four) hipLaunchKernelGGL((k_layer_up<BITS, WIDE, false, 4>), up, block, 0, s, a);
  else hipLaunchKernelGGL((k_layer_up<BITS, WIDE, false, 8>), up, block, 0, s, a);
  if (!a.y_bf16) down_waves<BITS, WIDE, 3, 4>(s, a);
  else if (four) down_waves<BITS, WIDE, 1, 4>(s, a);
  else down_waves<BITS, WIDE, 1, 8>(s, a);
}

template <int BITS>
static void ly_bits(hipStream_t s, const LayerArgs& a) {
  if (a.group % 128 == 0) ly_go<BITS, true>(s, a);
  else ly_go<BITS, false>(s, a);
}

hipError_t launch_layer(hipStream_t s, const LayerArgs& args) {
  LayerArgs a = args;
  a.table = a.ws;
  a.H = reinterpret_cast<uint16_t*>(static_cast<char*>(a.ws) + table_bytes(a.T, a.slots, a.E, a.y_bf16));
  a.pieces = layer_pieces(a.y_bf16);
  a.plane = (int64_t)a.slots * a.d;
  if (a.bits == 2) ly_bits<2>(s, a);
  else if (a.bits == 3) ly_bits<3>(s, a);
  else ly_bits<4>(s, a);
  return hipGetLastError();
}

}  // namespace gq

// Grouped matrix-matrix products (gfx950, wave64, MFMA, fp32 or int32
// accumulation):
//   NT  y[p][n]     = sum_k x[row(p)][k] w[e][n][k]   (bf16, or int8 codes)
//   NN  dx[p][k]    = sum_n dy[p][n] w[e][n][k]
//   TN  dw[e][n][k] = sum_p dy[p][n] x[row(p)][k]
// over the ragged groups of rows of each expert.
//
// One 8-wave workgroup computes one output tile of up to 256 x 256 over the
// whole reduction.  Operands travel straight from global memory into LDS
// (16 bytes a lane, whole cache lines), steps of 64 reduction elements (128 of
// int8) ahead of the MFMAs.  An operand whose reduction runs along memory (NT
// both, NN the rows dy) is staged as [rows][128 bytes] and read as it lies;
// one whose reduction runs across rows (NN the weights, TN both) is staged as
// [64 rows][256 bytes] and read with the transposing LDS read, so no operand is
// ever transposed in memory.
//
// Which rows a workgroup has comes from the group offsets on the device: each
// wave scans them itself (a few loads and a wave scan) instead of waiting for
// a map made by a launch of its own.
//
// Large tiles are bound by the K loop: 16384 rows, 4 experts of 4096 x 4096:
// 451 us = 1.22 PFLOP/s (NT), 448 us (NN), 430 us = 1.28 (TN); int8 8192^3 2.4 to
// 2.6 POP/s (against 1.38 PFLOP/s and 2.0 POP/s of library products here).  Its
// clusters alone, without transfers, run at 1.65 (NT) to 2.0 PFLOP/s (TN), the
// transfers and LDS reads alone at the time of 1.33 to 1.6: what the two cost
// each other is what is left.  Many small experts are bound by the stream of
// the weights (4096 tokens x 8 over 256 experts of 1024 x 2048: 220 us = 5.3 TB/s
// of weights, tokens and results, 1158 MB), and weight gradients over short
// groups by their results, which nothing overlaps with the next tile's loads
// (the same rows: 395 us for 1.07 GB in bf16, 560 us for 2.15 GB in fp32).
// Tiles of one group that follow each other in a workgroup overlap the two (4096 x
// 16384, NT in us: K 256 76 -> 52, 1024 132 -> 120, 2048 224 -> 211); where all tiles
// run at a time they are low ones (ops_tile.h).
#include "ops_tile.h"

namespace moe {
namespace {

// Row-tiled products (NT, NN).
template <OpKind KIND, bool I8, int GX>
__global__ __launch_bounds__(512, 1) void k_op_rows(TileArgs p) {
  __shared__ u32x4_t lds[10 * HU];  // 160 KB
  row_tile<KIND, I8, GX>(p, lds);
}
template <OpKind KIND>
__global__ __launch_bounds__(512, 1) void k_op_rows_chain(TileArgs p) {
  __shared__ u32x4_t lds[10 * HU];
  row_chain<KIND>(p, lds);
}

// Weight gradients (TN).
template <int GX>
__global__ __launch_bounds__(512, 1) void k_op_wgrad(TileArgs p) {
  __shared__ u32x4_t lds[10 * HU];
  wgrad_tile<GX, StoreEpi, false>(p, blockIdx.x, lds);
}
// Of one matrix, whose units all take the same time: 32 workgroups of an XCD take its units in turn.
__global__ __launch_bounds__(512, 1) void k_op_wgrad_chain(TileArgs p) {
  __shared__ u32x4_t lds[10 * HU];
  int unit = blockIdx.x;
  TileJob t;
  if (wgrad_unit<false>(p, unit, &t) < 0) return;
  tile_product<OP_TN, false, 2, 2, GX_ROWS, false>(p, t, lds, nullptr, StoreEpi{},
                                                   chain_next([&](TileJob& t) __attribute__((always_inline)) {
                                                     unit += kChainGroups;
                                                     return wgrad_unit<false>(p, unit, &t) >= 0;
                                                   }));
}

}  // namespace

int64_t op_tile_units(OpKind kind, const Groups& g) {
  const int64_t pn = (g.N + TB - 1) / TB, pk = (g.K + TB - 1) / TB;
  if (kind == OP_TN) return wgrad_units(g, 1);
  return row_tile_units(g, kind == OP_NT ? pn : pk);
}

hipError_t launch_op_tile(OpKind kind, bool i8, const Groups& g, const void* a, const void* b, const Scales& sc,
                          void* out, bool fp32, hipStream_t s) {
  TileArgs t{};
  t.g = g;
  t.a = (const char*)a;
  t.b = (const char*)b;
  t.sc = sc;
  t.out = out;
  t.fp32 = fp32;
  t.nrow = (g.N + TB - 1) / TB;
  t.npan = ((kind == OP_NT ? g.N : g.K) + TB - 1) / TB;
  set_row_tiles(&t);
  const unsigned grid = (unsigned)op_tile_units(kind, g);
  const Launch lc{s, nullptr, nullptr};
  const bool far = rows_far(g, i8 ? 1 : 2);
  const bool chain = !i8 && !g.perm && (kind == OP_TN ? !g.offsets && grid > kChainGroups : takes_chain(g, grid));
  const dim3 gr(chain ? (unsigned)kChainGroups : grid), bl(512);
  if (kind == OP_TN) {
    if (chain) return launch(lc, k_op_wgrad_chain, gr, bl, t);
    if (!g.perm) return launch(lc, k_op_wgrad<GX_ROWS>, gr, bl, t);
    return far ? launch(lc, k_op_wgrad<GX_FAR>, gr, bl, t) : launch(lc, k_op_wgrad<GX_INDEX>, gr, bl, t);
  }
  if (kind == OP_NN)
    return chain ? launch(lc, k_op_rows_chain<OP_NN>, gr, bl, t)
                 : launch(lc, k_op_rows<OP_NN, false, GX_ROWS>, gr, bl, t);
  if (i8)
    return far ? launch(lc, k_op_rows<OP_NT, true, GX_FAR>, gr, bl, t)
               : launch(lc, k_op_rows<OP_NT, true, GX_ROWS>, gr, bl, t);
  if (chain) return launch(lc, k_op_rows_chain<OP_NT>, gr, bl, t);
  return far ? launch(lc, k_op_rows<OP_NT, false, GX_FAR>, gr, bl, t)
             : launch(lc, k_op_rows<OP_NT, false, GX_ROWS>, gr, bl, t);
}

}  // namespace moe

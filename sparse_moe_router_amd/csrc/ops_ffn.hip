// The products behind k_gated_grad in the backward pass of a gated feed-forward
// block (gfx950):
//   dx = d_pre W_gu,  dW_gu = d_pre^T x[row],  dW_d = dy^T h
// in one launch: none needs another's result, and the tiles of the later ones
// fill the compute units that the last tiles of the earlier ones leave (in three
// launches each waits for the slowest tile before it).  The rows' gradient comes
// first, whose tiles are the longest of most blocks.  Weight gradients with few
// tiles (few experts) are cut along their rows; the parts are added in a fixed
// order by a second launch.
//
// 8192 x 2 rows over 16 experts of 1024 x 2048: 352 to 429 us = 0.80 to 0.98 PFLOP/s (matrix units busy 50% at
// 1.8 GHz: tiles of 16 and 32 steps, whose prologue and epilogue nothing overlaps).  701 x 4 rows over 64
// skewed experts of 512 x 1032: 126 us, tiles of a few steps, each with up to 128 KB of results to store.
#include "ops_sum.h"
#include "ops_tile.h"

namespace moe {
namespace {

struct FfnTiles {
  TileArgs dx, gu, down;
  int dx_units, gu_units;  // multiples of 8: a workgroup's XCD is that of its unit
};

template <int GX>
__global__ __launch_bounds__(512, 1) void k_ffn_products(FfnTiles a) {
  __shared__ u32x4_t lds[10 * HU];
  int b = blockIdx.x;
  if (b < a.dx_units) {
    row_tile<OP_NN, false, GX_ROWS>(a.dx, lds);
    return;
  }
  b -= a.dx_units;
  if (b < a.gu_units)
    wgrad_tile<GX>(a.gu, b, lds);
  else
    wgrad_tile<GX_ROWS>(a.down, b - a.gu_units, lds);
}

Groups gu_groups(const FfnArgs& a) {
  Groups g = a.g;
  g.ldy = a.ld_dpre;
  return g;
}
Groups down_groups(const FfnArgs& a) {
  return Groups{a.g.rows, a.g.rows, a.ld_h, a.ld_dy, a.g.E, a.H, a.I, 1, a.g.offsets, nullptr};
}
Groups dx_groups(const FfnArgs& a) {
  Groups g = gu_groups(a);
  g.ldx = a.ld_dx;
  g.perm = nullptr;
  return g;
}
// dx's tiles are low ones where the weight gradients' leave them the room.
int64_t weight_units(const FfnArgs& a, int parts) { return wgrad_units(a.g, parts) + wgrad_units(down_groups(a), parts); }
int dx_room(const FfnArgs& a, int parts) {
  const int64_t weights = weight_units(a, parts);
  return weights < kChainGroups ? (int)(kChainGroups - weights) : 0;
}
int64_t dx_units(const FfnArgs& a, int parts) { return row_tile_units(a.g, (a.g.K + TB - 1) / TB, dx_room(a, parts)); }

int64_t tiles_of(int64_t rows, int64_t columns) { return (rows + TB - 1) / TB * ((columns + TB - 1) / TB); }

TileArgs weight_tiles(const Groups& g, const void* dy, const void* x, void* out, bool fp32, int splits) {
  TileArgs t{};
  t.g = g;
  t.a = (const char*)dy;
  t.b = (const char*)x;
  t.out = out;
  t.fp32 = fp32;
  t.nrow = (g.N + TB - 1) / TB;
  t.npan = (g.K + TB - 1) / TB;
  t.splits = splits;
  return t;
}

}  // namespace

// Parts of the weight gradients: those with which the launch takes least (launch_steps; a group of average
// size), of at least four steps of 64 rows.  Blocks of K = H, I and rows over E experts in us, by parts:
// 1024, 512, 4096 over 1: 1 part 121, 4 84, 10 97; 2048, 1024, 4096 over 1: 1 148, 2 170, 4 161; 1024, 512,
// 8192 over 4: 1 92, 2 115, 4 114; 1024, 512, 16384 over 1: 1 338, 4 157, 8 139, 16 171.
int ffn_splits(const FfnArgs& a) {
  const int64_t E = a.g.E, most = a.g.rows / (256 * E);
  const int64_t units = E * tiles_of(a.g.N, a.g.K) + E * tiles_of(a.H, a.I), dx = tiles_of(a.g.rows, a.g.K);
  const int64_t size = E * ((int64_t)a.g.N * a.g.K + (int64_t)a.H * a.I) * 4;
  int best = 1;
  int64_t least = 0;
  for (int n = 1; n <= (most > 1 ? most : 1) && (n == 1 || n * units <= kMostTiles); n = next_parts(n)) {
    const int64_t t = launch_steps(dx, a.g.N / 64 + kTileSteps, units * n, a.g.rows / (64 * E * n) + kTileSteps) +
                      (n > 1 ? kLaunchSteps + 2 * n * size / kStepBytes : 0);
    if (n == 1 || t < least) best = n, least = t;
  }
  return best;
}
size_t ffn_split_bytes(const FfnArgs& a) {
  const int n = ffn_splits(a);
  return n > 1 ? (size_t)n * a.g.E * ((size_t)a.g.N * a.g.K + (size_t)a.H * a.I) * 4 : 0;
}
int64_t ffn_units(const FfnArgs& a) {
  const int n = ffn_splits(a);
  return dx_units(a, n) + weight_units(a, n);
}

hipError_t launch_ffn_products(const FfnArgs& a, float* part, hipStream_t s) {
  const int n = ffn_splits(a);
  const int64_t gu_size = (int64_t)a.g.E * a.g.N * a.g.K, down_size = (int64_t)a.g.E * a.H * a.I;
  float* down_part = part + n * gu_size;
  FfnTiles f{};
  f.dx.g = dx_groups(a);
  f.dx.a = (const char*)a.d_pre;
  f.dx.b = (const char*)a.w_gate_up;
  f.dx.out = a.dx;
  f.dx.npan = (a.g.K + TB - 1) / TB;
  set_row_tiles(&f.dx, dx_room(a, n));
  f.gu = weight_tiles(gu_groups(a), a.d_pre, a.x, n > 1 ? part : a.dw_gate_up, n > 1 || a.dw32, n);
  f.down = weight_tiles(down_groups(a), a.dy, a.h, n > 1 ? down_part : a.dw_down, n > 1 || a.dw32, n);
  f.dx_units = a.g.rows > 0 ? (int)dx_units(a, n) : 0;
  f.gu_units = (int)wgrad_units(a.g, n);
  const dim3 grid((unsigned)(f.dx_units + f.gu_units + wgrad_units(f.down.g, n))), block(512);
  const Launch lc{s, nullptr, nullptr};
  const hipError_t e = !a.g.perm          ? launch(lc, k_ffn_products<GX_ROWS>, grid, block, f)
                       : rows_far(a.g, 2) ? launch(lc, k_ffn_products<GX_FAR>, grid, block, f)
                                          : launch(lc, k_ffn_products<GX_INDEX>, grid, block, f);
  if (e != hipSuccess || n == 1) return e;
  return launch_sum_parts(n, SumOf{part, gu_size, a.dw_gate_up}, SumOf{down_part, down_size, a.dw_down}, nullptr, a.dw32, s);
}

}  // namespace moe

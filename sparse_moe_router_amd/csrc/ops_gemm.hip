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
#include <type_traits>

#include "ops_internal.h"

namespace moe {
namespace {

constexpr int TB = kOpTile;  // tile edge
constexpr int HU = 1024;     // 16-byte units of a half-tile stage: 128 rows x 128 bytes, or 64 x 256 (16 KB)
constexpr int GI = 8192;     // rows of x whose indexes the weight gradient holds in LDS at a time

typedef __attribute__((__vector_size__(4 * sizeof(int16_t)))) int16_t i16x4_t;

struct TileArgs {
  Groups g;
  const char* a;
  const char* b;
  Scales sc;
  void* out;
  int fp32;
  int npan;    // tiles along the second output dimension
  int nrow;    // TN: tiles along n
};

// Transfers go through range-checked buffer descriptors: a lane whose offset
// lies past the descriptor's range gets zeros in LDS, so rows, columns and
// steps past an operand's end need no branches, and a transfer needs one
// register of address (64-bit addresses took twice the issue time beside the
// other group's MFMAs: a memory part with two transfers 400 cycles).
// The transfers are issued by asm statements without outputs: the loop below
// counts them itself, and the compiler, which tells apart at most eight
// destinations of transfers in flight, would wait for all of them at every LDS
// read of a ninth.  A wait of the compiler's own for another load counts later
// transfers as if they were not there and so only waits longer.  m0 is the LDS
// address of a transfer; the wait states cover a scalar operand that a vector
// instruction has just written.
struct window_t {
  u32x4_t d;  // buffer descriptor: base, stride 0, range in bytes, raw format
};
constexpr uint32_t kOut = 0x80000000u;  // an offset past every range
// (A scalar offset must stay below the window's range, against whose rest lanes are checked.)
constexpr int64_t kRange = 0x7FFFFFFF;  // largest range of a descriptor
__device__ __forceinline__ window_t window(const char* base, int64_t bytes) {
  const uint32_t n = bytes < 0 ? 0u : bytes > kRange ? (uint32_t)kRange : (uint32_t)bytes;
  const uint64_t b = (uint64_t)base;
  return window_t{u32x4_t{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, n, 0x00020000u}};
}
// The compiler warns of a clobber of m0, which it allocates to nothing; it does honour it where it
// keeps a value of m0 of its own.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// lane i of the wave writes the 16 bytes at offset off + step_off of the window to LDS address dst + 16 i
__device__ __forceinline__ void dma(window_t w, uint32_t off, int step_off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(dst), "v"(off),
               "s"(w.d), "s"(step_off)
               : "memory", "m0");
}
// the same with the non-temporal hint: weights that one workgroup alone reads leave the caches to the
// rows (4096 tokens x 8 over 256 experts 249 -> 226 us; weights that several tiles read lose by it,
// and so do rows off the cache lines, whose lines two steps share: 2501 x 4 over 60 skewed experts
// of 2832-byte rows 53 -> 83 us)
__device__ __forceinline__ void dma_once(window_t w, uint32_t off, int step_off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(dst), "v"(off),
               "s"(w.d), "s"(step_off)
               : "memory", "m0");
}
// by 64-bit addresses, for rows of x that lie more than a descriptor's range apart
__device__ __align__(16) const uint32_t kZero[4] = {0, 0, 0, 0};
__device__ __forceinline__ void dma64(const char* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src)
               : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return ((int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
// waits until at most N of the wave's transfers are in flight and its LDS reads are done
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
}
__device__ __forceinline__ void bar() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The row tile and panel of a workgroup: group, first row, rows.  A group of c
// rows has ceil(c / 256) tiles, all of 256 rows but the last.
struct RowTile {
  int e;  // -1: none
  int64_t p0;
  int rows;
  int panel;
  int once;  // the group's only tile, of weight rows in whole cache lines
};

// One group: the units (tile, panel) are cut into eight equal runs, one for
// each XCD, and within a run into blocks of four tiles, panel by panel: the 32
// workgroups that an XCD runs at a time then read about as many tiles' rows as
// panels' weights (int8 4096 x 8192 x 4096: 126 -> 119 us).
__device__ __forceinline__ RowTile find_tile_dense(const Groups& g, int xcd, int64_t local, int npan, bool aligned) {
  constexpr int SG = 4;
  const int64_t total = (g.rows + TB - 1) / TB;
  const int64_t run = (total * npan + 7) / 8, unit = xcd * run + local;
  if (local >= run || unit >= total * npan) return RowTile{-1, 0, 0, 0, 0};
  const int64_t sg = unit / (SG * npan), sr = unit - sg * SG * npan;
  const int64_t height = total - sg * SG < SG ? total - sg * SG : SG;
  const int64_t p0 = (sg * SG + sr % height) * TB;
  return RowTile{0, p0, (int)(g.rows - p0 < TB ? g.rows - p0 : TB), (int)(sr / height), total == 1 && aligned};
}

// Groups: the tiles in three classes, the tallest first, so that the short
// ones fill the end of the launch; of each class, in group order, one eighth
// goes to each XCD: an expert's tiles and a tile's panels then share its
// weights and rows in one L2, and the XCDs stream from distant experts.
// Against tiles dealt to the XCDs one by one, and against one run for each XCD
// in group order: 8192 tokens x 2 over 16 experts 122, 136 and 148 us; 4096 x
// 8 over 256 experts 241, 304, 241; 2501 x 4 over 60 skewed ones 51, 52, 60.
// With fewer than 64 tiles single panels are dealt out.
// Lane l scans the groups [l * per, (l + 1) * per); every wave does the same scan.
constexpr int kDealTiles = 64;
// The ranges of groups e .. e + 3, empty from group `end` or E on; their loads are in flight together.
__device__ __forceinline__ void four_ranges(const Groups& g, int e, int end, Range (&r)[4]) {
  int32_t v[5];
  end = end < g.E ? end : g.E;
#pragma unroll
  for (int u = 0; u < 5; ++u) v[u] = g.offsets[e + u < end ? e + u : end];
#pragma unroll
  for (int u = 0; u < 4; ++u) r[u] = limited(g, v[u], v[u + 1]);
}
__device__ __forceinline__ int tile_class(int rest) { return rest > 192 ? 0 : rest > 64 ? 1 : 2; }
__device__ __forceinline__ RowTile find_tile(const Groups& g, int xcd, int64_t local, int npan, bool aligned) {
  if (!g.offsets) return find_tile_dense(g, xcd, local, npan, aligned);
  const int lane = threadIdx.x & 63, per = (g.E + 63) / 64;
  // tiles of this lane's groups in each class: bits 0..31, 32..47, 48..63
  uint64_t mine = 0;
  for (int j = 0; j < per; j += 4) {
    Range r[4];
    four_ranges(g, lane * per + j, lane * per + per, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t c = (uint32_t)r[u].size(), rest = c % TB;
      mine += c / TB;
      if (rest > 0) mine += (uint64_t)1 << (tile_class(rest) == 0 ? 0 : 16 + 16 * tile_class(rest));
    }
  }
  uint64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  const uint64_t all = __shfl(incl, 63, 64);
  const int64_t n0 = (uint32_t)all, n1 = (all >> 32) & 0xFFFF, total = n0 + n1 + (int64_t)(all >> 48);
  const int64_t n2 = (int64_t)(all >> 48);
  int64_t i;  // place in the class
  int cl, panel;
  if (total >= kDealTiles) {
    i = local / npan;
    panel = (int)(local % npan);
    const int64_t a0 = n0 * xcd / 8, m0 = n0 * (xcd + 1) / 8 - a0;
    const int64_t a1 = n1 * xcd / 8, m1 = n1 * (xcd + 1) / 8 - a1;
    const int64_t a2 = n2 * xcd / 8, m2 = n2 * (xcd + 1) / 8 - a2;
    if (i < m0) {
      cl = 0, i += a0;
    } else if (i < m0 + m1) {
      cl = 1, i += a1 - m0;
    } else if (i < m0 + m1 + m2) {
      cl = 2, i += a2 - m0 - m1;
    } else {
      return RowTile{-1, 0, 0, 0, 0};
    }
  } else {
    i = (local * 8 + xcd) / npan;
    panel = (int)((local * 8 + xcd) % npan);
    if (i >= total) return RowTile{-1, 0, 0, 0, 0};
    cl = i < n0 ? 0 : i < n0 + n1 ? 1 : 2;
    i -= cl == 0 ? 0 : cl == 1 ? n0 : n0 + n1;
  }
  const int shift = cl == 0 ? 0 : 16 + 16 * cl;
  const uint64_t mask = cl == 0 ? 0xFFFFFFFFu : 0xFFFFu;
  const int src = __builtin_ctzll(__ballot((int64_t)((incl >> shift) & mask) > i));
  i -= (int64_t)((__shfl(incl - mine, src, 64) >> shift) & mask);
  for (int j = 0; j < per; j += 4) {
    Range r[4];
    four_ranges(g, src * per + j, src * per + per, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t full = r[u].size() / TB;
      const int rest = (int)(r[u].size() % TB);
      const int64_t here = (cl == 0 ? full : 0) + (rest > 0 && tile_class(rest) == cl);
      if (i < here) {
        const int64_t k = cl == 0 ? i : full;  // the tile's place in its group
        return RowTile{src * per + j + u, r[u].lo + k * TB, k < full ? TB : rest, panel, r[u].size() <= TB && aligned};
      }
      i -= here;
    }
  }
  return RowTile{-1, 0, 0, 0, 0};  // not reached: the lane's count says that one of its groups holds the tile
}

// One output tile, eight waves: wm = wave / 4, wn = wave % 4.  The tile's rows
// come in two halves of 64 RB0 and 64 RB1 rows (RB1 may be 0), its 256 columns
// in two halves of 128; wave (wm, wn) has rows [32 RB wm, +32 RB) of each row
// half and 32 columns of each column half: four quadrants.
//
// A K-step runs as one cluster per quadrant: a memory part (LDS reads of the
// quadrant's operands, transfers for a later step) and a multiply part, each
// closed by a barrier.  The waves wm = 1 run one barrier behind those with
// wm = 0, the two waves of a SIMD being one of each: while one multiplies the
// other reads, so the matrix unit, the LDS and the transfers work at the same
// time without competing for the SIMD's issue.
//
// Stages hold whole steps; with both row halves there are two of them (128 KB),
// with one half three (144 KB), with a quarter four (160 KB).  A half-tile is
// refilled as soon as both groups have read it (the second group reads one
// barrier later), so every transfer has more than a step's time to land; every
// wave waits for its own part (a count of the transfers issued after it) at a
// barrier before the first group reads it.  Transfers are never conditional:
// those of steps past the end fetch zeros, or the last step again, into a
// stage nobody reads.
//
// GX: how rows of x are found: GX_ROWS in order (NT: or gathered), GX_INDEX
// gathered (TN), GX_FAR gathered, by 64-bit addresses.
enum { GX_ROWS = 0, GX_INDEX = 1, GX_FAR = 2 };
// ONCE: this tile alone reads its panel of weights, whose rows are whole cache
// lines (a template, because a branch at each transfer costs tiles bound by
// the matrix units 6%).
template <OpKind KIND, bool I8, int RB0, int RB1, int GX, bool ONCE>
__device__ __forceinline__ void tile_product(const TileArgs& p, int e, int64_t p0, int rows, int64_t len, int r0t,
                                             int panel, u32x4_t* lds, int32_t* gidx) {
  constexpr bool AT = KIND == OP_TN, BT = KIND != OP_NT;  // operand reduces across its rows
  constexpr int ES = I8 ? 1 : 2;                          // bytes an element
  constexpr int ST = RB1 > 0 ? 2 : RB0 == 2 ? 3 : 4;      // stages
  constexpr int RBM = RB0 > RB1 ? RB0 : RB1;
  static_assert(!AT || (RB0 == 2 && RB1 == 2), "weight gradients have full tiles");
  typedef typename std::conditional<I8, i32x16_t, f32x16_t>::type acc_t;
  const Groups& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 3, wm = wave >> 2;

  // ---- LDS of a stage: the two column halves, then the row halves
  constexpr int STAGE = 2 * HU + (RB0 + RB1) * HU / 2;
  static_assert(ST * STAGE <= 10 * HU, "160 KB");
  // its LDS address, 0 where the array is the kernel's first
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) u32x4_t*)lds;
  auto sb = [&](int j, int st) { return lds + st * STAGE + j * HU; };
  auto sa = [&](int h, int st) { return lds + st * STAGE + 2 * HU + (h ? RB0 * HU / 2 : 0); };

  const int ncols = KIND == OP_NT ? g.N : g.K;
  const int c0 = panel * TB;
  constexpr int BKE = I8 ? 128 : 64;  // reduction elements of a step
  // first column of the tile's 32-column block wn of column half j.  Weights read along memory: a
  // wave's two blocks side by side, so that it writes whole cache lines; across: halves of 128.
  auto col_of = [&](int j, int blk) { return BT ? 128 * j + 32 * blk : 64 * blk + 32 * j; };

  // ---- transfers.  Along-memory operand: a transfer fills 8 stage rows of 128
  // bytes, lane -> row lane/8, chunk position lane%8, source chunk
  // (lane%8) ^ ((row/2) % 8): 16 consecutive rows' reads then fall on all
  // banks.  Across-rows operand: 4 stage rows of 256 bytes, lane -> row
  // lane/16, position lane%16, source chunk position ^ 4 (row % 4): the four
  // rows a transposing read takes together lie in different 64-byte parts.
  const int lr = lane >> 3;
  constexpr bool G64 = GX == GX_FAR;
  const bool gather = KIND == OP_TN ? GX != GX_ROWS : KIND == OP_NT && g.perm;
  const int64_t lda = KIND == OP_NT ? g.ldx : g.ldy;
  int64_t red = KIND == OP_NT ? g.K : KIND == OP_NN ? g.N : len;  // reduction length (TN: of this chunk)
  int64_t base = p0;                                              // TN: first row of the chunk
  int nsteps = 0, last = 0;  // steps; reduction elements of the last one
  // window of the first step, and what a step adds to its base (across) or to the offsets (along: 128)
  const char *abase, *bbase;
  int64_t abytes = 0, bbytes = 0;
  const int64_t astep = g.ldy * 128, bstep = (KIND == OP_NN ? (int64_t)g.K : g.ldx) * 128;
  // window of step s of an operand that reduces across its rows: the step's rows that exist
  auto step_window = [&](const char* at, int64_t step, int s, int width) {
    const int n = s < nsteps - 1 ? 64 : s == nsteps - 1 ? last : 0;
    window_t w = window(at + s * step, 0);
    w.d[2] = n > 0 ? (uint32_t)((n - 1) * (int)(step >> 6) + width) : 0u;
    return w;
  };
  uint32_t aoff[2][RBM], boff[2][2];  // a lane's offsets in its window
  bool aend[2][RBM], bend[2][2];      // along: the lane's chunk lies in the last step
  const char* a64[2][RBM];
  auto set_steps = [&]() {
    nsteps = (int)((red + BKE - 1) / BKE);
    last = (int)(red - (int64_t)(nsteps - 1) * BKE);
    if (AT) {
      abase = p.a + base * g.ldy * 2;
    } else {
      abase = p.a + (gather ? 0 : p0 * lda * ES);
      abytes = (((gather ? g.x_rows : rows) - 1) * lda + red) * ES;
    }
    if (KIND == OP_NT) {
      bbase = p.b + ((int64_t)e * g.N + c0) * g.K * ES;
      bbytes = (int64_t)(g.N - c0) * g.K * ES;
    } else if (KIND == OP_NN) {
      bbase = p.b + (int64_t)e * g.N * g.K * 2;
    } else {
      bbase = p.b + (gather ? 0 : base * g.ldx * 2);
      bbytes = ((g.x_rows - 1) * g.ldx + g.K) * 2;  // gathered
    }
  };
  auto set_a = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RBM; ++i) {
        if (i >= (h ? RB1 : RB0)) continue;
        if (!AT) {
          const int srow = (wave * (h ? RB1 : RB0) + i) * 8 + lr, row = (h ? 64 * RB0 : 0) + srow;
          const int q = (lane & 7) ^ ((srow >> 1) & 7);
          aend[h][i] = q * (16 / ES) < last;
          if (gather) {
            const int64_t t = row < rows ? source_row(g, p0 + row) : -1;
            if (G64)
              a64[h][i] = t < 0 ? nullptr : p.a + t * lda * ES + q * 16;
            else
              aoff[h][i] = t < 0 ? kOut : (uint32_t)(t * lda * ES + q * 16);
          } else {
            aoff[h][i] = (uint32_t)(row * lda * ES + q * 16);  // rows past the tile's lie past the range
          }
        } else {
          const int row = (wave * 2 + i) * 4 + (lane >> 4);
          const int col = r0t * TB + 128 * h + ((lane & 15) ^ (4 * (row & 3))) * 8;
          aoff[h][i] = col >= g.N ? kOut : (uint32_t)((row * g.ldy + col) * 2);
        }
      }
  };
  auto set_b = [&]() {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!BT) {
          const int srow = (wave * 2 + i) * 8 + lr;
          const int q = (lane & 7) ^ ((srow >> 1) & 7);
          bend[j][i] = q * (16 / ES) < last;
          // rows past N lie past the range
          boff[j][i] = (uint32_t)((col_of(j, srow >> 5) + (srow & 31)) * g.K * ES + q * 16);
        } else {
          const int row = (wave * 2 + i) * 4 + (lane >> 4);
          const int col = c0 + 128 * j + ((lane & 15) ^ (4 * (row & 3))) * 8;
          const int64_t ld = KIND == OP_NN ? (int64_t)g.K : gather ? 0 : g.ldx;
          boff[j][i] = col >= g.K ? kOut : (uint32_t)((row * ld + col) * 2);
        }
      }
  };
  auto load_a = [&](int h, int st, int s) {
    const int sc = s < nsteps ? s : nsteps - 1;
#pragma unroll
    for (int i = 0; i < RBM; ++i) {
      if (i >= (h ? RB1 : RB0)) continue;
      const uint32_t dst = lds0 + (sa(h, st) - lds + (wave * (h ? RB1 : RB0) + i) * 64) * 16;
      if (AT) {
        dma(step_window(abase, astep, s, 2 * g.N), aoff[h][i], 0, dst);
      } else if (G64 && gather) {
        dma64(a64[h][i] && (s < nsteps - 1 || aend[h][i]) ? a64[h][i] + sc * 128 : (const char*)kZero, dst);
      } else {
        dma(window(abase, abytes), s >= nsteps - 1 && !aend[h][i] ? kOut : aoff[h][i], sc * 128, dst);
      }
    }
  };
  auto load_b = [&](int j, int st, int s) {
    const int sc = s < nsteps ? s : nsteps - 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = lds0 + (sb(j, st) - lds + (wave * 2 + i) * 64) * 16;
      if (!BT) {
        const uint32_t off = s >= nsteps - 1 && !bend[j][i] ? kOut : boff[j][i];
        if (ONCE)
          dma_once(window(bbase, bbytes), off, sc * 128, dst);
        else
          dma(window(bbase, bbytes), off, sc * 128, dst);
      } else if (KIND == OP_TN && gather) {
        // rows past the end have no index: -1
        const int32_t t = gidx[sc * 64 + (wave * 2 + i) * 4 + (lane >> 4)];
        const bool in = t >= 0 && boff[j][i] != kOut;
        if (G64)
          dma64(in ? bbase + (int64_t)t * g.ldx * 2 + boff[j][i] : (const char*)kZero, dst);
        else
          dma(window(bbase, bbytes), in ? (uint32_t)(t * (int)g.ldx * 2) + boff[j][i] : kOut, 0, dst);
      } else if (ONCE) {
        dma_once(step_window(bbase, bstep, s, 2 * g.K), boff[j][i], 0, dst);
      } else {
        dma(step_window(bbase, bstep, s, 2 * g.K), boff[j][i], 0, dst);
      }
    }
  };

  acc_t acc[2][RBM][2];  // [row half][block][column half]
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < RBM; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[h][b][j] = (acc_t){};

  // ---- operand reads: sub-step kk, lane half take the reduction elements
  // 32 half + 8 kk .. +8 of a step (int8: 64 half + 16 kk .. +16) on both operands
  auto read_along = [&](const u32x4_t* st, int row32, int kk) -> u32x4_t {
    return st[(row32 + l32) * 8 + ((4 * half + kk) ^ ((l32 >> 1) & 7))];
  };
  const int ti = lane & 15, tsub = (lane >> 4) & 1;
  auto read_across = [&](const u32x4_t* st, int col32, int kk) -> u32x4_t {
    // two transposing reads of 4 rows each; lane ti of 16 supplies row ti/4, columns 4 (ti%4) .. +4
    const int row = 32 * half + 8 * kk + (ti >> 2);
    const int q = (col32 / 8 + 2 * tsub + ((ti & 3) >> 1)) ^ (4 * (ti >> 2));
    const char* at = (const char*)(st + row * 16 + q) + 8 * (ti & 1);
    const uint64_t lo = __builtin_bit_cast(
        uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)at));
    const uint64_t hi = __builtin_bit_cast(
        uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(at + 4 * 256)));
    return u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  };
  u32x4_t af[RBM][4], bf[2][4];
  auto read_a = [&](int h, int st) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int b = 0; b < RBM; ++b) {
        if (b >= (h ? RB1 : RB0)) continue;
        const int r = 32 * ((h ? RB1 : RB0) * wm + b);
        af[b][kk] = AT ? read_across(sa(h, st), r, kk) : read_along(sa(h, st), r, kk);
      }
  };
  auto read_b = [&](int j, int st) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      bf[j][kk] = BT ? read_across(sb(j, st), 32 * wn, kk) : read_along(sb(j, st), 32 * wn, kk);
  };
  // the multiply part of a cluster, between its two barriers
  auto multiply = [&](int h, int j) {
    bar();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int b = 0; b < RBM; ++b) {
        if (b >= (h ? RB1 : RB0)) continue;
        if constexpr (I8)
          acc[h][b][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, af[b][kk]),
                                                               __builtin_bit_cast(i32x4_t, bf[j][kk]), acc[h][b][j], 0,
                                                               0, 0);
        else
          acc[h][b][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, af[b][kk]),
                                                                 __builtin_bit_cast(bf16x8_t, bf[j][kk]), acc[h][b][j],
                                                                 0, 0, 0);
      }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    bar();
  };

  // One pass over the reduction; weight gradients with gathered rows pass in
  // chunks whose row indexes fit the LDS.
  for (int64_t done = 0; KIND != OP_TN ? done == 0 : done < len; done += GI) {
    if (KIND == OP_TN && gather) {
      red = len - done < GI ? len - done : GI;
      base = p0 + done;
      // up to a whole number of steps, rows past the end as -1
      for (int i = tid; i < (red + 63) / 64 * 64; i += 512) gidx[i] = i < red ? (int32_t)source_row(g, base + i) : -1;
      __syncthreads();
    } else if (done > 0) {
      break;
    }
    set_steps();
    set_b();
    if constexpr (RB1 > 0) {
      // memory parts: 8, 4, 8 and 4 reads of a block, two transfers a wave in each.  The first column
      // half of a step is read in the last part of the step before.
      constexpr int WB = 6 + RB0 + 2 * RB1, WA = 6 + 2 * RB0 + RB1;
      // the columns' transfers are on their way while the rows' indexes are read
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        load_b(0, d, d);
        load_b(1, d, d);
      }
      set_a();
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        load_a(0, d, d);
        load_a(1, d, d);
      }
      wait_vm<RB0 + 2 * RB1>();  // all columns, first row half of step 0
      bar();
      read_b(0, 0);
      // read by every wave before the first memory part refills it
      wait_vm<63>();
      bar();
      if (wm == 1) bar();
      for (int s0 = 0; s0 < nsteps; s0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int s = s0 + u;
          if (s >= nsteps) break;  // uniform
          read_a(0, u);
          load_b(0, u, s + 2);
          wait_vm<WB>();  // second column half of this step
          multiply(0, 0);
          read_b(1, u);
          load_a(0, u, s + 2);
          // second row half of this step; in step 0 fewer transfers come after it than later on
          if (s == 0)
            wait_vm<2 + 2 * RB0 + RB1>();
          else
            wait_vm<WA>();
          multiply(0, 1);
          read_a(1, u);
          load_b(1, u, s + 2);
          wait_vm<WA>();  // first column half of the next step
          multiply(1, 0);
          read_b(0, u ^ 1);
          load_a(1, u, s + 2);
          if (s == 0)  // first row half of the next step
            wait_vm<4 + RB0 + 2 * RB1>();
          else
            wait_vm<WB>();
          multiply(1, 1);
        }
      }
    } else {
      constexpr int W = 2 * (ST - 1) + (ST - 2) * (RB0 + 2);
#pragma unroll
      for (int d = 0; d < ST; ++d) {
        load_b(0, d, d);
        if (d < ST - 1) load_b(1, d, d);
      }
      set_a();
#pragma unroll
      for (int d = 0; d < ST; ++d) load_a(0, d, d);
      wait_vm<(ST - 1) * RB0>();  // all columns, rows of step 0
      bar();
      read_b(0, 0);
      if (wm == 1) bar();
      for (int s0 = 0; s0 < nsteps; s0 += ST) {
#pragma unroll
        for (int u = 0; u < ST; ++u) {
          const int s = s0 + u;
          if (s >= nsteps) break;  // uniform
          read_a(0, u);
          load_b(1, (u + ST - 1) % ST, s + ST - 1);
          // second column half of this step, first halves of the next; in the first steps fewer
          // transfers come after those than later on
          if (s == 0)
            wait_vm<(ST - 2) * RB0 + 2>();
          else if (ST == 4 && s == 1)
            wait_vm<(ST - 2) * RB0 + 6>();
          else
            wait_vm<W>();
          multiply(0, 0);
          read_b(1, u);
          read_b(0, (u + 1) % ST);
          load_a(0, u, s + ST);
          load_b(0, u, s + ST);
          wait_vm<63>();
          multiply(0, 1);
        }
      }
    }
    if (wm == 0) bar();
    // transfers of steps past the end have landed and every wave has read its
    // last operands before the LDS is used again
    wait_vm<0>();
    bar();
  }

  // ---- epilogue.  Block layout: lane -> column lane%32, register r -> row
  // 8 (r/4) + 4 (lane/32) + r%4.
  const int nrows = KIND == OP_TN ? (g.N - r0t * TB < TB ? g.N - r0t * TB : TB) : rows;
  const int64_t ldo = KIND == OP_NT ? g.ldy : KIND == OP_NN ? g.ldx : g.K;
  const int64_t row_base = KIND == OP_TN ? (int64_t)e * g.N + (int64_t)r0t * TB : p0;
  float* s_scale = (float*)lds;  // I8: the rows' scales
  if (I8) {
    if (tid < rows) {
      const int64_t t = source_row(g, p0 + tid);
      s_scale[tid] = t < 0 ? 0.0f : p.sc.x[t];
    }
    __syncthreads();
  }
  float ws[2] = {1.0f, 1.0f}, bi[2] = {0.0f, 0.0f};
  if (I8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = c0 + col_of(j, wn) + l32;
      if (n < ncols) {
        ws[j] = p.sc.w[(int64_t)e * g.N + n];
        if (p.sc.bias) bi[j] = p.sc.bias[n];
      }
    }
  }
  // 32 x 64 results at a time through a part of the LDS of the wave's own, then 16 bytes a lane
  float* stage = (float*)(lds + HU) + wave * (32 * 64);
  auto write = [&](auto type) {
    typedef decltype(type) T;
    constexpr int EC = 16 / sizeof(T);  // results of a 16-byte chunk
    T* st = (T*)stage;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RBM; ++b) {
        if (b >= (h ? RB1 : RB0)) continue;
        const int row0 = (h ? 64 * RB0 : 0) + 32 * ((h ? RB1 : RB0) * wm + b);
        if (row0 >= nrows) continue;  // uniform
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int row = 8 * (r >> 2) + 4 * half + (r & 3);
            float v;
            if constexpr (I8)
              v = (float)acc[h][b][j][r] * (s_scale[row0 + row] * ws[j]) + bi[j];
            else
              v = acc[h][b][j][r];
            if constexpr (sizeof(T) == 4)
              st[row * 64 + 32 * j + l32] = v;
            else
              st[row * 64 + 32 * j + l32] = (T)f32_to_bf16(v);
          }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int c = lane; c < 32 * 64 / EC; c += 64) {
          const int row = c / (64 / EC), at = c % (64 / EC) * EC;  // column among the wave's 64
          const int grow = row0 + row, col = c0 + col_of(at >> 5, wn) + (at & 31);
          if (grow < nrows && col < ncols)
            *(u32x4_t*)((T*)p.out + (row_base + grow) * ldo + col) = *(const u32x4_t*)(st + row * 64 + at);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      }
  };
  if (p.fp32)
    write(0.0f);
  else
    write((uint16_t)0);
}

// Row-tiled products (NT, NN).  Workgroup b runs on XCD b % 8; a row tile's
// panels stay on one XCD, whose L2 then serves the tile's rows again.
template <OpKind KIND, bool I8, int GX>
__global__ __launch_bounds__(512, 1) void k_op_rows(TileArgs p) {
  __shared__ u32x4_t lds[10 * HU];  // 160 KB
  RowTile tl = find_tile(p.g, blockIdx.x & 7, blockIdx.x >> 3, p.npan, p.g.K * (I8 ? 1 : 2) % 128 == 0);
  // the same in every lane, which the compiler cannot see behind the scan
  tl = RowTile{__builtin_amdgcn_readfirstlane(tl.e), uniform64(tl.p0), __builtin_amdgcn_readfirstlane(tl.rows),
               __builtin_amdgcn_readfirstlane(tl.panel), __builtin_amdgcn_readfirstlane(tl.once)};
  if (tl.e < 0) return;
  auto run = [&](auto r0, auto r1, auto once) {
    tile_product<KIND, I8, r0(), r1(), GX, once()>(p, tl.e, tl.p0, tl.rows, 0, 0, tl.panel, lds, nullptr);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  if (tl.rows > 192) {
    run(c2, c2, std::false_type{});
  } else if (tl.once) {
    if (tl.rows > 128)
      run(c2, c1, std::true_type{});
    else if (tl.rows > 64)
      run(c2, c0, std::true_type{});
    else
      run(c1, c0, std::true_type{});
  } else {
    if (tl.rows > 128)
      run(c2, c1, std::false_type{});
    else if (tl.rows > 64)
      run(c2, c0, std::false_type{});
    else
      run(c1, c0, std::false_type{});
  }
}

// Weight gradients (TN): a workgroup per expert and 256 x 256 tile of dw, in
// eight equal runs, one for each XCD: an expert's tiles share dy and x in one
// L2.
template <int GX>
__global__ __launch_bounds__(512, 1) void k_op_wgrad(TileArgs p) {
  __shared__ u32x4_t lds[8 * HU];
  __shared__ int32_t gidx[GX == GX_ROWS ? 1 : GI];  // 32 KB
  const int per = p.nrow * p.npan;
  const int run = (p.g.E * per + 7) / 8, unit = (int)(blockIdx.x & 7) * run + (int)(blockIdx.x >> 3);
  if (unit >= p.g.E * per) return;
  const int e = unit / per, tile = unit % per;
  const Range r = group_range(p.g, e);
  tile_product<OP_TN, false, 2, 2, GX, false>(p, e, uniform64(r.lo), 0, uniform64(r.size()), tile / p.npan, tile % p.npan, lds,
                                       gidx);
}

}  // namespace

int64_t op_tile_units(OpKind kind, const Groups& g) {
  const int64_t pn = (g.N + TB - 1) / TB, pk = (g.K + TB - 1) / TB;
  if (kind == OP_TN) return (g.E * pn * pk + 7) / 8 * 8;
  const int64_t npan = kind == OP_NT ? pn : pk;
  const int64_t tiles = (g.rows + TB - 1) / TB + (g.offsets ? (g.E < g.rows ? g.E : g.rows) : 0);
  return g.offsets && tiles >= kDealTiles ? ((tiles + 7) / 8 + 3) * 8 * npan : (tiles * npan + 7) / 8 * 8;
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
  const unsigned grid = (unsigned)op_tile_units(kind, g);
  const Launch lc{s, nullptr, nullptr};
  // Gathered rows past the range of a buffer descriptor are fetched by 64-bit addresses.  So are they
  // where x has no row at all: every index then stands for zeros, which that form reads from kZero,
  // while a descriptor of range 0 would not hold lanes back at the later steps' scalar offsets (the
  // check is against range - scalar offset, which wraps).
  const bool far = g.perm && (g.x_rows == 0 || ((g.x_rows - 1) * g.ldx + g.K) * (i8 ? 1 : 2) > kRange);
  const dim3 gr(grid), bl(512);
  if (kind == OP_TN) {
    if (!g.perm) return launch(lc, k_op_wgrad<GX_ROWS>, gr, bl, t);
    return far ? launch(lc, k_op_wgrad<GX_FAR>, gr, bl, t) : launch(lc, k_op_wgrad<GX_INDEX>, gr, bl, t);
  }
  if (kind == OP_NN) return launch(lc, k_op_rows<OP_NN, false, GX_ROWS>, gr, bl, t);
  if (i8)
    return far ? launch(lc, k_op_rows<OP_NT, true, GX_FAR>, gr, bl, t)
               : launch(lc, k_op_rows<OP_NT, true, GX_ROWS>, gr, bl, t);
  return far ? launch(lc, k_op_rows<OP_NT, false, GX_FAR>, gr, bl, t)
             : launch(lc, k_op_rows<OP_NT, false, GX_ROWS>, gr, bl, t);
}

}  // namespace moe

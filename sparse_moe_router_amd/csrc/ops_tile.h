// The output tile of the matrix-matrix kernels (gfx950, wave64, MFMA): the
// search for a workgroup's tile, the reduction loop, and the epilogue that
// stores the tile.  Kernels that do something else with a tile give
// tile_product an epilogue of their own.
#pragma once

#include <type_traits>

#include "ops_internal.h"
#include "ops_paths.h"

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
  int tiles, height;    // NT, NN, one group: number of row tiles, rows of each (set_row_tiles)
  int shift;            // several groups: exponent of 2 of the height
  int splits;           // TN: parts of the reduction (0 and 1: the whole)
  const float* factor;  // ScaledEpi
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

// The wave's LDS writes are visible to its own reads, and its reads done before its next writes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// v, unknown to the compiler: what follows from it is computed here, not carried from one tile to the
// next in registers that the loop needs.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
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

// Heights of row tiles: where all of them run at a time, low ones, each of which takes less (a tile takes 0.6
// us a step of up to 64 rows, 1 of 128 and 1.45 of 256; measured, us, tiles of 256 and these: 2000 x 2048 x
// 2048 40 and 26, 256 x 8192 x 1024 25 and 16, 8192 x 512 x 4096 67 and 43, 400 x 1024 x 4096 66 and 34, by
// rows of int8 42 and 28 for 1000 x 4096 x 4096; 1000 x 2048 against 1000 columns of logits 46 and 26).  Of
// several groups, forward products of rows x N x K: 1024 x 4096 x 4096 over 2 67 and 44, 700 x 4096 x 2048 over 2
// 38 and 22, 2000 x 512 x 1024 over 8 23.8 and 13.4, 600 x 1536 x 2048 over 8 33 and 25, 4000 x 256 x 512 over 4
// 16.0 and 9.3; where the weights' stream bounds both, and two to four low tiles of a group read its weights: 512 x
// 4096 x 4096 over 8 67 and 62 with skewed groups, 70 and 67 with even ones, 512 x 2048 x 4096 over 8 skewed 68 and
// 54, 512 x 8192 x 2048 over 4 44 and 42.
// `room`: the workgroups that the tiles of all panels may take.
// Of one group: the number of its tiles.
inline int64_t dense_tiles(int64_t rows, int64_t npan, int room) {
  for (int h = 64; h < TB; h += 64) {
    const int64_t n = (rows + h - 1) / h;
    if (n * npan <= room) return n;
  }
  return (rows + TB - 1) / TB;
}
// Of several groups, whose sizes only the device knows: the exponent of 2 of the height.
inline int64_t most_tiles(const Groups& g, int shift) {
  return (g.rows >> shift) + (g.E < g.rows ? g.E : g.rows);
}
inline int tile_shift(const Groups& g, int64_t npan, int room) {
  return most_tiles(g, 6) * npan <= room ? 6 : most_tiles(g, 7) * npan <= room ? 7 : 8;
}
static_assert(TB == 1 << 8, "tile_shift");
// The heights for the kernels, from g and npan (found by every workgroup, 8-bit products of 4096 x 4096 x 256 take
// 18.9 us, not 18.3; rows' gradients of 32768 rows over 256 experts of 512 x 2048 162.8, not 161.6).
inline void set_row_tiles(TileArgs* t, int room = kChainGroups) {
  const int64_t n = dense_tiles(t->g.rows, t->npan, room);
  t->tiles = (int)n;
  // Where all units run at a time, the tiles share the rows evenly, in whole blocks of 32: the tallest one
  // takes the time of the launch (257 rows against 32003 columns of 2048: 256 + 1 rows 56 us, 160 + 97 50).
  t->height = n > 0 && n * t->npan <= kChainGroups ? (int)((t->g.rows + 32 * n - 1) / (32 * n)) * 32 : TB;
  t->shift = tile_shift(t->g, t->npan, room);
}

// One group: the units (tile, panel) are cut into eight equal runs, one for
// each XCD, and within a run into blocks of four tiles, panel by panel: the 32
// workgroups that an XCD runs at a time then read about as many tiles' rows as
// panels' weights (int8 4096 x 8192 x 4096: 126 -> 119 us).
__device__ __forceinline__ RowTile find_tile_dense(const TileArgs& p, int xcd, int local, bool aligned) {
  constexpr int SG = 4;
  const Groups& g = p.g;
  const int total = p.tiles, npan = p.npan;  // at most kOpMaxUnits units
  const int run = (total * npan + 7) / 8, unit = xcd * run + local;
  if (local >= run || unit >= total * npan) return RowTile{-1, 0, 0, 0, 0};
  const int sg = unit / (SG * npan), sr = unit - sg * SG * npan;
  const int height = total - sg * SG < SG ? total - sg * SG : SG, panel = sr / height;
  const int64_t p0 = (int64_t)(sg * SG + sr - panel * height) * p.height;
  if (p0 >= g.rows) return RowTile{-1, 0, 0, 0, 0};
  return RowTile{0, p0, (int)(g.rows - p0 < p.height ? g.rows - p0 : p.height), panel, total == 1 && aligned};
}

// Groups: the tiles in three classes, the tallest first, so that the short
// ones fill the end of the launch; of each class, in group order, one eighth
// goes to each XCD: an expert's tiles and a tile's panels then share its
// weights and rows in one L2, and the XCDs stream from distant experts.
// Against tiles dealt to the XCDs one by one, and against one run for each XCD
// in group order: 8192 tokens x 2 over 16 experts 122, 136 and 148 us; 4096 x
// 8 over 256 experts 241, 304, 241; 2501 x 4 over 60 skewed ones 51, 52, 60.
// With fewer than 64 tiles single panels are dealt out.  Low tiles are one class.
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
__device__ __forceinline__ RowTile find_tile(const TileArgs& p, int xcd, int local, bool aligned) {
  if (!p.g.offsets) return find_tile_dense(p, xcd, local, aligned);
  const Groups& g = p.g;
  const int npan = p.npan, shift = p.shift, low = (1 << shift) - 1;
  const int lane = threadIdx.x & 63, per = (g.E + 63) / 64;
  // tiles of this lane's groups in each class: bits 0..31, 32..47, 48..63
  uint64_t mine = 0;
  for (int j = 0; j < per; j += 4) {
    Range r[4];
    four_ranges(g, lane * per + j, lane * per + per, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t c = (uint32_t)r[u].size(), rest = c % TB;
      mine += shift < 8 ? (c + low) >> shift : c / TB;
      if (shift == 8 && rest > 0) mine += (uint64_t)1 << (tile_class(rest) == 0 ? 0 : 16 + 16 * tile_class(rest));
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
    panel = local % npan;
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
    panel = (local * 8 + xcd) % npan;
    if (i >= total) return RowTile{-1, 0, 0, 0, 0};
    cl = i < n0 ? 0 : i < n0 + n1 ? 1 : 2;
    i -= cl == 0 ? 0 : cl == 1 ? n0 : n0 + n1;
  }
  const int at = cl == 0 ? 0 : 16 + 16 * cl;
  const uint64_t mask = cl == 0 ? 0xFFFFFFFFu : 0xFFFFu;
  const int src = __builtin_ctzll(__ballot((int64_t)((incl >> at) & mask) > i));
  i -= (int64_t)((__shfl(incl - mine, src, 64) >> at) & mask);
  for (int j = 0; j < per; j += 4) {
    Range r[4];
    four_ranges(g, src * per + j, src * per + per, r);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t size = r[u].size(), full = size >> shift;
      const int rest = (int)(size & low);
      const int64_t here = (cl == 0 ? full : 0) + (rest > 0 && (shift < 8 || tile_class(rest) == cl));
      if (i < here) {
        const int64_t k = cl == 0 ? i : full;  // the tile's place in its group
        return RowTile{src * per + j + u, r[u].lo + (k << shift), k < full ? low + 1 : rest, panel, size <= low + 1 && aligned};
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
// EPI: what becomes of the tile.  StoreEpi stores it as the output of p; any
// other type's member tile() takes it from the accumulators.  EPI::kGated (NT):
// an expert has two weight matrices of N rows, one after the other, and a tile
// 128 columns of each: column half j holds those of matrix j, so that a wave has
// the same 32 columns of both in the same registers.
struct StoreEpi {
  static constexpr bool kGated = false, kFactor = false;
};
// The same, times p.factor (a type of its own: the products cost short weight gradients 3%).
struct ScaledEpi {
  static constexpr bool kGated = false, kFactor = true;
};
template <class EPI>
constexpr bool kStores = std::is_same<EPI, StoreEpi>::value || std::is_same<EPI, ScaledEpi>::value;
// Where an epilogue's tile lies, and the thread's place in it.
struct TileOut {
  int64_t p0;       // first row
  int rows;         // rows that exist
  int c0, panel;    // first column, panel
  int tid, wave, wm, wn, lane;
};
// A tile: expert, first row of its group's rows, rows of it that exist (NT, NN) or rows to reduce (TN),
// tile along n (TN), panel.
struct TileJob {
  int e;
  int64_t p0;
  int rows;
  int64_t len;
  int r0t, panel;
};
// next(job): the workgroup's following tile, if it is of the same kind.  With one, its first transfers
// are issued before the epilogue of the tile at hand, which then hides their way: a tile of 256 x 256
// costs 9.5 us beside its steps without it (4096 x 16384 x 256 .. 4096, at 1.45 us a step).
struct NoNext {
  static constexpr bool kChain = false;
  __device__ __forceinline__ bool operator()(TileJob&) const { return false; }
};
template <class F>
struct ChainNext {
  static constexpr bool kChain = true;
  F f;
  __device__ __forceinline__ bool operator()(TileJob& t) const { return f(t); }
};
template <class F>
__device__ __forceinline__ ChainNext<F> chain_next(F f) {
  return ChainNext<F>{f};
}
// Row tiles of one group do where there are more, and where few of their rows are missing ones: a short
// tile alone costs less than a whole one (1 to 192 rows 0.4 to 0.8 of it).
inline bool takes_chain(const Groups& g, int64_t units) {
  const int64_t rest = g.rows % TB;
  return !g.offsets && units > kChainGroups && (rest == 0 || rest > 192 || g.rows >= 8 * TB);
}
// LDS of the epilogues, a part of each wave's own: of tiles that follow each other the 32 KB behind the
// stages of two whole row halves, else any 64 KB.
constexpr int EPI_AT = 8 * HU;
template <bool CHAIN>
constexpr int kEpiUnits = CHAIN ? HU / 4 : HU / 2;
template <bool CHAIN>
__device__ __forceinline__ u32x4_t* epi_lds(u32x4_t* lds, int wave) {
  return lds + (CHAIN ? EPI_AT : HU) + wave * kEpiUnits<CHAIN>;
}

template <OpKind KIND, bool I8, int RB0, int RB1, int GX, bool ONCE, class EPI = StoreEpi, class NEXT = NoNext>
__device__ __forceinline__ void tile_product(const TileArgs& p, TileJob job, u32x4_t* lds, int32_t* gidx,
                                             const EPI& epi = EPI{}, const NEXT& next = NEXT{}) {
  constexpr bool GATED = EPI::kGated, CHAIN = NEXT::kChain;
  static_assert(!CHAIN || (RB0 == 2 && RB1 == 2 && !I8), "tiles in a row are whole ones");
  static_assert(!GATED || (KIND == OP_NT && !I8), "two matrices an expert: bf16 NT products");
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
  // the tile whose steps run, or are being fetched
  int e = 0, rows = 0, r0t = 0, c0 = 0;
  int64_t p0 = 0, len = 0;
  auto set_job = [&](const TileJob& t) __attribute__((always_inline)) {
    e = t.e, p0 = t.p0, rows = t.rows, len = t.len, r0t = t.r0t;
    c0 = t.panel * (GATED ? TB / 2 : TB);
  };
  constexpr int BKE = I8 ? 128 : 64;  // reduction elements of a step
  // first column of the tile's 32-column block wn of column half j.  Weights read along memory: a
  // wave's two blocks side by side, so that it writes whole cache lines; across: halves of 128.
  // Of a gated product's half: of its own matrix.
  auto col_of = [&](int j, int blk) { return GATED ? 32 * blk : BT ? 128 * j + 32 * blk : 64 * blk + 32 * j; };

  // ---- transfers.  Along-memory operand: a transfer fills 8 stage rows of 128
  // bytes, lane -> row lane/8, chunk position lane%8, source chunk
  // (lane%8) ^ ((row/2) % 8): 16 consecutive rows' reads then fall on all
  // banks.  Across-rows operand: 4 stage rows of 256 bytes, lane -> row
  // lane/16, position lane%16, source chunk position ^ 4 (row % 4): the four
  // rows a transposing read takes together lie in different 64-byte parts.
  constexpr bool G64 = GX == GX_FAR;
  const bool gather = KIND == OP_TN ? GX != GX_ROWS : KIND == OP_NT && g.perm;
  const int64_t lda = KIND == OP_NT ? g.ldx : g.ldy;
  int64_t red = KIND == OP_NT ? g.K : g.N;  // reduction length (TN: of this chunk)
  int64_t base = 0;                         // TN: first row of the chunk
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
  auto set_steps = [&]() __attribute__((always_inline)) {
    nsteps = (int)((red + BKE - 1) / BKE);
    last = (int)(red - (int64_t)(nsteps - 1) * BKE);
    if (AT) {
      abase = p.a + base * g.ldy * 2;
    } else {
      abase = p.a + (gather ? 0 : p0 * lda * ES);
      // whole chunks of 16 bytes (rows of dy may end inside one, in zeros)
      abytes = (((gather ? g.x_rows : rows) - 1) * lda + (red + 7) / 8 * 8) * ES;
    }
    if (KIND == OP_NT) {
      bbase = p.b + ((int64_t)e * (GATED ? 2 : 1) * g.N + c0) * g.K * ES;
      bbytes = (int64_t)(g.N - c0) * g.K * ES;
    } else if (KIND == OP_NN) {
      bbase = p.b + (int64_t)e * g.N * g.K * 2;
    } else {
      bbase = p.b + (gather ? 0 : base * g.ldx * 2);
      bbytes = ((g.x_rows - 1) * g.ldx + g.K) * 2;  // gathered
    }
  };
  auto set_a = [&]() __attribute__((always_inline)) {
    const int lane = CHAIN ? here(tid & 63) : tid & 63, lr = lane >> 3;
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
  auto set_b = [&]() __attribute__((always_inline)) {
    const int lane = CHAIN ? here(tid & 63) : tid & 63, lr = lane >> 3;
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
  auto load_a = [&](int h, int st, int s) __attribute__((always_inline)) {
    const int sc = s < nsteps ? s : nsteps - 1;
#pragma unroll
    for (int i = 0; i < RBM; ++i) {
      if (i >= (h ? RB1 : RB0)) continue;
      const uint32_t dst = lds0 + (sa(h, st) - lds + (wave * (h ? RB1 : RB0) + i) * 64) * 16;
      if (AT) {
        dma(step_window(abase, astep, s, (g.N + 7) / 8 * 16), aoff[h][i], 0, dst);
      } else if (G64 && gather) {
        dma64(a64[h][i] && (s < nsteps - 1 || aend[h][i]) ? a64[h][i] + sc * 128 : (const char*)kZero, dst);
      } else {
        dma(window(abase, abytes), s >= nsteps - 1 && !aend[h][i] ? kOut : aoff[h][i], sc * 128, dst);
      }
    }
  };
  const int64_t bhalf = GATED ? (int64_t)g.N * g.K * 2 : 0;  // from an expert's first matrix to its second
  auto load_b = [&](int j, int st, int s) __attribute__((always_inline)) {
    const int sc = s < nsteps ? s : nsteps - 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = lds0 + (sb(j, st) - lds + (wave * 2 + i) * 64) * 16;
      if (!BT) {
        const uint32_t off = s >= nsteps - 1 && !bend[j][i] ? kOut : boff[j][i];
        if (ONCE)
          dma_once(window(bbase + j * bhalf, bbytes), off, sc * 128, dst);
        else
          dma(window(bbase + j * bhalf, bbytes), off, sc * 128, dst);
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
  auto read_a = [&](int h, int st) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int b = 0; b < RBM; ++b) {
        if (b >= (h ? RB1 : RB0)) continue;
        const int r = 32 * ((h ? RB1 : RB0) * wm + b);
        af[b][kk] = AT ? read_across(sa(h, st), r, kk) : read_along(sa(h, st), r, kk);
      }
  };
  auto read_b = [&](int j, int st) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      bf[j][kk] = BT ? read_across(sb(j, st), 32 * wn, kk) : read_along(sb(j, st), 32 * wn, kk);
  };
  // the multiply part of a cluster, between its two barriers
  auto multiply = [&](int h, int j) __attribute__((always_inline)) {
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

  // ---- epilogue.  Block layout: lane -> column lane%32, register r -> row
  // 8 (r/4) + 4 (lane/32) + r%4.
  auto epilogue_of = [&](const TileOut& at, int c0, int rows, int e, int r0t, int64_t p0) __attribute__((always_inline)) {
    const int lane = at.lane, half = lane >> 5, l32 = lane & 31;
    if constexpr (!kStores<EPI>) {
      epi.template tile<RB0, RB1>(p, at, acc, lds);
      return;
    } else {
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
    float factor = 1.0f;
    if constexpr (EPI::kFactor) factor = *p.factor;
    // 64 columns of some of a block's rows at a time through a part of the LDS of the wave's own, then
    // 16 bytes a lane
    auto write = [&](auto type) __attribute__((always_inline)) {
      typedef decltype(type) T;
      constexpr int EC = 16 / sizeof(T);                            // results of a 16-byte chunk
      constexpr int RT = kEpiUnits<CHAIN> * 16 / (64 * sizeof(T)), PR = RT < 32 ? RT : 32;  // rows at a time
      T* st = (T*)epi_lds<CHAIN>(lds, wave);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < RBM; ++b) {
          if (b >= (h ? RB1 : RB0)) continue;
          const int row0 = (h ? 64 * RB0 : 0) + 32 * ((h ? RB1 : RB0) * wm + b);
#pragma unroll
          for (int q = 0; q < 32 / PR; ++q) {
            if (row0 + PR * q >= nrows) continue;  // uniform
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int r = PR / 2 * q; r < PR / 2 * (q + 1); ++r) {
                const int row = 8 * (r >> 2) + 4 * half + (r & 3);
                float v;
                if constexpr (I8)
                  v = (float)acc[h][b][j][r] * (s_scale[row0 + row] * ws[j]) + bi[j];
                else
                  v = EPI::kFactor ? acc[h][b][j][r] * factor : acc[h][b][j][r];
                if constexpr (sizeof(T) == 4)
                  st[(row - PR * q) * 64 + 32 * j + l32] = v;
                else
                  st[(row - PR * q) * 64 + 32 * j + l32] = (T)f32_to_bf16(v);
              }
            wave_sync();
#pragma unroll
            for (int i = 0; i < PR / EC; ++i) {
              const int c = i * 64 + lane;
              const int row = c / (64 / EC), at = c % (64 / EC) * EC;  // column among the wave's 64
              const int grow = row0 + PR * q + row, col = c0 + col_of(at >> 5, wn) + (at & 31);
              if (grow < nrows && col < ncols)
                *(u32x4_t*)((T*)p.out + (row_base + grow) * ldo + col) = *(const u32x4_t*)(st + row * 64 + at);
            }
            wave_sync();
          }
        }
    };
    if (p.fp32)
      write(0.0f);
    else
      write((uint16_t)0);
    }
  };

  // The first transfers of a pass over the reduction from its row `done` on.
  auto prologue = [&](int64_t done) __attribute__((always_inline)) {
    if (KIND == OP_TN) {
      red = gather && len - done > GI ? GI : len - done;
      base = p0 + done;
    }
    if (KIND == OP_TN && gather) {
      // up to a whole number of steps, rows past the end as -1
      for (int i = tid; i < (red + 63) / 64 * 64; i += 512) gidx[i] = i < red ? (int32_t)source_row(g, base + i) : -1;
      __syncthreads();
    }
    set_steps();
    set_b();
    if constexpr (RB1 > 0) {
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
    } else {
#pragma unroll
      for (int d = 0; d < ST; ++d) {
        load_b(0, d, d);
        if (d < ST - 1) load_b(1, d, d);
      }
      set_a();
#pragma unroll
      for (int d = 0; d < ST; ++d) load_a(0, d, d);
    }
  };

  bool fetched = false;  // the first transfers are on their way
  set_job(job);
  for (;;) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RBM; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[h][b][j] = (acc_t){};
    // One pass over the reduction; weight gradients with gathered rows pass in
    // chunks whose row indexes fit the LDS.
    for (int64_t done = 0; KIND != OP_TN ? done == 0 : done < len; done += KIND != OP_TN ? 1 : gather ? GI : len) {
      if (!fetched) prologue(done);
      fetched = false;
      if constexpr (RB1 > 0) {
        // memory parts: 8, 4, 8 and 4 reads of a block, two transfers a wave in each.  The first column
        // half of a step is read in the last part of the step before.  (Stores of the tile before count
        // as transfers in these waits, which they only make longer.)
        constexpr int WB = 6 + RB0 + 2 * RB1, WA = 6 + 2 * RB0 + RB1;
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

    const int c0t = c0, rowst = rows, et = e, r0tt = r0t;  // of the tile that is done
    const int64_t p0t = p0;
    const int ln = CHAIN ? here(lane) : lane;
    const TileOut at{p0, rows, c0, job.panel, wave * 64 + ln, wave, wm, wn, ln};
    bool more = false;
    if constexpr (CHAIN) {
      more = next(job);
      if (more) {
        set_job(job);
        if (KIND != OP_TN || len > 0) {
          prologue(0);
          fetched = true;
        }
      }
    }
    epilogue_of(at, c0t, rowst, et, r0tt, p0t);
    if (!CHAIN || !more) break;
    // the epilogue's LDS is free again for every wave
    wait_vm<63>();
    bar();
  }
}
// The workgroup's tile of a row-tiled product (NT, NN).  Workgroup b runs on XCD
// b % 8; a row tile's panels stay on one XCD, whose L2 then serves the tile's
// rows again.
template <OpKind KIND, bool I8, int GX, class EPI = StoreEpi>
__device__ __forceinline__ void row_tile(const TileArgs& p, u32x4_t* lds, const EPI& epi = EPI{}) {
  RowTile tl = find_tile(p, blockIdx.x & 7, blockIdx.x >> 3, p.g.K * (I8 ? 1 : 2) % 128 == 0);
  // the same in every lane, which the compiler cannot see behind the scan
  tl = RowTile{__builtin_amdgcn_readfirstlane(tl.e), uniform64(tl.p0), __builtin_amdgcn_readfirstlane(tl.rows),
               __builtin_amdgcn_readfirstlane(tl.panel), __builtin_amdgcn_readfirstlane(tl.once)};
  if (tl.e < 0) return;
  auto run = [&](auto r0, auto r1, auto once) __attribute__((always_inline)) {
    tile_product<KIND, I8, r0(), r1(), GX, once(), EPI>(p, TileJob{tl.e, tl.p0, tl.rows, 0, 0, tl.panel}, lds, nullptr, epi);
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

// The same for one group of many tiles, in a launch of kChainGroups workgroups:
// each takes every 32nd tile of its XCD, one after the other, and all of them as
// whole ones.
template <OpKind KIND, class EPI = StoreEpi>
__device__ __forceinline__ void row_chain(const TileArgs& p, u32x4_t* lds, const EPI& epi = EPI{}) {
  int local = blockIdx.x >> 3;
  auto take = [&](TileJob* t) __attribute__((always_inline)) {
    const RowTile tl = find_tile_dense(p, blockIdx.x & 7, local, false);
    *t = TileJob{0, tl.p0, tl.rows, 0, 0, tl.panel};
    return tl.e >= 0;
  };
  TileJob t;
  if (!take(&t)) return;
  tile_product<KIND, false, 2, 2, GX_ROWS, false, EPI>(p, t, lds, nullptr, epi,
                                                       chain_next([&](TileJob& t) __attribute__((always_inline)) {
                                                         local += kChainGroups / 8;
                                                         return take(&t);
                                                       }));
}

// Weight gradients: a unit is an expert, a part of its rows and a 256 x 256 tile
// of its dw, in eight equal runs, one for each XCD: an expert's tiles share dy and
// x in one L2.  Unit b of an XCD b % 8; returns the part, -1 past the end.
inline int64_t wgrad_units(const Groups& g, int splits) {
  return ((int64_t)g.E * splits * ((g.N + TB - 1) / TB) * ((g.K + TB - 1) / TB) + 7) / 8 * 8;
}
template <bool PARTS>
__device__ __forceinline__ int wgrad_unit(const TileArgs& p, int b, TileJob* t) {
  const int parts = PARTS && p.splits > 1 ? p.splits : 1, per = p.nrow * p.npan, all = p.g.E * parts * per;
  const int run = (all + 7) / 8, local = b >> 3, unit = (b & 7) * run + local;
  if (local >= run || unit >= all) return -1;
  const int group = unit / per, tile = unit - group * per;
  const int e = PARTS && parts > 1 ? group / parts : group, part = group - e * parts;
  Range r = group_range(p.g, e);
  if (PARTS && parts > 1) {
    // whole steps of rows each
    const int64_t each = (r.size() + 64 * parts - 1) / (64 * parts) * 64, lo = r.lo + part * each;
    r = Range{lo < r.hi ? lo : r.hi, lo + each < r.hi ? lo + each : r.hi};
  }
  *t = TileJob{e, uniform64(r.lo), 0, uniform64(r.size()), tile / p.npan, tile % p.npan};
  return part;
}
// The tile of unit b; parts of a reduction as fp32, one after the other [part][E][N][K].  Without PARTS there
// are none (a tile's way to its rows is then shorter by a division and an address: weight gradients of 512
// rows over 32 experts of 1024 x 2048 34.7 -> 34.2 us, gathered 37.8 -> 37.3).
template <int GX, class EPI = StoreEpi, bool PARTS = true>
__device__ __forceinline__ void wgrad_tile(const TileArgs& args, int b, u32x4_t* lds) {
  static_assert(GI * 4 <= 2 * HU * 16, "indexes behind the stages");
  TileJob t;
  const int part = wgrad_unit<PARTS>(args, b, &t);
  if (part < 0) return;
  if constexpr (PARTS) {
    TileArgs p = args;
    p.out = (char*)p.out + (int64_t)part * p.g.E * p.g.N * p.g.K * 4;
    tile_product<OP_TN, false, 2, 2, GX, false, EPI>(p, t, lds, (int32_t*)(lds + 8 * HU));
  } else {
    tile_product<OP_TN, false, 2, 2, GX, false, EPI>(args, t, lds, (int32_t*)(lds + 8 * HU));
  }
}

// Workgroups of a launch of row tiles with npan panels each.
inline int64_t row_tile_units(const Groups& g, int64_t npan, int room = kChainGroups) {
  if (!g.offsets) return (dense_tiles(g.rows, npan, room) * npan + 7) / 8 * 8;
  const int shift = tile_shift(g, npan, room);
  const int64_t tiles = most_tiles(g, shift);
  return tiles >= kDealTiles ? ((tiles + 7) / 8 + 3) * 8 * npan : (tiles * npan + 7) / 8 * 8;
}
// Gathered rows past the range of a buffer descriptor are fetched by 64-bit addresses.  So are they
// where x has no row at all: every index then stands for zeros, which that form reads from kZero,
// while a descriptor of range 0 would not hold lanes back at the later steps' scalar offsets (the
// check is against range - scalar offset, which wraps).
inline bool rows_far(const Groups& g, int es) {
  return g.perm && (g.x_rows == 0 || ((g.x_rows - 1) * g.ldx + g.K) * es > kRange);
}

// ---- for epilogues

// f(row0, a0, a1) for each 32-row block of the wave that has rows: its first row in the tile and the
// accumulators of the two column halves.
template <int RB0, int RB1, class ACC, class F>
__device__ __forceinline__ void each_block(const TileOut& o, ACC& acc, F&& f) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < (RB0 > RB1 ? RB0 : RB1); ++b) {
      if (b >= (h ? RB1 : RB0)) continue;
      const int row0 = (h ? 64 * RB0 : 0) + 32 * ((h ? RB1 : RB0) * o.wm + b);
      if (row0 >= o.rows) continue;  // uniform
      f(row0, acc[h][b][0], acc[h][b][1]);
    }
}
// Row of a block that register r of a lane holds.
__device__ __forceinline__ int block_row(int r, int lane) { return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); }
// 4 KB of LDS of the wave, whether or not the tile has a follower.
__device__ __forceinline__ void* epi_stage(u32x4_t* lds, const TileOut& o) { return epi_lds<true>(lds, o.wave); }
// Rows 16 q .. +16 of a block there, columns 0..31 of the first column half, 32..63 of the second; the
// 16-byte chunks of a row change places with its number, so that a chunk of all rows lies on all banks.
__device__ __forceinline__ void stage16(float* st, int q, int lane, const f32x16_t& a0, const f32x16_t& a1) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = block_row(i, lane), col = lane & 31;
    float* at = st + row * 64 + (((col >> 2) ^ row) & 15) * 4 + (col & 3);
    *at = a0[8 * q + i];
    at = st + row * 64 + (((col >> 2 | 8) ^ row) & 15) * 4 + (col & 3);
    *at = a1[8 * q + i];
  }
}
__device__ __forceinline__ const f32x4_t* staged(const float* st, int row, int chunk) {
  return (const f32x4_t*)(st + row * 64 + ((chunk ^ row) & 15) * 4);
}

}  // namespace
}  // namespace moe

// Which kernel a forward product (y = x W^T) runs on, and into how many parts a
// reduction is cut: rules on sizes alone (host code without HIP).
#pragma once

#include <stdint.h>

namespace moe {

// Matrix-vector or matrix-matrix kernel.  The latter takes the time of one
// tile's reduction however few tiles there are (measured 5.7 us + 2.9 ns a byte
// of a weight row for tiles of up to 64 rows, 6.5 us + 6.9 ns for 256).  The former is bound in two ways:
//  - all its workgroups together by the touched weights (at most min(E, rows)
//    experts'): 3 us + those at 3.9 TB/s, by 1/43 longer for each row of a
//    group.  That is less while the touched weight rows, so weighted, are fewer
//    than 3.9 TB/s * 2.9 ns = about 12000, whatever their length.  Both sides, us
//    (matrix-vector / matrix-matrix): rows of 4 KB, N 4096, one expert: 8 rows
//    6.5 / 16.2, 64 rows 12.1 / 16.8, 128 rows 22.8 / 17.7; N 1024, top-8 of 256:
//    1 token 8.9 / 19.0, 2 tokens 18.3 / 19.3, 4 tokens 34.9 / 24.1; N 8192 of 16
//    KB: 16 rows 38.5 / 53.0, 64 rows 82 / 55; N 2048 of 1 KB, top-8: 1 token 10.8
//    / 9.6; N 4096 of 128 B: 8 rows 3.9 / 4.3, 64 rows 5.2 / 4.7.
//  - each workgroup by its group's rows, which it takes 64 at a time, one after
//    the other, however few workgroups a narrow output has.  One group, N 64,
//    weight rows of 512 B, 2 KB and 8 KB: 64 rows 5.1 / 5.7, 6.9 / 10.6 and 20 /
//    31 us, 128 rows 8.8 / 5.9, 12.5 / 10.8 and 38 / 31, 256 rows 16 / 5.9, 24 / 11
//    and 74 / 31, 4096 rows 236 / 6.1, 487 / 11 and 1281 / 31 (N 8 to 1024 and int8
//    much the same; N 392 of 8 KB: 64 rows 21 / 46, 128 rows 40 / 31).
//    Several groups share their rows, evenly or not: 256 rows of 2 KB over 4
//    groups of N 64 take 7.4 / 11.7 evenly and 23.8 / 21.5 when one group has
//    them all, over 16 groups 4.5 / 11.4 and 23.5 / 21.3; 512 rows of one of 4
//    groups 46 / 22.
constexpr int64_t kSkinnyWeightRows = 12000;
inline bool takes_matrix_vector(int64_t rows, int E, int N) {
  const int64_t groups = rows < E ? rows : E;
  return N * (43 * groups + rows) < 43 * kSkinnyWeightRows && rows <= (groups > 1 ? 256 : 128);
}

// bf16 tokens for int8 weights that the matrix-vector kernel quantises itself,
// every workgroup for its own use, instead of a launch before it (one token, K
// 2048, N 4096: 4.9 against 6.1 us and 2 us less of host time): up to four
// tokens and 16384 elements, 64 elements a thread, where a group has at most
// the four rows that it quantises at a time (as many as tokens, when a token's
// experts differ).
constexpr int kInsideRows = 4, kInsideElems = 16384;
inline bool quantizes_inside(int64_t rows, int64_t x_rows, int E, int N, int K) {
  return takes_matrix_vector(rows, E, N) && x_rows <= kInsideRows && x_rows * K <= kInsideElems &&
         rows <= (int64_t)kInsideRows * E;
}

// Logits of tokens against a vocabulary, and their gradients: the matrix-vector
// kernel takes 64 tokens and 16 columns a workgroup, so that small ones do not
// wait for a tile's whole reduction (0.6 us a step of 64 elements and 10), while
// it reads tokens and weights from the caches many times over: where all its
// workgroups run at a time.  Both sides, us (matrix-vector / tiles), rows of 128,
// 512, 2048 and 4096 elements: 1 token, 1000 columns (63 workgroups) 6.7 / 8.8, 7.2
// / 11.4, 8.6 / 24.4 and 11.5 / 43.4; 16 tokens, 4000 columns (250) 7.7 / 9.4, 8.5 /
// 13.1, 11.2 / 27.5 and 15.9 / 46.7; 64 tokens, 4000 columns (250) 10.7 / 10.0, 12.1
// / 14.3, 17.9 / 30.9 and 27.8 / 51.9; 200 tokens, 1000 columns (252) 10.7 / 10.0,
// 12.0 / 12.4, 18.6 / 22.1 and 27.9 / 35.1; 400 tokens, 1000 columns (441) 11.8 /
// 10.0, 14.4 / 12.4, 28.2 / 22.2 and 48.1 / 35.9; 1000 tokens, 1000 columns (1008)
// 19.5 / 10.2, 23.2 / 12.6, 51.3 / 22.4 and 90.6 / 35.8; 16 tokens, 16000 columns
// (1000) 12.9 / 10.1, 15.1 / 13.9, 26.5 / 31.1 and 43.7 / 53.1.  Beyond that the tiles lose up to a third to
// 1 to 16 tokens of 16000 columns, and nothing from 32000 on, where their 125 and more workgroups share the
// weights' stream: rows of 1024, 2048 and 4096 elements, 1 token x 16000 columns 15.8 / 18.3, 21.1 / 29.3 and
// 34.0 / 49.8; x 32000 26.1 / 20.1, 37.2 / 35.9 and 62.5 / 63.9, 16 tokens 33.0 / 20.0, 47.7 / 36.2 and 82.5 /
// 64.9; 1 token x 64000 47.1 / 28.5, 68.7 / 66.5 and 119.6 / 105.2; x 128000 88.2 / 52.8, 132 / 113 and 233 /
// 204, 16 tokens 116 / 52.7, 175 / 116 and 310 / 207.
constexpr int64_t kSkinnyLogitGroups = 256;
inline bool takes_matrix_vector_logits(int64_t rows, int64_t columns) {
  return (rows + 63) / 64 * ((columns + 15) / 16) <= kSkinnyLogitGroups;
}

// Backward pass of a gated feed-forward block (H columns of dy, I features, K columns of x): the kernels for
// few rows read an expert's weights once a row, mostly from the caches, where a tile waits for its whole
// reduction; with many experts both are bound by the gradients that they write.  Both sides, us (few rows /
// tiles), with H = K, 1, 8, 16, 32 and 64 rows: 1 expert of 512 x 2048 15.6 / 40.3, 16.8 / 39.8, 23.9 / 40.5,
// 34 / 42, 55 / 44; 1 of 2048 x 4096 47 / 103, 58 / 104, 80 / 106, 144 / 110; 4 of 584 x 1456 19.9 / 39.1, 21.8
// / 38.3, 26 / 39, 35 / 39, 58 / 40; 8 of 88 x 376 8.2 / 17.8, 8.8 / 18.2, 9.5 / 18.1, 11.4 / 17.9, 15.1 / 18.8;
// 16 of 1408 x 4096 135 / 159, 192 / 195, 230 / 211, 311 / 230; 64 of 512 x 2048 90 / 97, 103 / 113, 118 / 121,
// 139 / 136; 256 of 512 x 2048 287 / 287, 302 / 291, 319 / 298, 351 / 332; 8 of 1024 x 2048 35 / 70, 57 / 69, 61 /
// 69, 75 / 69.  With all rows on one of the experts, 8, 16 and 32 rows: 8 of 1024 x 2048 40 / 70, 47 / 71, 60 / 74;
// 64 of 512 x 2048 93 / 98, 99 / 101, 110 / 103; 64 of 128 x 512 17 / 23, 21 / 24, 28 / 25; 8 of 88 x 376 11.8 / 18.2,
// 15.5 / 18.8, 23.1 / 19.8 (a weight gradient's workgroup walks its expert's rows one after another).  The bounds
// are round ones: at their edges either side loses up to a fifth (16 rows of 2048 x 4096 take tiles at 106 for 80,
// 1 row over 16 of 1408 x 4096 at 160 for 135; 32 rows over 64 experts the few-row kernels at 145 for 133).
constexpr int64_t kFewRows = 32, kFewRead = 1 << 28, kFewWritten = 1 << 28;
inline bool takes_few_rows(int64_t rows, int64_t E, int64_t H, int64_t I, int64_t K) {
  const int64_t weights = I * (2 * K + H);
  return rows > 0 && rows <= kFewRows && rows * weights <= kFewRead && E * weights <= kFewWritten;
}

// Workgroups that run at a time, one a compute unit: those of a launch whose tiles follow each other.
constexpr int kChainGroups = 256;

// How many parts to cut a reduction into is a question of what fills the 256 workgroups that run at a
// time.  launch_steps: the time, in steps of 64, of a launch of n0 tiles of s0 steps and then n1 tiles of s1,
// each started where one before it ends.  A tile costs kTileSteps beside its own steps, a launch behind it
// kLaunchSteps, and kStepBytes of fp32 parts written or read one.  (Fitted to 450 timings of cross
// entropies' and feed-forward blocks' gradients at 1 to 32 slices and parts.  Over 8 blocks the choices are the
// best ones timed; over 19 cross entropies they cost 1.1% more with both gradients and 2.8% for dx alone, which
// a choice weighs a third of both: at worst 18%, 92 for 78 us, for the dx of 2000 tokens against 4000 x 1024.
// Those of a rule that filled the workgroups cost 7%.)
constexpr int kTileSteps = 7, kLaunchSteps = 2;
constexpr int64_t kStepBytes = 4 << 20;
constexpr int64_t kMostTiles = 2 * kChainGroups;  // of a cut reduction: more cost more
inline int64_t launch_steps(int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
  const int64_t q = n0 / kChainGroups, r = n0 % kChainGroups, early = kChainGroups - r;
  // the tiles of s1 start at t0 on `early` workgroups, at t1 on the others
  const int64_t t0 = q * s0, t1 = r ? t0 + s0 : t0;
  if (n1 <= 0) return t1;
  if (r == 0) return t0 + (n1 + kChainGroups - 1) / kChainGroups * s1;
  // ends with a tile of the former, or of the latter
  const int64_t up = (s0 + s1 - 1) / s1, down = s0 / s1;
  const int64_t j0 = early * up >= n1 ? (n1 + early - 1) / early : (n1 + r * up + kChainGroups - 1) / kChainGroups;
  const int64_t left = n1 - early * down, j1 = left > 0 ? (left + kChainGroups - 1) / kChainGroups : 0;
  const int64_t a = t0 + j0 * s1 > t1 ? t0 + j0 * s1 : t1, b = t1 + j1 * s1;
  return a < b ? a : b;
}
// The next count of parts to look at: 1 .. 8, then 10, 12, 15, ...
inline int next_parts(int n) { return n + (n < 8 ? 1 : n / 4); }

}  // namespace moe

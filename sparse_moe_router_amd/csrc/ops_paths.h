// Which kernel a forward product (y = x W^T) runs on: rules on sizes alone
// (host code without HIP).
#pragma once

#include <stdint.h>

namespace moe {

// Matrix-vector or matrix-matrix kernel.  The latter takes the time of one
// tile's reduction however few tiles there are (measured 5.7 us + 2.9 ns a byte
// of a weight row for up to 64 rows of a group, 6.5 us + 6.9 ns for 256 and
// more).  The former is bound in two ways:
//  - all its workgroups together by the touched weights (at most min(E, rows)
//    experts'): 3 us + those at 3.9 TB/s, by 1/43 longer for each row of a
//    group.  That is less while the touched weight rows, so weighted, are fewer
//    than 3.9 TB/s * 2.9 ns = about 12000, whatever their length.  Both sides, us
//    (matrix-vector / matrix-matrix): rows of 4 KB, N 4096, one expert: 8 rows
//    6.5 / 16.2, 64 rows 12.1 / 16.8, 128 rows 22.8 / 21.0; N 1024, top-8 of 256:
//    1 token 8.9 / 19.0, 2 tokens 18.3 / 19.3, 4 tokens 34.9 / 24.1; N 8192 of 16
//    KB: 16 rows 38.5 / 53.0, 64 rows 82 / 55; N 2048 of 1 KB, top-8: 1 token 10.8
//    / 9.6; N 4096 of 128 B: 8 rows 3.9 / 4.3, 64 rows 5.2 / 4.7.
//  - each workgroup by its group's rows, which it takes 64 at a time, one after
//    the other, however few workgroups a narrow output has.  One group, N 64,
//    weight rows of 512 B, 2 KB and 8 KB: 64 rows 5.3 / 5.6, 7.2 / 10.6 and 20 /
//    30 us, 128 rows 9.0 / 6.8, 12.8 / 12.8 and 38 / 37, 256 rows 16 / 10, 24 / 20
//    and 74 / 63, 4096 rows 236 / 10, 476 / 21 and 1276 / 63 (N 8 to 1024 and int8
//    much the same; by tiles, N 392 and more of 8 KB take 44 us for 64 rows and 50
//    for 128).
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
// wait for a tile's whole reduction (0.6 us a step of 64 elements for up to 64
// tokens, 1 us for more, and 10), while it reads tokens and weights from the caches
// many times over.  Both sides, us (tiles / matrix-vector), rows of 128, 512, 2048
// and 4096 elements: 1 token, 1000 columns 9.0 / 10.4, 10.9 / 9.2, 22.6 / 9.7 and
// 43.5 / 13.4; 64 tokens, 4000 columns 9.7 / 11.1, 13.8 / 12.6, 26.6 / 19.0 and 49 /
// 29; 400 tokens, 1000 columns 15.0 / 12.3, 20.5 / 13.9, 41 / 28 and 72 / 49; 200
// tokens, 4000 columns (1000 workgroups) 14.9 / 18.7, 20.2 / 22.5, 41 / 44 and 71 /
// 77; 1000 tokens, 1000 columns 16.7 / 19.3, 21.9 / 23.0, 43 / 52 and 73 / 91; 16
// tokens, 16000 columns 10.1 / 13.3, 12.1 / 15.6, 29.5 / 26.7 and 52 / 44.
constexpr int64_t kSkinnyLogitGroups = 700;
inline bool takes_matrix_vector_logits(int64_t rows, int64_t columns) {
  return (rows + 63) / 64 * ((columns + 15) / 16) <= kSkinnyLogitGroups;
}

}  // namespace moe

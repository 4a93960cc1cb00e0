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

}  // namespace moe

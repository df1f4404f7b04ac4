// Which kernel an 8-bit product takes.
#pragma once
#include <cstdint>

namespace nf {

// Whether a product goes to the kernel of few rows of A, which fills the GPU by cutting K
// (the fewer tiles of weights, the more rows), or to tiles of 128 rows x 256, which read the
// weights once for all rows.  Few rows / tiles, us, K 4096, by tiles of 128 weight rows:
//   64 (8192): 64 rows 10.8 / 15.6, 128 rows 13.2 / 15.8; 256 rows of 6144 19.1 / 15.6;
//   SwiGLU, 32 (2048): 128 rows 11.3 / 12.7; 64 (4096): 64 rows 12.0 / 14.5, 128 rows 15.4 / 14.6;
//   112 (14336): 64 rows 14.8 / 16.9, 128 rows 19.5 / 17.4;
//   224 (28672): 16 rows 23.2 / 30.5, 32 rows 23.5 / 23.4, 64 rows 25.1 / 23.8;
//   224 (SwiGLU, 14336): 32 rows 23.6 / 24.1, 64 rows 25.8 / 24.2;
//   1002 (128256): 16 rows 89 / 96, 32 rows 97 / 89.
// By groups, with the rows' mean (a tile has room for twice as many, of SwiGLU for 64):
//   8 of 1024 x 4096 (64): 64 rows 13.5 / 19.0; SwiGLU, 8 of 512 (64): 32 rows 12.5 / 19.4, 64
//   rows 21.9 / 19.5; 8 of 2048 (128): 32 rows 16.4 / 20.0, 64 rows 19.9 / 20.6;
//   8 of 14336 x 4096 SwiGLU: 1 row 73 / 102, 8 rows 139 / 140, 32 rows 165 / 142;
//   64 of 2048 x 2048: 8 rows 58 / 48 (a CTA a tile: short ones do not pay), 64 of 768 x 2048:
//   2 rows 25.5 / 24.0.  At a row a group or less, with more tiles than SMs, short K pays where
//   tiles are few; 1 row (0.5 rows) of 64 of 2048 x 1024 28 / 22 (18.4 / 16.2), of 128 of 1024 x
//   1024 30 / 23, of 16 of 8192 x 1024 25 / 21; of 64 of 2048 x 2048 40 / 37 (26.9 / 26.6), of
//   768 x 2048 15.8 / 16.1, of 128 of 512 x 2048 28 / 26 (14.4 / 15.8), of 16 of 4096 x 2048
//   23.8 / 23.9, of 8 of 8192 x 2048 15.6 / 17.9; of 64 of 1024 x 4096 41 / 44, of 2048 x 4096
//   67 / 66, of 768 x 2048 SwiGLU 25.5 / 29.7.
// A capped product takes the tiles, which loop (a unit of the other kernel is a cluster of its
// own): 1 row of 4096 x 14336 13.5 us without a cap, 22.5 under one of 76 SMs or more, 30.5
// under 38; 64 rows 15.6, 23.0, 31.4.
inline bool few_rows(int M, int N, int K, int groups, bool two, int sms) {
  const int rows = (M + groups - 1) / groups;
  const int64_t ops = two ? 2 : 1;
  const int64_t tiles = (N + 127LL) / 128 * ops * (M < groups ? M : groups);
  if (groups > 1) {
    if (tiles > sms)
      return rows <= 16 && (K * ops >= 8192 || (M <= groups && (K * ops >= 4096 || (K * ops >= 2048 && tiles <= 4LL * sms))));
    return rows <= (tiles <= sms / 2 && !two ? 64 : 32);
  }
  return rows <= (tiles <= sms / (two ? 4 : 2) ? 128 : tiles <= sms ? 64 : tiles <= 2 * sms ? 32 : 16);
}

}  // namespace nf

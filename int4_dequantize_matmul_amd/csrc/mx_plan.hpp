// Which tile a product with MX FP4 weights and many activation rows takes.
// Plain host code, so that it can be checked without a GPU.
#pragma once

#include <cstdint>

namespace q4 {

inline int64_t mx_tiles(int64_t M, int64_t N, int64_t bm, int64_t bn) {
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

// W4A4, by activation rows x weight rows.  The smallest tile whose grid the
// CUs take at once, its K shared out among the waves (a workgroup's time is its
// stages' latencies then); past that 128 x 128, two workgroups a CU, and 256 x
// 256 once those fill three quarters of the CUs.  Microseconds on 256 CUs,
// smaller tile | larger tile:
//   N 2048 K 5632: 32 x 64 at 256 rows (9.4 | 10.6), 64 x 64 at 512 (11.4 | 15.0)
//   N 13312 K 2048: 64 x 64 at 64 rows (6.6 | 7.4), 128 x 128 at 512 (14.4 |
//     19.1), 256 x 256 at 1024 (24.6 | 22.3)
// large: not for f32 results whose scales do not start on 16 bytes: 256 x 256
// would spill 142 of its registers there (2048 rows, N 13312 K 2080: 169 us
// against 87 with 128 x 128; 8192 rows, N 2048 K 5600: 194 against 103).
enum class MxW4A4Tile : int { k32x64, k64x64, k128x128, k256x256 };

inline MxW4A4Tile mx_w4a4_tile(int64_t M, int64_t N, int64_t cus, bool large) {
  if (mx_tiles(M, N, 32, 64) <= cus) return MxW4A4Tile::k32x64;
  if (mx_tiles(M, N, 64, 64) <= cus) return MxW4A4Tile::k64x64;
  if (large && 4 * mx_tiles(M, N, 256, 256) >= 3 * cus) return MxW4A4Tile::k256x256;
  return MxW4A4Tile::k128x128;
}

// W4A16.  The same up to the large tiles of 128 x 256.  Microseconds on 256
// CUs, smaller tile | larger tile:
//   N 2048 K 5632: 32 x 64 up to 256 rows (14.7 | 19.3), 64 x 64 at 512
//     (21.2 | 26.8), 64 x 128 at 1024 (28.3 | 35.0)
//   N 13312 K 2048: 32 x 64 at 32 rows (8.1 | 9.2), 64 x 64 at 64 (9.6 |
//     12.0), 64 x 128 at 128 (12.6 | 15.5)
// Between them and one round of 128 x 256: 128 x 128 where those are more than
// the CUs (N 13312 K 2048, 512 rows: 30.6 against 35.2), else the large tiles
// in quarters, which are 64 x 128 without a cut of K, three and more a CU (the
// same at 256 rows: 19.1 against 21.7).  large: whether the operands are aligned
// as the large tiles need (rows of activations on 16 bytes, of scales on 4);
// 128 x 128 otherwise.
enum class MxW4A16Tile : int { k32x64, k64x64, k64x128, k128x128, kLarge };

inline MxW4A16Tile mx_w4a16_tile(int64_t M, int64_t N, int64_t cus, bool large) {
  if (mx_tiles(M, N, 32, 64) <= cus) return MxW4A16Tile::k32x64;
  if (mx_tiles(M, N, 64, 64) <= cus) return MxW4A16Tile::k64x64;
  if (mx_tiles(M, N, 64, 128) <= cus) return MxW4A16Tile::k64x128;
  if (large && (mx_tiles(M, N, 128, 256) >= cus || mx_tiles(M, N, 128, 128) <= cus)) return MxW4A16Tile::kLarge;
  return MxW4A16Tile::k128x128;
}

}  // namespace q4

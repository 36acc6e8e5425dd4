// Parts that the LDS-tiled MX FP4 products share: the order of tiles, the
// order of weight rows in the matrix instructions, and the stores.
#pragma once

#include "mx_device.hpp"

namespace q4 {

constexpr int kFar = 0x7FFFFFF0;   // a buffer offset past every range: the load gives 0

// bf16 results: a lane's four results of two neighbouring instructions are 8
// neighbouring columns of y, which it stores in 16 bytes.  The instruction's
// rows are weight rows in an order of its own for that: row i of instruction
// t is weight row 32 (t / 2) + 8 (i / 4) + 4 (t % 2) + i % 4.  f32 results:
// four columns are 16 bytes, rows in order.
template <bool BOUT>
__device__ __forceinline__ int w_row(int t, int i) {
  return BOUT ? 32 * (t >> 1) + 8 * (i >> 2) + 4 * (t & 1) + (i & 3) : 16 * t + i;
}

// Workgroups are dealt to the 8 XCDs in turn.  The place of workgroup id of n
// in an order that gives each XCD a run of neighbours.
__device__ __forceinline__ int xcd_run(int id, int n) {
  const int q = n >> 3, rem = n & 7, xcd = id & 7;
  return xcd * q + min(xcd, rem) + (id >> 3);
}

// Tile i of tiles_m x tiles_n: bands of 8 tiles of activation rows, and the
// tiles of a weight panel next to each other in a band, so that the tiles an
// XCD works on at a time share few panels of both operands in its L2.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int i, int tiles_m, int tiles_n) {
  const int band = i / (8 * tiles_n), at = i - band * 8 * tiles_n, rows = min(tiles_m - 8 * band, 8);
  // (the divisions leave uniform values in vector registers)
  return {__builtin_amdgcn_readfirstlane(8 * band + at % rows), __builtin_amdgcn_readfirstlane(at / rows)};
}

// Stores of a wave of 16 TM rows by 16 TN weight rows: lane (c, q) has row c of each 16 activation rows, from
// row m0 and column n0 on.
template <int TN, int TM, bool BOUT>
__device__ __forceinline__ void store_tile(void *y, int64_t M, int64_t N, int64_t m0, int64_t n0,
                                           const f32x4 (&acc)[TM][TN]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int64_t m = m0 + 16 * tm + r;
    if (m >= M) continue;
    if constexpr (BOUT) {
#pragma unroll
      for (int tn = 0; tn < TN; tn += 2) {
        const int64_t n = n0 + 16 * tn + 8 * g;
        const f32x4 u = acc[tm][tn], v = acc[tm][tn + 1];
        if (n + 8 <= N) {
          store_any(static_cast<uint16_t *>(y) + m * N + n,
                    make_uint4(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
        } else {
          if (n < N) store_y4<true>(y, m, n, N, u);
          if (n + 4 < N) store_y4<true>(y, m, n + 4, N, v);
        }
      }
    } else {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int64_t n = n0 + 16 * tn + 4 * g;
        if (n < N) store_y4<false>(y, m, n, N, acc[tm][tn]);
      }
    }
  }
}

// The same for results of 32 x 32 instructions: the row i of an instruction is
// weight row w_row32(i) of its 32, so that lane (c, h) has 16 neighbouring
// columns of y.
__device__ __forceinline__ int w_row32(int i) { return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3); }

template <bool BOUT>
__device__ __forceinline__ void store_16(void *y, int64_t m, int64_t n, int64_t N, const f32x16 &v) {
  if constexpr (BOUT) {
#pragma unroll
    for (int j = 0; j < 16; j += 8) {
      uint16_t *p = static_cast<uint16_t *>(y) + m * N + n + j;
      if (n + j + 8 <= N) {
        store_any(p, make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                      pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7])));
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (n + j + i < N) p[i] = static_cast<uint16_t>(pack_bf16(v[j + i], 0.0f));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const f32x4 u = {v[j], v[j + 1], v[j + 2], v[j + 3]};
      if (n + j + 4 <= N) store_any(static_cast<float *>(y) + m * N + n + j, u);
      else if (n + j < N) store_y4<false>(y, m, n + j, N, u);
    }
  }
}

// Stores of a wave's 32 TM rows by 32 TN columns of 32 x 32 results, in whole
// lines past the caches: through LDS of the wave's own (64 TM TN 32 bytes),
// half of the columns at a time if they are f32.  A lane's own 16 columns would
// be 16-byte pieces of as many lines, which have to meet in L2 and are written
// back from there when the kernel ends.
template <int TM, int TN, bool BOUT>
__device__ __forceinline__ void store_lines(uint8_t *lds, void *y, int64_t M, int64_t N, int64_t m0, int64_t n0,
                                            const f32x16 (&acc)[TM][TN]) {
  constexpr int PASSES = BOUT ? 1 : 2, T = TN / PASSES;         // column tiles of a pass
  constexpr int W = T * 32 * (BOUT ? 2 : 4), C = W / 16, PER = BOUT ? 8 : 4;
  static_assert(C == 8 || C == 16, "rows of 128 or 256 bytes");
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2)));
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  auto place = [](int row, int q) { return row * W + ((q ^ (C == 16 ? row & 15 : (row >> 1) & 7)) << 4); };
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const f32x16 &v = acc[tm][p * T + t];
#pragma unroll
        for (int j = 0; j < 16; j += PER) {
          uint4 u;
          if constexpr (BOUT)
            u = make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]), pack_bf16(v[j + 4], v[j + 5]),
                           pack_bf16(v[j + 6], v[j + 7]));
          else
            u = make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                           __float_as_uint(v[j + 3]));
          *reinterpret_cast<uint4 *>(lds + place(32 * tm + r, (32 * t + 16 * h + j) / PER)) = u;
        }
      }
#pragma unroll
    for (int i = 0; i < 32 * TM * C / 64; ++i) {
      const int row = i * (64 / C) + lane / C, q = lane % C;
      const uint4 u = load16(lds + place(row, q));
      const int64_t m = m0 + row, n = n0 + p * T * 32 + q * PER;
      if (m >= M) continue;
      if (n + PER <= N) {
        uint8_t *to = static_cast<uint8_t *>(y) + (m * N + n) * (BOUT ? 2 : 4);
        __builtin_nontemporal_store(__builtin_bit_cast(U, u), reinterpret_cast<U *>(to));
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < PER - 1; ++j)
          if (n + j < N) {
            if constexpr (BOUT) static_cast<uint16_t *>(y)[m * N + n + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
            else static_cast<uint32_t *>(y)[m * N + n + j] = w[j];
          }
      }
    }
  }
}

}  // namespace q4

// What the attention kernels share: the operands of their matrix products, the
// rows of a tile and the keys that they see.
#pragma once

#include "kv_device.hpp"

namespace q4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// acc += A B over 16 columns of 32 rows; operands and results lie as in mfma_bf16_32x32x16.
__device__ __forceinline__ f32x16 mfma_f16_32x32x16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Four int8 codes -> four halves, exactly: with the sign bit turned, a byte b
// under the exponent 0x64 is the half 1024 + b, b = code + 128.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const f16x2 bias = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
  const f16x2 lo = __builtin_bit_cast(f16x2, perm_b32(0x64646464u, u, 0x04010400u)) - bias;
  const f16x2 hi = __builtin_bit_cast(f16x2, perm_b32(0x64646464u, u, 0x04030402u)) - bias;
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}
__device__ __forceinline__ uint4 codes_to_f16(uint32_t a, uint32_t b) {
  const uint2 x = codes_to_f16(a), y = codes_to_f16(b);
  return make_uint4(x.x, x.y, y.x, y.y);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f16x2 v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
// What rounding v to a half leaves, as a half.
__device__ __forceinline__ float rest_f16(float v) { return v - static_cast<float>(static_cast<_Float16>(v)); }

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// 2^n as a float, n in -126 .. 127.
__device__ __forceinline__ float power2(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

// Rows of a tile: row r of a sequence and key head is query head g = r mod G of
// that key head's G, of the sequence's row r / G, so that all rows of a tile
// share their keys.
struct RowTile {
  int i;                  // sequence, or -1: nothing to do
  int64_t r0, rows;       // first row, rows of the sequence in all
  Sequence s;
  // ROWS a tile; sequence i has the slots from floor(starts[i] G / ROWS) + i on
  __device__ __forceinline__ RowTile(const KvSeqs &q, int64_t slot, int64_t G, int ROWS)
      : i(search_last<64>(static_cast<int>(q.N), slot, [&](int j) { return start(q, j, G, ROWS); })),
        s(q, i < 0 ? 0 : i) {
    if (i < 0) return;
    r0 = (slot - start(q, i, G, ROWS)) * ROWS;
    rows = s.n * G;
    if (r0 >= rows) i = -1;
  }
  static __device__ __forceinline__ int64_t start(const KvSeqs &q, int j, int64_t G, int ROWS) {
    return Sequence::clamp(q.starts[j], q.T) * G / ROWS + j;
  }
};
inline int64_t tile_slots(int64_t T, int64_t N, int64_t G, int ROWS) { return T * G / ROWS + N; }

// The keys that rows at positions p0 .. p1 see together, as blocks of 16 in a
// row: sinks' blocks, then those from the window's first key to the last row's own.
struct KeyBlocks {
  int sink_blocks, skip, count;   // block v is v, or v + skip from sink_blocks on
  __device__ __forceinline__ KeyBlocks(int64_t p0, int64_t p1, int64_t window, int64_t sinks) {
    const int end = p1 < 0 ? 0 : static_cast<int>(p1 / kKvBlock) + 1;
    const int64_t w0 = window > 0 && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
    const int first = static_cast<int>(w0 / kKvBlock);
    const int64_t sb = (sinks + kKvBlock - 1) / kKvBlock;
    sink_blocks = sb < first ? static_cast<int>(sb) : first;
    skip = first - sink_blocks;
    count = end - skip;
  }
  __device__ __forceinline__ int block(int v) const { return v < sink_blocks ? v : v + skip; }
};

}  // namespace q4

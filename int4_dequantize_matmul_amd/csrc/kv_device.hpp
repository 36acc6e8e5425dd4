// The paged 8-bit cache on the device: where blocks lie, and which sequence a
// workgroup works for.
//
// A block is 16 tokens of one key head: keys int8 [D/16][16 tokens][16 columns],
// values int8 [D][16 tokens], 16 D bytes each, under one scale byte b = 2^(b -
// 127) (255: NaN).  A page holds its heads one after the other, a head its
// blocks.  So a lane's 16-byte load is 16 columns of a key or 16 tokens of a
// value column, neighbouring lanes' loads are neighbours, and both are operands
// of the matrix instructions as they come.
#pragma once

#include "kernels.hpp"
#include "mx_device.hpp"

namespace q4 {

constexpr int kKvBlock = 16;

// The last i in 0 .. n - 1 with f(i) <= x, f not decreasing; -1 if there is
// none.  G lanes (a power of two, 16 or 64) search together, all of them active.
template <int G, class F>
__device__ __forceinline__ int search_last(int n, int64_t x, F f) {
  const int lane = threadIdx.x & (G - 1), base = threadIdx.x & 63 & ~(G - 1);
  int lo = 0;
  while (n > 0) {
    const int step = (n + G - 1) / G, i = lane * step;
    const bool yes = i < n && f(lo + i) <= x;
    unsigned long long b = __ballot(yes) >> base;
    if constexpr (G < 64) b &= (1ull << G) - 1;
    const int c = __popcll(b);
    if (c == 0) return -1;             // only in the first turn
    lo += (c - 1) * step;
    if (step == 1) break;
    n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
  }
  return lo;
}

// A sequence's rows of this call (its last tokens) and where they stand.
struct Sequence {
  int64_t row, n;      // first row, rows
  int64_t len, first;  // tokens with them; position of the first row (below 0: more rows than tokens)
  __device__ __forceinline__ Sequence(const KvSeqs &s, int i) {
    const int64_t a = clamp(s.starts[i], s.T), b = clamp(s.starts[i + 1], s.T);
    row = a;
    n = b > a ? b - a : 0;
    len = s.lengths[i] > 0 ? s.lengths[i] : 0;
    first = len - n;
  }
  static __device__ __forceinline__ int64_t clamp(int64_t v, int64_t T) { return v < 0 ? 0 : v > T ? T : v; }
};

// The number in the pool of block b of a head of sequence i, or -1 where its
// page is not in the table or not in the pool.
__device__ __forceinline__ int64_t block_at(const KvPool &c, int i, int64_t b, int64_t head) {
  const int64_t p = b >> c.page_blocks_log2;
  if (p >= c.width) return -1;
  const int64_t id = c.pages[i * c.width + p];
  if (id < 0 || id >= c.n_pages) return -1;
  return ((id * c.Hk + head) << c.page_blocks_log2) + (b & ((int64_t(1) << c.page_blocks_log2) - 1));
}

// Blocks of 16 tokens that a call touches: workgroup slots are shared out so
// that sequence i has the slots from floor(starts[i] / 16) + 2 i on, at least as
// many as its n rows touch (floor(n / 16) + 2), with no sum over sequences.
inline int64_t block_slots(int64_t T, int64_t N) { return T / kKvBlock + 2 * N; }

struct BlockOf {
  int i;             // the sequence, or -1: nothing to do
  int64_t b;         // its block
  __device__ __forceinline__ BlockOf(const KvSeqs &s, int64_t slot) {
    const auto f = [&](int j) { return Sequence::clamp(s.starts[j], s.T) / kKvBlock + 2 * int64_t(j); };
    i = search_last<64>(static_cast<int>(s.N), slot, f);
    if (i < 0) return;
    const Sequence q(s, i);
    const int64_t lo = q.first > 0 ? q.first : 0;
    b = lo / kKvBlock + (slot - f(i));
    if (q.n == 0 || b * kKvBlock >= q.len) i = -1;
  }
};

}  // namespace q4

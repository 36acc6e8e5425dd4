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

// What all lanes have the same of, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A sequence's rows of this call (its last tokens) and where they stand; 32 bits,
// as starts and lengths have.
struct Sequence {
  int i;            // its number, or -1: none
  int row, n;       // first row, rows
  int len, first;   // tokens with them; position of the first row (below 0: more rows than tokens)
  __device__ __forceinline__ void set(int a, int b, int l) {
    row = a;
    n = b > a ? b - a : 0;
    len = l > 0 ? l : 0;
    first = len - n;
  }
  static __device__ __forceinline__ int clamp(int v, int64_t T) { return v < 0 ? 0 : v > T ? static_cast<int>(T) : v; }
};

// The last sequence i with f(starts[i], i) <= x, f not decreasing.  G lanes (1, or
// 64 with the same x) search together, all of them active; what they find is the
// same in each.  Fewer than 64 sequences take one round of loads.
template <int G, class F>
__device__ __forceinline__ Sequence find_sequence(const KvSeqs &s, uint32_t x, F f) {
  Sequence q;
  const int N = static_cast<int>(s.N), lane = threadIdx.x & 63;
  if (G == 64 && N < 64) {
    const int start = Sequence::clamp(s.starts[min(lane, N)], s.T), length = s.lengths[min(lane, N - 1)];
    q.i = __popcll(__ballot(lane < N && f(static_cast<uint32_t>(start), lane) <= x)) - 1;
    if (q.i >= 0)
      q.set(__builtin_amdgcn_readlane(start, q.i), __builtin_amdgcn_readlane(start, q.i + 1),
            __builtin_amdgcn_readlane(length, q.i));
    return q;
  }
  int lo = 0, n = N;
  q.i = -1;
  if constexpr (G == 1) {
    const bool few = N < 64;               // then every lane has one's start
    const int start = few ? Sequence::clamp(s.starts[min(lane, N)], s.T) : 0;
    auto at = [&](int i) { return few ? __shfl(start, i) : Sequence::clamp(s.starts[i], s.T); };
    int hi = N;                            // f(lo) <= x < f(hi), taken that way at the ends
    for (int m = N; m > 0; m >>= 1) {      // the same turns in every lane
      const int mid = (lo + hi) >> 1;
      const bool yes = f(static_cast<uint32_t>(at(mid)), mid) <= x;
      if (yes) lo = mid;
      else hi = mid > lo ? mid : hi;
    }
    const int from = at(lo), to = at(lo + 1);   // by all lanes
    q.i = f(static_cast<uint32_t>(from), lo) <= x ? lo : -1;
    q.set(from, to, s.lengths[lo]);
    return q;
  }
  while (true) {
    const int step = (n + 63) / 64, i = lane * step;
    const bool yes = i < n && f(static_cast<uint32_t>(Sequence::clamp(s.starts[lo + (i < n ? i : 0)], s.T)), lo + i) <= x;
    const int c = __popcll(__ballot(yes));
    if (c == 0) return q;                  // only in the first turn
    lo += (c - 1) * step;
    if (step == 1) break;
    n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
  }
  q.i = lo;
  q.set(Sequence::clamp(s.starts[lo], s.T), Sequence::clamp(s.starts[lo + 1], s.T), s.lengths[lo]);
  q.i = uniform(q.i), q.row = uniform(q.row), q.n = uniform(q.n), q.len = uniform(q.len), q.first = uniform(q.first);
  return q;
}

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
  Sequence s;        // i = -1: nothing to do
  int b;             // its block
  __device__ __forceinline__ BlockOf(const KvSeqs &seqs, uint32_t slot) {
    const auto f = [&](uint32_t start, int j) { return start / kKvBlock + 2 * static_cast<uint32_t>(j); };
    s = find_sequence<64>(seqs, slot, f);
    if (s.i < 0) return;
    const uint32_t ahead = slot - f(static_cast<uint32_t>(s.row), s.i);
    b = max(s.first, 0) / kKvBlock + static_cast<int>(ahead);
    // (a number of blocks past any sequence's)
    if (s.n == 0 || ahead > (1u << 28) || b * static_cast<int64_t>(kKvBlock) >= s.len) s.i = -1;
  }
};

}  // namespace q4

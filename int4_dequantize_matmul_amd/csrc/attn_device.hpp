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

// acc += A B over 32 columns of 16 rows: lane (r, q) has 8 columns of row r; result register i of lane (c, q) is the
// element of A's row 4 q + i and B's row c.
__device__ __forceinline__ f32x4 mfma_f16_16x16x32(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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
// The same of two numbers and their halves: one operation each that takes the half as it lies, subtracts and rounds
// (with a factor that the compiler does not know, or it would convert, subtract and round in three).
__device__ __forceinline__ uint32_t rest_f16(uint32_t halves, float lo, float hi) {
  float minus = -1.0f;
  asm("" : "+v"(halves), "+s"(minus));
  const f16x2 h = __builtin_bit_cast(f16x2, halves);
  return pack_f16(__builtin_fmaf(static_cast<float>(h[0]), minus, lo), __builtin_fmaf(static_cast<float>(h[1]), minus, hi));
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Rows of a tile: row r of a sequence and key head is query head g = r mod G of
// that key head's G, of the sequence's row r / G, so that all rows of a tile
// share their keys.
template <int ROWS>
struct RowTile {
  Sequence s;             // i = -1: nothing to do
  int r0, rows;           // first row, rows of the sequence in all
  // sequence i has the slots from floor(starts[i] G / ROWS) + i on
  __device__ __forceinline__ RowTile(const KvSeqs &q, uint32_t slot, uint32_t G) {
    const auto f = [&](uint32_t start, int j) { return start * G / ROWS + static_cast<uint32_t>(j); };
    s = find_sequence<64>(q, slot, f);
    if (s.i < 0) return;
    const uint32_t at = (slot - f(static_cast<uint32_t>(s.row), s.i)) * static_cast<uint64_t>(ROWS) > INT32_MAX
                            ? INT32_MAX
                            : (slot - f(static_cast<uint32_t>(s.row), s.i)) * ROWS;
    r0 = static_cast<int>(at);
    rows = s.n * static_cast<int>(G);
    if (r0 >= rows) s.i = -1;
  }
};
inline int64_t tile_slots(int64_t T, int64_t N, int64_t G, int ROWS) { return T * G / ROWS + N; }

// Which keys a row sees, in 32 bits (positions are; a larger window or number of
// sinks is like the largest position).
struct Sight {
  int window, sinks;   // window 0 on the outside: all
  __device__ __forceinline__ Sight(int64_t w, int64_t s)
      : window(w > 0 && w < INT32_MAX ? static_cast<int>(w) : INT32_MAX),
        sinks(s < INT32_MAX ? static_cast<int>(s) : INT32_MAX) {}
  // The row at pos does not see key k; pos - k only wraps where k > pos.
  __device__ __forceinline__ bool hides(int pos, int k) const {
    return k > pos || (static_cast<int>(static_cast<uint32_t>(pos) - static_cast<uint32_t>(k)) >= window && k >= sinks);
  }
  // Every row at positions p0 .. p1 sees the 16 keys from k on.
  __device__ __forceinline__ bool whole(int p0, int p1, int k) const {
    return k + 15 <= p0 && (p1 - k < window || k + 15 < sinks);
  }
};

// The keys that rows at positions p0 .. p1 see together, as blocks of 16 in a
// row: sinks' blocks, then those from the window's first key to the last row's own.
// Blocks past the table are NaN: of them the first that each row sees is enough, so
// that the work is bounded by the table and not by what `lengths` says.
struct KeyBlocks {
  int sink_blocks, skip, count;   // block v is v, or v + skip from sink_blocks on
  __device__ __forceinline__ KeyBlocks(int p0, int p1, const Sight &s, const KvPool &pool) {
    const int table = static_cast<int>(pool.width << pool.page_blocks_log2);
    const int first = p0 >= s.window ? (p0 - s.window + 1) / kKvBlock : 0;
    const int last_first = p1 >= s.window ? (p1 - s.window + 1) / kKvBlock : 0;   // the last row's
    const int end = p1 < 0 ? 0 : min(p1 / kKvBlock, max(table, last_first)) + 1;
    sink_blocks = min(min((s.sinks >> 4) + ((s.sinks & 15) != 0), first), table + 1);
    skip = first - sink_blocks;
    count = end - skip;
  }
  __device__ __forceinline__ int block(int v) const { return v < sink_blocks ? v : v + skip; }
};

constexpr float kLog2e = 1.44269504088896340736f;

struct Types {
  bool in_bf16, out_bf16;
};

// A query row as operands, S lanes a row (2 or 4), lane h of them with the columns 16 (S s + h) .. + 15 in f[2 s] and
// f[2 s + 1].
template <int N, int S, bool TWO>
struct Query {
  uint4 hi[2 * N], lo[TWO ? 2 * N : 1];
  float factor;   // what a product's result is multiplied with: scores in powers of two, without the key's scale
  __device__ __forceinline__ void load(const AttnArgs &a, const Types &t, int64_t at, bool live, int h) {
    const int D = static_cast<int>(a.pool.D);
    float x[N][16];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const int c = 16 * (S * s + h);
      const bool in = live && c < D;
#pragma unroll
      for (int u = 0; u < 16; u += 8) {
        if (t.in_bf16) {
          Run8<true> r;
          if (in) r.load(a.q, at + c + u);
          else r.zero();
#pragma unroll
          for (int j = 0; j < 8; ++j) x[s][u + j] = __uint_as_float(j & 1 ? r.v[j / 2] & 0xFFFF0000u : r.v[j / 2] << 16);
        } else {
          Run8<false> r;
          if (in) r.load(a.q, at + c + u);
          else r.zero();
#pragma unroll
          for (int j = 0; j < 8; ++j) x[s][u + j] = r.v[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[s][j]) & 0x7FFFFFFFu);
    }
    if constexpr (S == 4) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
    // exponent of the largest: top in [2^e, 2^(e + 1)), but for rows below 2^-100, which are scaled as if they reached
    // it; a NaN or an infinity makes the whole row NaN
    const int e = max(static_cast<int>(top >> 23) - 127, -100);
    factor = top >= 0x7F800000u ? __builtin_nanf("") : ldexpf(fabsf(a.scale) * kLog2e, e - 14);
    const float to = __uint_as_float(static_cast<uint32_t>(14 - min(e, 127) + 127) << 23) * (a.scale < 0.0f ? -1.0f : 1.0f);
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t w[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = x[s][8 * u + 2 * j] * to, q = x[s][8 * u + 2 * j + 1] * to;
          w[j] = pack_f16(p, q);
          v[j] = pack_f16(rest_f16(p), rest_f16(q));
        }
        hi[2 * s + u] = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (TWO) lo[2 * s + u] = make_uint4(v[0], v[1], v[2], v[3]);
      }
  }
};

// The largest of the S lanes' values, and their sum.
template <int S>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (S == 4) v = max_xor16(v);
  return max_xor32(v);
}
template <int S>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (S == 4) v = add_xor16(v);
  return add_xor32(v);
}

// Running softmax of one query row a lane, which S lanes share (2 or 4), each with
// the scores of one block of 16 keys a step.  Scores s
// are in powers of two; `a` and `d` are whole numbers: l is this lane's sum of
// weights 2^(s - a); y holds the results, sums of 2^(s - a + e - d + kOffset) times
// codes, e the exponent of their values' scale.  So the weights that meet the
// codes are rounded next to the largest product of a weight and its values'
// scale, whatever the scales are.  `a` is as large as scores come; e, d and
// kOffset stay below 2^9 and are never added to a sum that would round them away.
// No maximum is taken as long as the weights
// stay halves: their sum, which is needed anyway, tells.
template <class V, int N, int S, bool TWO>   // N vectors of results
struct State {
  static constexpr int kOffset = TWO ? 10 : 9;
  float a = -__builtin_inff(), d = -__builtin_inff(), l = 0.0f;
  bool far = false;   // some row's `a` has few bits behind the point or none
  V y[N];
  __device__ __forceinline__ State() {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = V{};
  }
  // 16 keys of one block: scores x times f, then weights as operands.
  struct Keys {
    f32x16 x;
    float f, e, sum, shift;
    uint4 p[2], rest[2];
    // Products x of the row with the keys, factor f; kb and vb: the scale bytes of
    // the block's keys and values; hidden(j): the row does not see key j.
    template <bool MASK, class F>
    __device__ __forceinline__ void scores(f32x16 products, float factor, int kb, int vb, F hidden) {
      f = factor * __uint_as_float(kb ? static_cast<uint32_t>(kb) << 23 : 0x400000u);
      if (kb == 255 || vb == 255) f = __builtin_nanf("");
      e = static_cast<float>(vb - 127);
      x = products;
      if constexpr (MASK) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = hidden(j) ? -__builtin_inff() : x[j] * f;
        f = 1.0f;
      }
    }
    // Under the powers a and d.
    __device__ __forceinline__ void weigh(float a, float d, bool far) {
      // nothing seen so far: any finite number will do
      const float fa = a == -__builtin_inff() ? 0.0f : a, fd = d == -__builtin_inff() ? 0.0f : d;
      // weights of 2^-60 and less of what counts are 0 as halves; kept that large, their f32 sum stays right
      shift = fmaxf(e + static_cast<float>(kOffset) - fd, -60.0f);
      float w[16];
      if (__builtin_expect(far, 0)) {
        // the same rounded products as in top(), whose differences from `a` are exact where they matter
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = exp2_fast((x[j] * f - fa) + shift);
      } else {
        const float both = shift - fa;   // exact below 2^22
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = exp2_fast(fmaf(x[j], f, both));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t q[4], r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = w[8 * u + 2 * j], hi = w[8 * u + 2 * j + 1];
          q[j] = pack_f16(lo, hi);
          if constexpr (TWO) {
            r[j] = rest_f16(q[j], lo, hi);
          }
        }
        p[u] = make_uint4(q[0], q[1], q[2], q[3]);
        if constexpr (TWO) rest[u] = make_uint4(r[0], r[1], r[2], r[3]);
      }
#pragma unroll
      for (int n = 8; n > 0; n /= 2)
#pragma unroll
        for (int j = 0; j < n; ++j) w[j] = w[j] + w[j + n];
      sum = w[0];
    }
    __device__ __forceinline__ float top() const {
      float v = x[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) v = fmaxf(v, x[j]);
      return v * f;
    }
  };
  // The weights of the T blocks that this lane has; x: their scores.
  template <int T>
  __device__ __forceinline__ void weights(Keys (&x)[T]) {
    bool again = d == -__builtin_inff();
#pragma unroll
    for (int i = 0; i < T; ++i) {
      x[i].weigh(a, d, far);
      // too large for halves, or kept larger than they are; sums are that of T blocks at most
      again |= x[i].sum > 32768.0f || x[i].shift <= -60.0f;
    }
    if (__any(again)) {
      float top[T], ta = -__builtin_inff(), td = ta;
#pragma unroll
      for (int i = 0; i < T; ++i) top[i] = x[i].top(), ta = fmaxf(ta, top[i]);
      const float na = fmaxf(a, ceilf(row_max<S>(ta))), fa = na == -__builtin_inff() ? 0.0f : na;
#pragma unroll
      for (int i = 0; i < T; ++i) td = fmaxf(td, (top[i] - fa) + x[i].e);
      // what was relative to a and d, relative to na
      const float by = a == na ? 0.0f : a - na, nd = fmaxf(by + d, ceilf(row_max<S>(td)));
      const float ga = exp2_fast(by), gd = by + d == nd ? 1.0f : exp2_fast(by + d - nd);   // from -inf: 0
      a = na, d = nd, far = __any(fabsf(fa) > 0x1p22f);
      l *= ga;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] *= gd;
#pragma unroll
      for (int i = 0; i < T; ++i) x[i].weigh(a, d, far);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) l = fmaf(x[i].sum, exp2_fast(-x[i].shift), l);
  }
};

// What a part's sum of weights relative to 2^a counts relative to 2^to, and its
// results relative to 2^(a + d) relative to 2^(to + td); l is the part's sum: one that saw
// nothing counts 0, one with NaN alone its NaN.
__device__ __forceinline__ float rescale(float a, float l, float to) {
  if (a == -__builtin_inff()) return l == 0.0f ? 0.0f : 1.0f;
  return exp2_fast(a - to);
}
__device__ __forceinline__ float rescale(float a, float d, float l, float to, float td) {
  if (a == -__builtin_inff()) return l == 0.0f ? 0.0f : 1.0f;
  return exp2_fast((a - to) + d - td);
}
// A part's d relative to 2^to, the largest of the parts' a.
__device__ __forceinline__ float lag(float a, float d, float to) {
  return a == -__builtin_inff() ? a : (a - to) + d;
}

// Results over their sum of weights; a row that sees nothing is 0.
struct Quotient {
  float n;
  int e;
  __device__ __forceinline__ Quotient(float d, float l, int offset)
      : n(l == 0.0f ? 0.0f : 1.0f / l), e(d == -__builtin_inff() ? 0 : static_cast<int>(d) - offset) {}
  __device__ __forceinline__ float operator()(float y) const { return ldexpf(y * n, e); }
};

// Four results of one row from column d on.
__device__ __forceinline__ void store4(void *y, bool bf16, int64_t i, float a, float b, float c, float d) {
  if (bf16) store_any(static_cast<uint16_t *>(y) + i, make_uint2(pack_bf16(a, b), pack_bf16(c, d)));
  else store_any(static_cast<float *>(y) + i, make_float4(a, b, c, d));
}


// Many rows a sequence (attention_tiled.hip); attention_plan chooses.  two: queries
// or results in f32.
bool attention_tiled_ok(int64_t D, bool two);
hipError_t launch_attention_tiled(const AttnArgs &a, const Types &t, hipStream_t st);

}  // namespace q4

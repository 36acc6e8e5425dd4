// Keys and values into the paged 8-bit cache, and out of it again.
//
// Append: a row of a key head is normalised (if asked for) and its first R
// columns are rotated by its position's angles, as in qk_norm_rope.hip; then
// the rows of a block of 16 tokens share the scale 2^e, the smallest power of
// two with max|x| <= 127 2^e, and a code is x / 2^e rounded to the nearest, ties
// to even.  Where the block has tokens already, e only grows, and their codes
// are rounded again, c -> rint(c 2^(old - new)): as steps at least double, what
// such roundings add up to stays below one step of the last scale.  Key rows are
// computed in f64, so that a code and the scale depend on no sum's order;
// scaling by a power of two is exact.  Query rows, rounded to 24 or 8 bits, go
// in f32 (the norm of one whose squares f32 does not hold in f64).
//
// Bound: memory for queries, the codes' arithmetic beside it for keys and values;
// 12000 tokens of 32 + 8 heads of 128, norm and rotation of halves: bf16 61 us (26 of
// them the cache's part; queries alone cannot do without 38), neighbours 65, f32 113;
// read back 15.  One token 5.4 us, a chain of loads: sequence, page, scale and codes.
//
// A block of a head has one owner, so nothing is shared between workgroups, and a
// block's scale is written by who writes its codes; keys, values and queries are
// workgroups of their own.  A row of a query or key head belongs to D / 16 lanes
// (rounded up to a power of two) of 16 columns, two runs of 8, one in each half of
// the columns, that are rotated with each other where the halves' distance allows it
// (with 16 columns in a row the 16-byte pieces lie 64 bytes apart: f32 neighbours 128
// us, not 112); they keep their angles and gains over the heads that their workgroup
// has.  Four value columns of a block belong to a lane, 16 tokens a column, so that
// turning them costs nothing.
#include <type_traits>

#include "kv_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float element(const Run8<BF16> &r, int j) {
  if constexpr (BF16) return __uint_as_float(j & 1 ? r.v[j / 2] & 0xFFFF0000u : r.v[j / 2] << 16);
  else return r.v[j];
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&o)[8]) {
  Run8<BF16> t;
  t.load(p, i);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = element(t, j);
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, const float (&o)[8]) {
  if constexpr (BF16)
    store_any(static_cast<uint16_t *>(p) + i, make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                         pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])));
  else {
    float *q = static_cast<float *>(p) + i;
    store_any(q, make_float4(o[0], o[1], o[2], o[3]));
    store_any(q + 4, make_float4(o[4], o[5], o[6], o[7]));
  }
}

// Orders this wave's LDS writes before its later LDS reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// How a row's rotation meets its lanes.
enum Rotation : int {
  kPlain = 0,        // none
  kNeighbours = 1,   // columns 2 i and 2 i + 1: in one run
  kHalves = 2,       // i and i + R / 2, R a multiple of 16: in the two runs of one lane
  kHalvesLds = 3     // any other R: through LDS
};

// The 16 columns of one lane of a head's row, and what is the same for all heads of
// its token: gains and angles.
template <class real, int MODE>
struct Lane {
  int c[2];          // first columns of the two runs
  bool in;           // D / 16 lanes have columns
  bool rotated;      // kHalves: these runs are
  float g[2][8];
  float co[2][8], si[2][8];   // kNeighbours: of pairs 0 .. 3 of each run; kHalves: of run 0's columns; kHalvesLds: of each column
  // p: which of the row's lanes
  __device__ __forceinline__ Lane(const AppendArgs &a, const void *gain, int p, int64_t pos) {
    const int D = static_cast<int>(a.pool.D), R = static_cast<int>(a.R);
    in = p < D / 16;
    rotated = MODE == kHalves && p < R / 16;
    // runs of neighbouring lanes are neighbours, in the first half of the columns and in the second
    const int from = MODE == kHalves && !rotated ? R : 0, all = MODE != kHalves ? D : rotated ? R : D - R;
    c[0] = from + 8 * p - from / 2;
    c[1] = c[0] + all / 2;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!a.norm || !gain || !in) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[u][j] = 1.0f;
      } else if (a.g_bf16) {
        load8<true>(gain, c[u], g[u]);
      } else {
        load8<false>(gain, c[u], g[u]);
      }
    }
    if (MODE == kPlain || !in) return;
    const bool known = pos >= 0 && pos < a.P;   // an unknown position gives NaN, not a wild read
    const float *cs = a.table + (known ? pos : 0) * R, *sn = cs + R / 2;
    if constexpr (MODE == kHalves) {
      if (rotated) load8<false>(cs, c[0], co[0]), load8<false>(sn, c[0], si[0]);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (MODE == kNeighbours && c[u] + 8 <= R) {
          const float4 f = load_any<float4>(cs + c[u] / 2), h = load_any<float4>(sn + c[u] / 2);
          co[u][0] = f.x, co[u][1] = f.y, co[u][2] = f.z, co[u][3] = f.w;
          si[u][0] = h.x, si[u][1] = h.y, si[u][2] = h.z, si[u][3] = h.w;
          continue;
        }
#pragma unroll
        for (int j = 0; j < (MODE == kNeighbours ? 4 : 8); ++j) {
          const int col = c[u] + (MODE == kNeighbours ? 2 * j : j);
          if (col >= R) break;
          const int i = MODE == kNeighbours ? col / 2 : col < R / 2 ? col : col - R / 2;
          co[u][j] = cs[i], si[u][j] = sn[i];
        }
      }
    }
    if (!known) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) co[u][j] = __builtin_nanf("");
    }
  }
  // The row's norm, over L lanes, and rotation.  turn: D numbers of LDS of the row's own (kHalvesLds).
  __device__ __forceinline__ void finish(const AppendArgs &a, int L, real (&y)[2][8], real *turn) const {
    const int D = static_cast<int>(a.pool.D), R = static_cast<int>(a.R);
    if (a.norm) {
      real ss = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_elementwise_fma(y[u][j], y[u][j], ss);
      for (int d = 1; d < L; d <<= 1) ss += __shfl_xor(ss, d);
      const real mean = ss / D + static_cast<real>(a.eps);
      bool plain = true;
      if constexpr (std::is_same_v<real, float>) {
        // squares past the range of f32, or so small that what it lost of them (256 times 2^-149) may count: in f64
        plain = mean > 0x1p-90f && mean < __builtin_inff();
        if (__builtin_expect(__any(!plain), 0)) {
          double sum = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(y[u][j]), static_cast<double>(y[u][j]), sum);
          for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d);
          const double mean64 = sum / D + static_cast<double>(a.eps);
          const double root = mean64 < __builtin_inf() ? inverse_root(mean64) : 1.0 / mean64;
          if (!plain) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 8; ++j) y[u][j] = static_cast<float>(y[u][j] * root * g[u][j]);
          }
        }
      }
      if (plain) {
        const real root = inverse_root(mean);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) y[u][j] = y[u][j] * root * static_cast<real>(g[u][j]);
      }
    }
    if constexpr (MODE == kNeighbours) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          if (c[u] + j >= R) break;
          const real p = y[u][j], q = y[u][j + 1], cj = co[u][j / 2], sj = si[u][j / 2];
          y[u][j] = __builtin_elementwise_fma(p, cj, -(q * sj));
          y[u][j + 1] = __builtin_elementwise_fma(q, cj, p * sj);
        }
    } else if constexpr (MODE == kHalves) {
      if (rotated) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const real p = y[0][j], q = y[1][j], cj = co[0][j], sj = si[0][j];
          y[0][j] = __builtin_elementwise_fma(p, cj, -(q * sj));
          y[1][j] = __builtin_elementwise_fma(q, cj, p * sj);
        }
      }
    } else if constexpr (MODE == kHalvesLds) {
      if (in) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) turn[c[u] + j] = y[u][j];
      }
      wave_sync();
      if (in) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = c[u] + j;
            if (col >= R) break;
            const bool low = col < R / 2;
            const real other = turn[low ? col + R / 2 : col - R / 2], cj = co[u][j], sj = si[u][j];
            y[u][j] = low ? y[u][j] * cj - other * sj : y[u][j] * cj + other * sj;
          }
      }
      wave_sync();   // the next head's row comes to the same place
    }
  }
};

// What decides a scale byte of |v|: its high word, rounded up.  Infinity and NaN are last.
__device__ __forceinline__ uint32_t size_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (static_cast<uint32_t>(b >> 32) & 0x7FFFFFFFu) + (static_cast<uint32_t>(b) != 0);
}
constexpr uint32_t kNotFinite = 0x7FF00000u;

// The scale byte of a block whose largest magnitude has size t: the smallest
// e + 127 >= 0 with it <= 127 2^e; 127 is 1.984375 2^6.
__device__ __forceinline__ int scale_byte(uint32_t t) {
  if (t >= kNotFinite) return 255;
  const int e = static_cast<int>(t >> 20) - 1023 - 6;
  const bool over = (t & 0xFFFFFu) > 0xFC000u;   // 0.984375 of a mantissa
  const int b8 = max(e + (over ? 1 : 0) + 127, 0);
  return min(b8, 255);
}

// Four codes -> the same at a scale 2^shift times as large.
__device__ __forceinline__ uint32_t coarser(uint32_t w, int shift) {
  const float f = ldexpf(1.0f, -min(shift, 126));
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = static_cast<int8_t>(w >> (8 * j));
    o |= (static_cast<uint32_t>(static_cast<int>(rintf(static_cast<float>(c) * f))) & 0xFFu) << (8 * j);
  }
  return o;
}

// Bytes 0 .. 3 of four words, one a column -> four words, one a byte place.
__device__ __forceinline__ void turn4(const uint32_t (&w)[4], uint32_t (&o)[4]) {
  const uint32_t a = perm_b32(w[1], w[0], 0x05010400u), b = perm_b32(w[3], w[2], 0x05010400u);
  const uint32_t c = perm_b32(w[1], w[0], 0x07030602u), d = perm_b32(w[3], w[2], 0x07030602u);
  o[0] = perm_b32(b, a, 0x05040100u), o[1] = perm_b32(b, a, 0x07060302u);
  o[2] = perm_b32(d, c, 0x05040100u), o[3] = perm_b32(d, c, 0x07060302u);
}

// What a call touches of a block, and its scale.
struct Open {
  int had, have;      // tokens 0 .. had - 1 were there, had .. have - 1 are new
  int old, byte;      // the scale bytes before and now
  __device__ __forceinline__ void set(int need) { byte = had ? max(old, need) : need; }
  // powers of two that the codes of what was there lose
  __device__ __forceinline__ int shift() const { return had && byte != 255 ? byte - old : 0; }
};

// Workgroups of a launch: for each slot of a block the keys, key_groups times `heads`
// heads, and the values, value_groups times as many heads as 256 lanes have; then
// query rows, 256 / L tokens and `per` heads each.
struct AppendPlan {
  uint32_t key_groups, value_groups, blocks, query_groups;
  int log2_L, heads, per;
};

template <bool BF16, bool OB, int MODE>
__global__ __launch_bounds__(kThreads, MODE == kHalvesLds ? 2 : 3) void kv_append_kernel(AppendArgs a, AppendPlan p, uint32_t first) {
  extern __shared__ double lds[];
  __shared__ uint32_t tops[16];
  __shared__ uint32_t value_tops[kThreads / 4];
  const uint32_t id = first + blockIdx.x;
  const int D = static_cast<int>(a.pool.D), L = 1 << p.log2_L, lane = threadIdx.x & (L - 1), row_of = threadIdx.x >> p.log2_L;
  const int Hk = static_cast<int>(a.pool.Hk);

  if (id >= p.blocks) {   // queries
    const uint32_t tile = (id - p.blocks) / p.query_groups, group = (id - p.blocks) % p.query_groups;
    const int64_t t = static_cast<int64_t>(tile) * (kThreads >> p.log2_L) + row_of;
    const bool in_rows = t < a.seqs.T;
    const Sequence s = find_sequence<1>(a.seqs, in_rows ? static_cast<uint32_t>(t) : 0, [&](uint32_t start, int) { return start; });
    const bool live = in_rows && s.i >= 0 && t - s.row < s.n;   // not behind the last sequence
    const Lane<float, MODE> ln(a, a.gq, lane, live ? s.first + (t - s.row) : -1);
    const int h0 = static_cast<int>(group) * p.per, h1 = min(h0 + p.per, static_cast<int>(a.Hq));
    const bool mine = live && ln.in;
    Run8<BF16> x[2];
    x[0].zero(), x[1].zero();
    float y[2][8];
    auto fetch = [&](int h) {
      if (mine)
        for (int u = 0; u < 2; ++u) x[u].load(a.q, t * a.q_t + h * a.q_h + ln.c[u]);
    };
    fetch(h0);
    for (int h = h0; h < h1; ++h) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[u][j] = element(x[u], j);
      if (h + 1 < h1) fetch(h + 1);
      ln.finish(a, L, y, reinterpret_cast<float *>(lds) + row_of * D);
      if (mine)
        for (int u = 0; u < 2; ++u) store8<OB>(a.qo, (t * a.Hq + h) * D + ln.c[u], y[u]);
    }
    return;
  }

  const uint32_t groups = p.key_groups + p.value_groups, group = id % groups;
  const BlockOf w(a.seqs, id / groups);
  const Sequence &s = w.s;
  if (s.i < 0) return;
  const int begin = w.b * kKvBlock;
  Open open = {max(max(s.first, 0) - begin, 0), min(s.len - begin, kKvBlock), 0, 0};
  const int64_t row0 = static_cast<int64_t>(s.row) + begin - s.first;   // of the block's token 0
  // The page is looked up while the rows are on their way; no such page: the tokens are dropped.
  const int64_t block0 = block_at(a.pool, s.i, w.b, 0);
  const int64_t unit = kKvBlock * D;

  if (group >= p.key_groups) {   // values: four columns of a head a lane
    const int quads = D / 4, each = kThreads / quads, hh = threadIdx.x / quads, c = 4 * (threadIdx.x - hh * quads);
    const int h = static_cast<int>(group - p.key_groups) * each + hh;
    const bool mine = hh < each && h < Hk;
    if (threadIdx.x < kThreads / 4) value_tops[threadIdx.x] = 0;
    using Raw = std::conditional_t<BF16, uint2, uint4>;   // four columns of a token
    Raw x[kKvBlock];
#pragma unroll
    for (int k = 0; k < kKvBlock; ++k) {
      x[k] = Raw{};
      if (k < open.had || k >= open.have || !mine) continue;
      const int64_t i0 = (row0 + k) * a.v_t + h * a.v_h + c;
      x[k] = load_any<Raw>(static_cast<const char *>(a.v) + i0 * (BF16 ? 2 : 4));
    }
    auto value = [&](int k, int i) {   // bits of an f32
      if constexpr (BF16) return (i < 2 ? x[k].x : x[k].y) << (i & 1 ? 0 : 16) & 0xFFFF0000u;
      else return i == 0 ? x[k].x : i == 1 ? x[k].y : i == 2 ? x[k].z : x[k].w;
    };
    if (block0 < 0) return;
    const int64_t at = block0 + (static_cast<int64_t>(mine ? h : 0) << a.pool.page_blocks_log2);
    uint4 codes[4] = {};
    if (open.had) {
      open.old = a.pool.vs[at];
      if (mine)
#pragma unroll
        for (int i = 0; i < 4; ++i) codes[i] = load16(a.pool.v + at * unit + (c + i) * 16);
    }
    uint32_t top = 0;   // magnitudes order as their bits; NaN and infinity come last
#pragma unroll
    for (int k = 0; k < kKvBlock; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, value(k, i) & 0x7FFFFFFFu);
    __syncthreads();
    if (mine) atomicMax(&value_tops[hh], top);
    __syncthreads();
    if (!mine) return;
    top = value_tops[hh];
    open.set(scale_byte(size_of(static_cast<double>(__uint_as_float(top)))));
    // x / 2^e, which the sum with 3 2^22 rounds to the nearest whole number, in its low bits
    const float f = ldexpf(1.0f, 127 - open.byte);
    const int shift = open.shift();
#pragma unroll
    for (int k = 0; k < kKvBlock; k += 4) {
      const int had = min(max(open.had - k, 0), 4);   // bytes of these words that the block has
      const uint32_t mask = had == 4 ? ~0u : (1u << (8 * had)) - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t q[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) q[m] = __float_as_uint(__builtin_fmaf(__uint_as_float(value(k + m, i)), f, 0x1.8p23f));
        uint32_t w = perm_b32(perm_b32(q[3], q[2], 0x0C0C0400u), perm_b32(q[1], q[0], 0x0C0C0400u), 0x05040100u);
        if (open.byte == 255) w = 0;
        uint32_t &o = k == 0 ? codes[i].x : k == 4 ? codes[i].y : k == 8 ? codes[i].z : codes[i].w;
        o = open.had ? (w & ~mask) | ((shift > 0 ? coarser(o, shift) : o) & mask) : w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(a.pool.v + at * unit + (c + i) * 16) = codes[i];
    if (c == 0) a.pool.vs[at] = static_cast<uint8_t>(open.byte);
    return;
  }

  // keys: 16 tokens of 16 / L heads at a time
  const int tok = row_of & 15, hh = row_of >> 4, at_once = 16 >> p.log2_L;
  const bool live = tok >= open.had && tok < open.have;
  const Lane<double, MODE> ln(a, a.gk, lane, begin + tok);
  const int h0 = static_cast<int>(group) * p.heads, h1 = min(h0 + p.heads, Hk);
  Run8<BF16> x[2];
  x[0].zero(), x[1].zero();
  auto fetch = [&](int h) {
    if (h < h1 && live && ln.in)
      for (int u = 0; u < 2; ++u) x[u].load(a.k, (row0 + tok) * a.k_t + h * a.k_h + ln.c[u]);
  };
  fetch(h0 + hh);
  if (block0 < 0) return;
  for (int hb = h0; hb < h1; hb += at_once) {
    const int h = hb + hh;
    const bool mine = h < h1;
    const int64_t at = block0 + (static_cast<int64_t>(mine ? h : h0) << a.pool.page_blocks_log2);
    if (threadIdx.x < 16) tops[threadIdx.x] = 0;
    open.old = open.had ? a.pool.ks[at] : 0;   // before the barrier behind which it is written
    double y[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) y[u][j] = element(x[u], j);
    fetch(h + at_once);
    ln.finish(a, L, y, lds + row_of * D);
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, size_of(y[u][j]));
    if (!(mine && live && ln.in)) top = 0;
    for (int d = 1; d < min(16 * L, 64); d <<= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    __syncthreads();
    if ((threadIdx.x & (min(16 * L, 64) - 1)) == 0) atomicMax(&tops[hh], top);
    __syncthreads();
    open.set(scale_byte(tops[hh]));
    const int shift = open.shift();
    if (mine && ln.in) {
      // times 2^(127 - byte), exactly; the sum with 3 2^51 is rounded to the nearest whole number, in its low bits
      const double f = ldexp(1.0, 127 - open.byte);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint2 *place = reinterpret_cast<uint2 *>(a.pool.k + at * unit + (ln.c[u] / 16) * 256 + tok * 16 + (ln.c[u] & 8));
        if (live) {
          uint32_t d[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t q = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, __builtin_fma(y[u][j], f, 0x1.8p52)));
            d[j / 4] |= (q & 0xFFu) << (8 * (j & 3));
          }
          *place = open.byte == 255 ? make_uint2(0, 0) : make_uint2(d[0], d[1]);
        } else if (tok < open.had && shift > 0) {
          const uint2 d = *place;
          *place = make_uint2(coarser(d.x, shift), coarser(d.y, shift));
        }
      }
      if (tok == 0 && lane == 0) a.pool.ks[at] = static_cast<uint8_t>(open.byte);
    }
    __syncthreads();   // before the next heads' maxima
  }
}

// Blocks as bf16 or f32 rows: keys 16 columns of a token a lane, values four columns
// of 16 tokens.
template <bool OB>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvPool pool, KvSeqs seqs, AppendPlan p, void *ko, void *vo,
                                                           uint32_t first) {
  const uint32_t id = first + blockIdx.x, groups = p.key_groups + p.value_groups, group = id % groups;
  const BlockOf w(seqs, id / groups);
  const Sequence &s = w.s;
  if (s.i < 0) return;
  const int D = static_cast<int>(pool.D), Hk = static_cast<int>(pool.Hk), begin = w.b * kKvBlock;
  const int lo = max(s.first - begin, 0), hi = min(s.len - begin, kKvBlock);   // tokens that are asked for
  const int64_t row0 = static_cast<int64_t>(s.row) + begin - s.first, unit = kKvBlock * D;
  const int64_t block0 = block_at(pool, s.i, w.b, 0);
  const bool known = block0 >= 0;            // no such page: NaN
  // a code's value under scale byte b: 2^(b - 127) in f32, subnormal for b = 0
  auto step = [](int b) {
    return b == 255 ? __builtin_nanf("") : __uint_as_float(b ? static_cast<uint32_t>(b) << 23 : 0x400000u);
  };
  auto at_head = [&](int h) { return (known ? block0 : 0) + (static_cast<int64_t>(h) << pool.page_blocks_log2); };
  if (group >= p.key_groups) {
    const int quads = D / 4, each = kThreads / quads, hh = threadIdx.x / quads, c = 4 * (threadIdx.x - hh * quads);
    const int h = static_cast<int>(group - p.key_groups) * each + hh;
    if (hh >= each || h >= Hk) return;
    uint4 codes[4] = {};
    if (known)
#pragma unroll
      for (int i = 0; i < 4; ++i) codes[i] = load16(pool.v + at_head(h) * unit + (c + i) * 16);
    const float f = step(known ? pool.vs[at_head(h)] : 255);
#pragma unroll
    for (int k = 0; k < kKvBlock; k += 4) {
      uint32_t columns[4], words[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) columns[i] = k == 0 ? codes[i].x : k == 4 ? codes[i].y : k == 8 ? codes[i].z : codes[i].w;
      turn4(columns, words);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (k + m < lo || k + m >= hi) continue;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = static_cast<float>(static_cast<int8_t>(words[m] >> (8 * i))) * f;
        const int64_t o = ((row0 + k + m) * Hk + h) * D + c;
        if constexpr (OB) store_any(static_cast<uint16_t *>(vo) + o, make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])));
        else store_any(static_cast<float *>(vo) + o, make_float4(y[0], y[1], y[2], y[3]));
      }
    }
    return;
  }
  const int L = 1 << p.log2_L, lane = threadIdx.x & (L - 1), row_of = threadIdx.x >> p.log2_L;
  const int tok = row_of & 15, at_once = 16 >> p.log2_L, h0 = static_cast<int>(group) * p.heads, h1 = min(h0 + p.heads, Hk);
  if (tok < lo || tok >= hi || lane >= D / 16) return;
  for (int h = h0 + (row_of >> 4); h < h1; h += at_once) {
    uint4 codes = make_uint4(0, 0, 0, 0);
    if (known) codes = load16(pool.k + at_head(h) * unit + lane * 256 + tok * 16);
    const float f = step(known ? pool.ks[at_head(h)] : 255);
    const uint32_t words[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = static_cast<float>(static_cast<int8_t>(words[2 * u + j / 4] >> (8 * (j & 3)))) * f;
      store8<OB>(ko, ((row0 + tok) * Hk + h) * D + 16 * lane + 8 * u, y);
    }
  }
}

// Shares for D columns, Hk heads and T rows: a workgroup has more than one set of
// heads only where there are enough workgroups without.
AppendPlan plan(const KvPool &pool, const KvSeqs &seqs, int64_t Hq) {
  AppendPlan p = {};
  while ((16 << p.log2_L) < pool.D) ++p.log2_L;
  const int at_once = 16 >> p.log2_L;
  const int64_t slots = block_slots(seqs.T, seqs.N), sets = (pool.Hk + at_once - 1) / at_once;
  auto share = [](int64_t all, int64_t most) {
    const int64_t n = all / 1024;
    return n < 1 ? 1 : n < most ? n : most;
  };
  p.heads = static_cast<int>(share(slots * sets, sets < 8 ? sets : 8) * at_once);
  p.key_groups = static_cast<uint32_t>((pool.Hk + p.heads - 1) / p.heads);
  const int64_t each = kThreads / (pool.D / 4);
  p.value_groups = static_cast<uint32_t>((pool.Hk + each - 1) / each);
  p.blocks = static_cast<uint32_t>(slots * (p.key_groups + p.value_groups));
  const int64_t tiles = (seqs.T + (kThreads >> p.log2_L) - 1) / (kThreads >> p.log2_L);
  p.per = static_cast<int>(share(tiles * Hq, Hq < 8 ? (Hq < 1 ? 1 : Hq) : 8));
  p.query_groups = static_cast<uint32_t>((Hq + p.per - 1) / p.per);
  return p;
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, bool bf16, bool out_bf16, hipStream_t st) {
  const AppendPlan p = plan(a.pool, a.seqs, a.Hq);
  const int64_t tiles = (a.seqs.T + (kThreads >> p.log2_L) - 1) / (kThreads >> p.log2_L);
  const int64_t all = p.blocks + (a.q ? tiles * p.query_groups : 0), most = max_groups(kThreads);
  const int mode = !a.table ? kPlain : a.neighbours ? kNeighbours : a.R % 16 == 0 ? kHalves : kHalvesLds;
  const size_t lds = mode == kHalvesLds ? (kThreads >> p.log2_L) * a.pool.D * sizeof(double) : 0;
  auto go = [&](auto kernel) {
    for (int64_t first = 0; first < all; first += most)
      kernel<<<static_cast<unsigned>(all - first < most ? all - first : most), kThreads, lds, st>>>(a, p, static_cast<uint32_t>(first));
  };
  auto pick = [&](auto in, auto out) {
    constexpr bool I = decltype(in)::value, O = decltype(out)::value;
    switch (mode) {
      case kPlain: return go(kv_append_kernel<I, O, kPlain>);
      case kNeighbours: return go(kv_append_kernel<I, O, kNeighbours>);
      case kHalves: return go(kv_append_kernel<I, O, kHalves>);
      default: return go(kv_append_kernel<I, O, kHalvesLds>);
    }
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (bf16) out_bf16 ? pick(yes, yes) : pick(yes, no);
  else out_bf16 ? pick(no, yes) : pick(no, no);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvPool &pool, const KvSeqs &seqs, void *ko, void *vo, bool out_bf16, hipStream_t st) {
  const AppendPlan p = plan(pool, seqs, 0);
  const int64_t all = p.blocks, most = max_groups(kThreads);
  const auto kernel = out_bf16 ? kv_read_kernel<true> : kv_read_kernel<false>;
  for (int64_t first = 0; first < all; first += most)
    kernel<<<static_cast<unsigned>(all - first < most ? all - first : most), kThreads, 0, st>>>(
        pool, seqs, p, ko, vo, static_cast<uint32_t>(first));
  return hipGetLastError();
}

}  // namespace q4

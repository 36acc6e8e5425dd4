// Attention over the paged 8-bit cache: for a query row at position p and the
// keys j <= p with j > p - window or j < sinks,
//   s_j = scale q . k_j,  y = sum_j exp(s_j) v_j / sum_j exp(s_j)
// in one pass over the keys with the running maximum and sum of the softmax.
//
// Products go through the f16 matrix instructions: int8 codes are halves
// exactly; a query row is scaled by a power of two to a maximum between 2^14
// and 2^15 and rounded to halves (11 bits, exact for bf16 down to 2^-25 of the
// row's maximum; f32 rows are two halves, 22 bits, at twice the products), and so
// are the weights exp(s), times the power of two that is their values' scale: two
// halves (22 bits down to 2^-24 of the largest such product, half a step of 2^-34
// of it below) for f32 queries or results, and for bf16 where a sequence has up to
// 16 rows of a key head, whose time is the cache's bytes (64 tokens of up to 8192
// keys 104 us, with one half 103, whose bf16 results differ in every 15th number).
// More bf16 rows have one half, 11 bits (2^-33): their time is the products' (512
// rows of 4096 keys 84 us, with two halves 95, and no registers for two in tiles of
// 128 columns), and against 64 bits it adds 0.8 % to the error that bf16 results
// have.  Maximum, sum and results are f32; what
// is subtracted from the scores are whole powers of two that may lag behind the
// maximum, so that results are seldom rescaled, and exactly.
//
// S^T = K Q^T and Y^T = V^T P^T, with the query rows as the second operands'
// rows, so that a lane's results belong to one query row.  The first product's
// rows are keys in an order that leaves a lane with the 16 scores of one block, in
// order: they are, rounded, its operand of the second product, whose other
// operand is 16 tokens of a value column a lane, as the cache has them.  Neither
// weights nor values change lanes.  Few rows (here): 16 x 16 x 32 instructions,
// lane (r, q) for query row r and block q of four; row r of the first product b
// is token 4 b + r mod 4 of block r / 4.  Many (attention_tiled.hip): 32 x 32 x
// 16, lane (c, h) and two blocks; row 8 a + 4 h + b is token 4 a + b of block h.
#include "attn_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256, kWaves = 4, kRows = 16, kMaxSplits = 64;

// Where the results begin behind a, d and l of `splits` parts of `all` rows, on 16 bytes.
__host__ __device__ constexpr int64_t results_at(int64_t splits, int64_t all) { return (3 * splits * all + 3) / 4 * 4; }

// Few rows a sequence: a workgroup has 16 rows of one key head and a share of
// their keys; its four waves share those out again, 64 keys a step straight from
// the cache to registers, and meet in LDS.  A step's keys are loaded as soon as
// those of the step before are multiplied, its values likewise.  Bound by memory
// for long contexts: one token, 131071 keys of 32 + 8 heads of 128 (268 MB) 54 us,
// 5.0 TB/s; 64 tokens of up to 8192 keys (462 MB) 100 us, 4.6 TB/s.  By the chain of
// loads (sequence, page, scales, codes) and the launch for short ones: 16 keys 7.5 us
// with the call.  Eight waves a workgroup take one more and, as a CU then has one
// workgroup, twice the time with many sequences (64 of 64 keys 16.6 us against 8.6).  parts: a, d, l
// and results of splits x rows for combine_kernel, or null with one split.
template <int NV, bool TWO_Q, bool TWO_W>   // 16 NV columns; queries and weights as two halves
__global__ __launch_bounds__(kThreads, NV <= 8 ? 2 : 1) void attention_rows_kernel(AttnArgs a, Types types, int splits,
                                                                                 float *parts, uint32_t first) {
  constexpr int NS = (NV + 3) / 4, D = 16 * NV;
  __shared__ float as[kWaves][kRows], ds[kWaves][kRows], ls[kWaves][kRows];
  __shared__ __attribute__((aligned(16))) float meet[kWaves - 1][kRows][D + 4];
  const uint32_t Hk = static_cast<uint32_t>(a.pool.Hk), G = static_cast<uint32_t>(a.G);
  const int split = static_cast<int>(blockIdx.x % splits);
  const int head = static_cast<int>(blockIdx.x / splits % Hk);
  const RowTile<kRows> tile(a.seqs, first + blockIdx.x / splits / Hk, G);
  if (tile.s.i < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 15, q4 = lane >> 4;
  const int rows = min(tile.rows - tile.r0, kRows);
  const int r = tile.r0 + (c < rows ? c : rows - 1), t = static_cast<int>(static_cast<uint32_t>(r) / G);
  const int64_t row = tile.s.row + t, qh = head * static_cast<int>(G) + (r - t * static_cast<int>(G));
  // lengths are int32, and so positions
  const int p0 = uniform(tile.s.first + tile.r0 / static_cast<int>(G));
  const int p1 = uniform(tile.s.first + (tile.r0 + rows - 1) / static_cast<int>(G)), pos = tile.s.first + t;
  const Sight sight(a.window, a.sinks);
  const KeyBlocks keys(p0, p1, sight, a.pool);

  const int steps = (keys.count + 3) / 4;
  const int w0 = static_cast<int>(static_cast<int64_t>(steps) * (split * kWaves + wave) / (splits * kWaves));
  const int w1 = static_cast<int>(static_cast<int64_t>(steps) * (split * kWaves + wave + 1) / (splits * kWaves));

  // blocks of this wave's keys, one a lane, a round of 16 steps ahead: pages, then scales
  struct Info {
    int at, bytes, blk;
  };
  const int32_t *pages = a.pool.pages + tile.s.i * a.pool.width;
  const int page_mask = (1 << a.pool.page_blocks_log2) - 1;
  auto page_of = [&](int round) {
    const int v = 4 * w0 + 64 * round + lane;
    const int64_t p = v < keys.count ? keys.block(v) >> a.pool.page_blocks_log2 : a.pool.width;
    return p < a.pool.width ? pages[p] : -1;
  };
  auto info_of = [&](int round, int page) {
    const int v = 4 * w0 + 64 * round + lane;
    Info f = {0, 0xFFFF, keys.block(v)};     // a page that is not there: NaN
    if (v < keys.count && page >= 0 && page < a.pool.n_pages) {
      f.at = ((page * static_cast<int>(Hk) + head) << a.pool.page_blocks_log2) + (f.blk & page_mask);
      f.bytes = a.pool.ks[f.at] | a.pool.vs[f.at] << 8;
    }
    return f;
  };

  State<f32x4, NV, 4, TWO_W> st;
  if (w0 < w1) {
    Info cur = info_of(0, page_of(0)), next = {};
    int page = -1;
    if (w1 - w0 > 16) page = page_of(1);
    uint4 k[4][NS], v[NV];
    // the four blocks of step s of a round
    auto load_keys = [&](int s) {
      // token 4 b + c mod 4 of block c / 4, 16 columns; columns past D, which the query has as 0, are the last ones again
      const int at = __shfl(cur.at, 4 * s + (c >> 2));
      const int8_t *p = a.pool.k + static_cast<int64_t>(at) * (kKvBlock * D) + (c & 3) * 16;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int chunk = 4 * j + 3 < NV ? 4 * j + q4 : min(4 * j + q4, NV - 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) k[b][j] = load16(p + chunk * 256 + b * 64);
      }
    };
    auto load_values = [&](int s) {
      const int at = __shfl(cur.at, 4 * s + q4);
      const int8_t *p = a.pool.v + static_cast<int64_t>(at) * (kKvBlock * D) + c * 16;
#pragma unroll
      for (int d = 0; d < NV; ++d) v[d] = load16(p + d * 256);
    };
    load_keys(0);
    load_values(0);
    Query<NS, 4, TWO_Q> q;
    q.load(a, types, row * a.q_t + qh * a.q_h, true, q4);
    for (int s = w0; s < w1; ++s) {
      const int l = (s - w0) & 15;
      const int bytes = __shfl(cur.bytes, 4 * l + q4), k0 = __shfl(cur.blk, 4 * l + q4) * kKvBlock;
      f32x16 x;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f32x4 acc = {};
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const uint4 lo = codes_to_f16(k[b][j].x, k[b][j].y), hi = codes_to_f16(k[b][j].z, k[b][j].w);
          acc = mfma_f16_16x16x32(lo, q.hi[2 * j], acc);
          acc = mfma_f16_16x16x32(hi, q.hi[2 * j + 1], acc);
          if constexpr (TWO_Q) {
            acc = mfma_f16_16x16x32(lo, q.lo[2 * j], acc);
            acc = mfma_f16_16x16x32(hi, q.lo[2 * j + 1], acc);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * b + j] = acc[j];
      }
      // each phase by itself: loads go out early, and codes become halves where they are used, which keeps registers free
      __builtin_amdgcn_sched_barrier(0);
      if (l == 0 && w1 - s > 16) {
        const int round = (s - w0) / 16 + 1;
        next = info_of(round, page);
        if (w1 - s > 32) page = page_of(round + 1);
      }
      if (l == 15) cur = next;
      if (s + 1 < w1) load_keys((l + 1) & 15);
      __builtin_amdgcn_sched_barrier(0);
      typename decltype(st)::Keys w[1];
      if (__all(sight.whole(p0, p1, k0)))
        w[0].template scores<false>(x, q.factor, bytes & 255, bytes >> 8, [](int) { return false; });
      else
        w[0].template scores<true>(x, q.factor, bytes & 255, bytes >> 8, [&](int j) { return sight.hides(pos, k0 + j); });
      st.weights(w);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < NV; ++d) {
        const uint4 lo = codes_to_f16(v[d].x, v[d].y), hi = codes_to_f16(v[d].z, v[d].w);
        st.y[d] = mfma_f16_16x16x32(lo, w[0].p[0], st.y[d]);
        st.y[d] = mfma_f16_16x16x32(hi, w[0].p[1], st.y[d]);
        if constexpr (TWO_W) {
          st.y[d] = mfma_f16_16x16x32(lo, w[0].rest[0], st.y[d]);
          st.y[d] = mfma_f16_16x16x32(hi, w[0].rest[1], st.y[d]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (s + 1 < w1) load_values((l + 1) & 15);
    }
  }

  // the four waves' parts relative to the same powers, then their sums in order, by the first wave
  st.l = row_sum<4>(st.l);
  if (q4 == 0) as[wave][c] = st.a, ds[wave][c] = st.d, ls[wave][c] = st.l;
  __syncthreads();
  float ma = as[0][c], md = -__builtin_inff(), l = 0.0f;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) ma = fmaxf(ma, as[w][c]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    md = fmaxf(md, lag(as[w][c], ds[w][c], ma));
    l += ls[w][c] * rescale(as[w][c], ls[w][c], ma);
  }
  const float f = rescale(st.a, st.d, st.l, ma, md);
#pragma unroll
  for (int d = 0; d < NV; ++d) st.y[d] *= f;
  if (wave > 0 && c < rows) {
#pragma unroll
    for (int d = 0; d < NV; ++d) *reinterpret_cast<f32x4 *>(&meet[wave - 1][c][16 * d + 4 * q4]) = st.y[d];
  }
  __syncthreads();
  if (wave > 0 || c >= rows) return;
  const Quotient quotient(md, l, decltype(st)::kOffset);
  const int64_t all = a.seqs.T * a.Hq, out = row * a.Hq + qh;
#pragma unroll
  for (int d = 0; d < NV; ++d) {
    const int col = 16 * d + 4 * q4;
    f32x4 sum = st.y[d];
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) sum += *reinterpret_cast<const f32x4 *>(&meet[w][c][col]);
    if (parts)
      *reinterpret_cast<f32x4 *>(parts + results_at(splits, all) + (split * all + out) * D + col) = sum;
    else
      store4(a.y, types.out_bf16, out * D + col, quotient(sum[0]), quotient(sum[1]), quotient(sum[2]), quotient(sum[3]));
  }
  if (parts && q4 == 0) {
    parts[split * all + out] = ma;
    parts[(splits + split) * all + out] = md;
    parts[(2 * splits + split) * all + out] = l;
  }
}

// Joins the splits of rows: D / 4 lanes times up to `splits` a row, which share the
// splits out and meet in LDS, in a fixed order; as many rows a workgroup as fit.
__global__ __launch_bounds__(kThreads) void combine_kernel(AttnArgs a, Types types, int offset, int splits, int groups,
                                                           int rows, const float *parts, int64_t first) {
  // rows x splits, at most: a split's factor and its part of l, and its row's d
  __shared__ float factors[kMaxSplits], terms[kMaxSplits], ds[kMaxSplits];
  __shared__ f32x4 sums[kThreads];
  __shared__ float ls[kThreads];
  const int64_t all = a.seqs.T * a.Hq, out0 = first + blockIdx.x * static_cast<int64_t>(rows);
  const int D = static_cast<int>(a.pool.D), quads = D / 4, each = quads * groups;
  const int64_t from = Sequence::clamp(a.seqs.starts[0], a.seqs.T) * a.Hq;
  const int64_t to = Sequence::clamp(a.seqs.starts[a.seqs.N], a.seqs.T) * a.Hq;
  if (threadIdx.x < kMaxSplits) {   // the first wave: a split a lane
    const int lane = threadIdx.x, row = lane / splits, s = lane - row * splits;
    const int64_t out = out0 + row;
    const bool has = row < rows && out < all;
    const float a1 = has ? parts[s * all + out] : -__builtin_inff(), d1 = has ? parts[(splits + s) * all + out] : 0.0f;
    const float l1 = has ? parts[(2 * splits + s) * all + out] : 0.0f;
    // the largest of the row's splits: of 2, 4, 8, ... from each one on, round and round
    auto row_max = [&](float v) {
      for (int n = 1; n < splits; n *= 2) {
        const int at = s + n < splits ? lane + n : lane + n - splits;
        v = fmaxf(v, __shfl(v, at));
      }
      return v;
    };
    const float ma = row_max(a1), md = row_max(lag(a1, d1, ma));
    factors[lane] = rescale(a1, d1, l1, ma, md);
    terms[lane] = l1 * rescale(a1, l1, ma);
    ds[lane] = md;
  }
  __syncthreads();
  const int r = threadIdx.x / each, x = threadIdx.x - r * each, g = x / quads, col = 4 * (x - g * quads);
  const int64_t out = out0 + r;
  // rows in front of the first sequence or behind the last are left as they were
  const bool live = r < rows && out >= from && out < to;
  float l = 0.0f;
  f32x4 sum = {};
  if (live) {
#pragma unroll 4
    for (int s = g; s < splits; s += groups) {
      const f32x4 o = *reinterpret_cast<const f32x4 *>(parts + results_at(splits, all) + (s * all + out) * D + col);
      sum += o * factors[r * splits + s];
      l += terms[r * splits + s];
    }
  }
  sums[threadIdx.x] = sum;
  ls[threadIdx.x] = l;
  __syncthreads();
  if (!live || g > 0) return;
  for (int i = 1; i < groups; ++i) sum += sums[threadIdx.x + i * quads], l += ls[threadIdx.x + i * quads];
  const Quotient q(ds[r * splits], l, offset);
  store4(a.y, types.out_bf16, out * D + col, q(sum[0]), q(sum[1]), q(sum[2]), q(sum[3]));
}

template <int NV, bool TWO_Q, bool TWO_W>
void go_rows(const AttnArgs &a, const Types &t, const AttnPlan &p, float *ws, hipStream_t st) {
  const int64_t slots = tile_slots(a.seqs.T, a.seqs.N, a.G, kRows), each = a.pool.Hk * p.splits;
  const int64_t most = max_groups(kThreads);
  for (int64_t first = 0; first < slots; first += most / each) {   // slots of a launch
    const int64_t n = slots - first < most / each ? slots - first : most / each;
    attention_rows_kernel<NV, TWO_Q, TWO_W><<<static_cast<unsigned>(n * each), kThreads, 0, st>>>(
        a, t, p.splits, p.splits > 1 ? ws : nullptr, static_cast<uint32_t>(first));
  }
  if (p.splits == 1) return;
  const int64_t all = a.seqs.T * a.Hq;
  const int quads = 4 * NV, groups = p.splits < kThreads / quads ? p.splits : kThreads / quads, rows = kThreads / (quads * groups);
  const int64_t per = most * rows;
  for (int64_t first = 0; first < all; first += per) {   // rows of a launch
    const int64_t n = all - first < per ? all - first : per;
    combine_kernel<<<static_cast<unsigned>((n + rows - 1) / rows), kThreads, 0, st>>>(
        a, t, State<f32x4, 1, 4, TWO_W>::kOffset, p.splits, groups, rows, ws, first);
  }
}

template <bool TWO_Q, bool TWO_W, int NV = 16>
void go(const AttnArgs &a, const Types &t, const AttnPlan &p, float *ws, hipStream_t st) {
  if (a.pool.D == 16 * NV) return go_rows<NV, TWO_Q, TWO_W>(a, t, p, ws, st);
  if constexpr (NV > 1) go<TWO_Q, TWO_W, NV - 1>(a, t, p, ws, st);
}

}  // namespace

// Rows kernel | tiles, us, of N sequences of L tokens, n of them rows, Hq / Hk heads
// of D.  bf16 with D above 64: from 128 tiles of 256 rows on (32/8 of 128: N 1 n 512 L
// 4096, 64 tiles, 88 | 126, n 1024 157 | 133, n 4096 345 | 162; 16/4 of 96, N 1 n 2048 L
// 4096, 128 tiles, 117 | 111), where a sequence half fills one (16/16 of 128, N 64 n 64 L
// 1024 128 | 128, N 16 n 128 L 2048 90 | 59).  D up to 64 from 192 on (8/1 of 64, N 1 n 4096
// L 4096, 128 tiles, 59 | 85; 32/8, N 1 n 2048 L 4096, 256 tiles, 135 | 91).  f32: from 256,
// where a sequence has two (32/8 of 64, N 16 n 128 L 2048 112 | 137, n 256 219 | 151).
// All sequences have one route: where lengths and rows differ much that costs (one token of
// 131071 keys 51, 512 rows of 4096 83, both in one call 453; 63 tokens of 4096 keys 105, a
// prompt of 4096 162, both 350).
static bool many_rows(int64_t T, int64_t N, int64_t G, int64_t Hk, int64_t D, bool two) {
  const int64_t rows = T * G / N, tiles = (rows + 255) / 256 * N * Hk;
  return two ? tiles >= 256 && rows >= 512 : tiles >= (D > 64 ? 128 : 192) && rows >= 128;
}

AttnPlan attention_plan(int64_t T, int64_t N, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len, int64_t window,
                        int64_t sinks, bool two, int path) {
  AttnPlan p = {};
  p.splits = 1;
  p.tiled = attention_tiled_ok(D, two) &&
            (path == kPathTiled || (path == kPathAuto && many_rows(T, N, Hq / Hk, Hk, D, two)));
  if (p.tiled) return p;
  const int64_t G = Hq / Hk, groups = (T * G + kRows * N - 1) / (kRows * N) * N * Hk;
  int64_t keys = max_len;
  if (window > 0 && window < keys && sinks < keys && window + sinks + 32 < keys) keys = window + sinks + 32;
  // Two workgroups a CU in all, what runs at once, or up to eight of 4096 keys or more, which even out lengths; a wave
  // at least 64 keys of what a sequence may have, and no splits below 1024 keys, where the join costs more than it gives.
  // 32 + 8 heads of 128, one token a sequence (weights of one half), two workgroups a CU and eight: 32 sequences of 1023 keys 19.5 and 26.4
  // us, of 4096 46.5 and 54.9, of 16384 189 and 192, of 1 to 16384 124 and 111 (four: 114).  One sequence of 512 keys
  // 8.4 us, in two splits 10.3; of 1023 11.0, in two 11.7, in four 10.9.
  int64_t s = (512 + groups - 1) / groups;
  const int64_t even = (2048 + groups - 1) / groups < keys / 4096 ? (2048 + groups - 1) / groups : keys / 4096;
  s = s > even ? s : even;
  const int64_t most = keys < 1024 ? 1 : keys / (64 * kWaves);
  s = s < most ? s : most;
  p.splits = static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
  p.ws = p.splits > 1 ? (results_at(p.splits, T * Hq) + p.splits * T * Hq * D) * sizeof(float) : 0;
  return p;
}

hipError_t launch_attention(const AttnArgs &a, const AttnPlan &p, bool bf16, bool out_bf16, void *ws, hipStream_t st) {
  const Types t = {bf16, out_bf16};
  if (p.tiled) return launch_attention_tiled(a, t, st);
  // up to 16 rows of a sequence and key head: bound by the cache's bytes
  const bool fine = !bf16 || !out_bf16 || a.seqs.T * a.G <= kRows * a.seqs.N;
  float *parts = static_cast<float *>(ws);
  if (!bf16) go<true, true>(a, t, p, parts, st);
  else if (fine) go<false, true>(a, t, p, parts, st);
  else go<false, false>(a, t, p, parts, st);
  return hipGetLastError();
}

}  // namespace q4

// Attention over the paged 8-bit cache: for a query row at position p and the
// keys j <= p with j > p - window or j < sinks,
//   s_j = scale q . k_j,  y = sum_j exp(s_j) v_j / sum_j exp(s_j)
// in one pass over the keys with the running maximum and sum of the softmax.
//
// Products go through the f16 matrix instructions: int8 codes are halves
// exactly; a query row is scaled by a power of two to a maximum between 2^14
// and 2^15 and rounded to halves (11 bits, exact for bf16 down to 2^-25 of the
// row's maximum), and so are the weights exp(s), times the power of two that is
// their values' scale (11 bits down to 2^-23 of the largest such product, half a
// step of 2^-33 of it below).  For f32 queries or results both come as two
// halves, 22 bits, at twice the products.  Maximum, sum and results are f32; what
// is subtracted from the scores are whole powers of two that may lag behind the
// maximum, so that results are seldom rescaled, and exactly.
//
// S^T = K Q^T and Y^T = V^T P^T on 32 x 32 x 16 instructions, a lane (c, h) for
// query row c.  Row 8 a + 4 h + b of the first product's keys is key 16 h + 4 a
// + b of the 32, so a lane ends with the 16 scores of block h, in order, and
// those are, rounded, its operand of the second product: neither the weights
// nor the values change lanes.
#include "attn_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256, kWaves = 4, kRows = 32;

// Where the results begin behind a, b and l of `splits` parts of `all` rows, on 16 bytes.
__host__ __device__ constexpr int64_t results_at(int64_t splits, int64_t all) { return (3 * splits * all + 3) / 4 * 4; }

// Few rows a sequence: a workgroup has 32 rows of one key head and a share of
// their keys; its four waves share those out again, 32 keys a step straight from
// the cache to registers, and meet in LDS.  parts: splits x rows of m, l and
// results for combine_kernel, or null with one split.
template <int ND, bool TWO>
__global__ __launch_bounds__(kThreads, ND <= 4 && !TWO ? 2 : 1) void attention_rows_kernel(AttnArgs a, Types types,
                                                                                         int splits, float *parts,
                                                                                         int64_t first) {
  constexpr int kMeet = ND < 4 ? ND : 4;   // tiles of 32 columns that meet in LDS at a time
  __shared__ float as[kWaves][kRows], bs[kWaves][kRows], ls[kWaves][kRows];
  __shared__ __attribute__((aligned(16))) float meet[kWaves - 1][kRows][32 * kMeet + 4];
  const int64_t id = first + blockIdx.x;
  const int split = static_cast<int>(id % splits);
  const int64_t head = id / splits % a.pool.Hk, slot = id / splits / a.pool.Hk;
  const int64_t G = a.Hq / a.pool.Hk;
  RowTile tile(a.seqs, slot, G, kRows);
  if (tile.i < 0) return;
  tile.i = uniform(tile.i), tile.r0 = uniform(tile.r0), tile.rows = uniform(tile.rows);
  tile.s.row = uniform(tile.s.row), tile.s.first = uniform(tile.s.first);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;
  const int D = static_cast<int>(a.pool.D);
  const int rows = tile.rows - tile.r0 < kRows ? static_cast<int>(tile.rows - tile.r0) : kRows;
  const int64_t r = tile.r0 + (c < rows ? c : rows - 1), t = r / G;
  const int64_t row = tile.s.row + t, qh = head * G + (r - t * G);
  const int64_t p0 = tile.s.first + tile.r0 / G, p1 = tile.s.first + (tile.r0 + rows - 1) / G;
  const int pos = static_cast<int>(tile.s.first + t);   // int32 lengths
  const KeyBlocks keys(p0, p1, a.window, a.sinks);
  const int64_t window = a.window > 0 ? a.window : INT64_C(1) << 40;

  const int steps = (keys.count + 1) / 2;
  const int w0 = static_cast<int>(static_cast<int64_t>(steps) * (split * kWaves + wave) / (splits * kWaves));
  const int w1 = static_cast<int>(static_cast<int64_t>(steps) * (split * kWaves + wave + 1) / (splits * kWaves));

  Query<ND, TWO> q;
  q.load(a, types, row * a.q_t + qh * a.q_h, true, h);
  State<ND, TWO> st;

  struct Tile {
    uint4 k[ND], v[ND];
  };
  for (int g0 = w0; g0 < w1; g0 += 32) {   // 32 steps: a block a lane
    const int n = w1 - g0 < 32 ? w1 - g0 : 32;
    const int v = 2 * g0 + lane, blk = keys.block(v);
    const bool in = lane < 2 * n && v < keys.count;
    int at = 0, bytes = 0;
    if (in) {
      const int64_t b = block_at(a.pool, tile.i, blk, head);
      at = b < 0 ? 0 : static_cast<int>(b);
      bytes = b < 0 ? 0xFFFF : a.pool.ks[b] | a.pool.vs[b] << 8;
    }

    auto load = [&](Tile &x, int s) {
      const int b0 = __builtin_amdgcn_readlane(at, 2 * s), b1 = __builtin_amdgcn_readlane(at, 2 * s + 1);
      // row c of the first product is key 16 (c / 4 mod 2) + 4 (c / 8) + c mod 4
      const int8_t *kp = a.pool.k + static_cast<int64_t>(c & 4 ? b1 : b0) * (kKvBlock * D) + (4 * (c >> 3) + (c & 3)) * 16;
      const int8_t *vp = a.pool.v + static_cast<int64_t>(h ? b1 : b0) * (kKvBlock * D);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const bool kin = 32 * d + 16 * h < D, vin = 32 * d + c < D;
        x.k[d] = kin ? load16(kp + (2 * d + h) * 256) : make_uint4(0, 0, 0, 0);
        x.v[d] = vin ? load16(vp + (32 * d + c) * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    auto compute = [&](const Tile &x, int s) {
      f32x16 acc = {};
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const uint4 k0 = codes_to_f16(x.k[d].x, x.k[d].y), k1 = codes_to_f16(x.k[d].z, x.k[d].w);
        acc = mfma_f16_32x32x16(k0, q.hi[2 * d], acc);
        acc = mfma_f16_32x32x16(k1, q.hi[2 * d + 1], acc);
        if constexpr (TWO) {
          acc = mfma_f16_32x32x16(k0, q.lo[2 * d], acc);
          acc = mfma_f16_32x32x16(k1, q.lo[2 * d + 1], acc);
        }
      }
      const int by0 = __builtin_amdgcn_readlane(bytes, 2 * s), by1 = __builtin_amdgcn_readlane(bytes, 2 * s + 1);
      const int bk0 = __builtin_amdgcn_readlane(blk, 2 * s) * kKvBlock;
      const int bk1 = __builtin_amdgcn_readlane(blk, 2 * s + 1) * kKvBlock;
      const int by = h ? by1 : by0, k0 = h ? bk1 : bk0;
      auto whole = [&](int b) { return b + 15 <= p0 && (b > p1 - window || b + 15 < a.sinks); };
      uint4 p[2], rest[2];
      if (whole(bk0) && whole(bk1)) {
        st.template weights<false>(acc, q.factor, by & 255, by >> 8, [](int) { return false; }, p, rest);
      } else {
        st.template weights<true>(acc, q.factor, by & 255, by >> 8,
                                  [&](int j) {
                                    const int k = k0 + j;
                                    return k > pos || (k <= pos - window && k >= a.sinks);
                                  },
                                  p, rest);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const uint4 v0 = codes_to_f16(x.v[d].x, x.v[d].y), v1 = codes_to_f16(x.v[d].z, x.v[d].w);
        st.y[d] = mfma_f16_32x32x16(v0, p[0], st.y[d]);
        st.y[d] = mfma_f16_32x32x16(v1, p[1], st.y[d]);
        if constexpr (TWO) {
          st.y[d] = mfma_f16_32x32x16(v0, rest[0], st.y[d]);
          st.y[d] = mfma_f16_32x32x16(v1, rest[1], st.y[d]);
        }
      }
    };
    Tile x, z;
    load(x, 0);
    for (int s = 0; s < n; s += 2) {
      if (s + 1 < n) load(z, s + 1);
      compute(x, s);
      if (s + 1 < n) {
        if (s + 2 < n) load(x, s + 2);
        compute(z, s + 1);
      }
    }
  }

  // the four waves' parts relative to the same powers, then their sums in order, by the first wave
  st.l = add_xor32(st.l);
  if (h == 0) as[wave][c] = st.a, bs[wave][c] = st.b, ls[wave][c] = st.l;
  __syncthreads();
  float ma = as[0][c], mb = bs[0][c], l = 0.0f;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) ma = fmaxf(ma, as[w][c]), mb = fmaxf(mb, bs[w][c]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) l += ls[w][c] * rescale(as[w][c], ls[w][c], ma);
  const float f = rescale(st.b, st.l, mb);
  const Quotient quotient(ma, mb, l, State<ND, TWO>::kOffset);
  const int64_t all = a.seqs.T * a.Hq, out = row * a.Hq + qh;
#pragma unroll
  for (int d0 = 0; d0 < ND; d0 += kMeet) {
    if (d0 > 0) __syncthreads();
#pragma unroll
    for (int d = d0; d < ND && d < d0 + kMeet; ++d)
#pragma unroll
      for (int j = 0; j < 16; ++j) st.y[d][j] *= f;
    if (wave > 0 && c < rows) {
#pragma unroll
      for (int d = d0; d < ND && d < d0 + kMeet; ++d)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4 *>(&meet[wave - 1][c][32 * (d - d0) + 2 * j + 4 * h]) =
              make_float4(st.y[d][j], st.y[d][j + 1], st.y[d][j + 2], st.y[d][j + 3]);
    }
    __syncthreads();
    if (wave == 0 && c < rows) {
#pragma unroll
      for (int d = d0; d < ND && d < d0 + kMeet; ++d)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int col = 32 * d + 2 * j + 4 * h;
          float4 sum = make_float4(st.y[d][j], st.y[d][j + 1], st.y[d][j + 2], st.y[d][j + 3]);
#pragma unroll
          for (int w = 0; w < kWaves - 1; ++w) {
            const float4 o = *reinterpret_cast<const float4 *>(&meet[w][c][32 * (d - d0) + 2 * j + 4 * h]);
            sum.x += o.x, sum.y += o.y, sum.z += o.z, sum.w += o.w;
          }
          if (col >= D) continue;
          if (parts)
            *reinterpret_cast<float4 *>(parts + results_at(splits, all) + (split * all + out) * D + col) = sum;
          else
            store4(a.y, types.out_bf16, out * D + col, quotient(sum.x), quotient(sum.y), quotient(sum.z), quotient(sum.w));
        }
    }
  }
  if (parts && wave == 0 && h == 0 && c < rows) {
    parts[split * all + out] = ma;
    parts[(splits + split) * all + out] = mb;
    parts[(2 * splits + split) * all + out] = l;
  }
}

// Joins the splits of a row in order.
__global__ __launch_bounds__(kThreads) void combine_kernel(AttnArgs a, Types types, int offset, int splits,
                                                           const float *parts, int64_t first) {
  const int64_t all = a.seqs.T * a.Hq;
  const int D = static_cast<int>(a.pool.D), quads = D / 4;
  const int64_t u = first + blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  const int64_t out = u / quads;
  const int col = 4 * static_cast<int>(u - out * quads);
  if (out >= all) return;
  const int64_t t = out / a.Hq;
  // rows in front of the first sequence or behind the last are left as they were
  if (t < Sequence::clamp(a.seqs.starts[0], a.seqs.T) || t >= Sequence::clamp(a.seqs.starts[a.seqs.N], a.seqs.T)) return;
  float ma = -__builtin_inff(), mb = ma;
  for (int s = 0; s < splits; ++s) ma = fmaxf(ma, parts[s * all + out]), mb = fmaxf(mb, parts[(splits + s) * all + out]);
  float l = 0.0f;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < splits; ++s) {
    const float ls = parts[(2 * splits + s) * all + out];
    if (ls == 0.0f) continue;             // saw nothing
    const float f = rescale(parts[(splits + s) * all + out], ls, mb);
    const float4 o = *reinterpret_cast<const float4 *>(parts + results_at(splits, all) + (s * all + out) * D + col);
    l = fmaf(ls, rescale(parts[s * all + out], ls, ma), l);
    sum.x = fmaf(o.x, f, sum.x), sum.y = fmaf(o.y, f, sum.y), sum.z = fmaf(o.z, f, sum.z), sum.w = fmaf(o.w, f, sum.w);
  }
  const Quotient q(ma, mb, l, offset);
  store4(a.y, types.out_bf16, out * D + col, q(sum.x), q(sum.y), q(sum.z), q(sum.w));
}

template <int ND, bool TWO>
void go_rows(const AttnArgs &a, const Types &t, const AttnPlan &p, float *ws, hipStream_t st) {
  const int64_t G = a.Hq / a.pool.Hk, all = tile_slots(a.seqs.T, a.seqs.N, G, kRows) * a.pool.Hk * p.splits;
  const int64_t most = max_groups(kThreads);
  for (int64_t first = 0; first < all; first += most)
    attention_rows_kernel<ND, TWO><<<static_cast<unsigned>(all - first < most ? all - first : most), kThreads, 0, st>>>(
        a, t, p.splits, p.splits > 1 ? ws : nullptr, first);
  if (p.splits == 1) return;
  const int64_t quads = a.seqs.T * a.Hq * (a.pool.D / 4), per = most * kThreads;
  for (int64_t first = 0; first < quads; first += per) {
    const int64_t n = quads - first < per ? quads - first : per;
    combine_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        a, t, State<ND, TWO>::kOffset, p.splits, ws, first);
  }
}

template <bool TWO>
void go(const AttnArgs &a, const Types &t, const AttnPlan &p, float *ws, hipStream_t st) {
  switch ((a.pool.D + 31) / 32) {
    case 1: return go_rows<1, TWO>(a, t, p, ws, st);
    case 2: return go_rows<2, TWO>(a, t, p, ws, st);
    case 3: return go_rows<3, TWO>(a, t, p, ws, st);
    case 4: return go_rows<4, TWO>(a, t, p, ws, st);
    case 5: return go_rows<5, TWO>(a, t, p, ws, st);
    case 6: return go_rows<6, TWO>(a, t, p, ws, st);
    case 7: return go_rows<7, TWO>(a, t, p, ws, st);
    default: return go_rows<8, TWO>(a, t, p, ws, st);
  }
}

}  // namespace

AttnPlan attention_plan(int64_t T, int64_t N, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len, int64_t window,
                        int64_t sinks, int path) {
  AttnPlan p = {};
  p.splits = 1;
  // rows of one key head a sequence, on average
  p.tiled = path == kPathTiled || (path == kPathAuto && T * (Hq / Hk) / N >= 64);
  if (p.tiled) return p;
  const int64_t G = Hq / Hk, groups = tile_slots(T, N, G, kRows) * Hk;
  int64_t keys = max_len;
  if (window > 0 && window + sinks + 32 < keys) keys = window + sinks + 32;
  // two workgroups a CU, a wave at least 64 keys of what a sequence may have
  int64_t s = 512 / groups, most = keys / 256;
  s = s < most ? s : most;
  p.splits = static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
  p.ws = p.splits > 1 ? (results_at(p.splits, T * Hq) + p.splits * T * Hq * D) * sizeof(float) : 0;
  return p;
}

hipError_t launch_attention(const AttnArgs &a, const AttnPlan &p, bool bf16, bool out_bf16, void *ws, hipStream_t st) {
  const Types t = {bf16, out_bf16};
  if (p.tiled) return launch_attention_tiled(a, t, st);
  if (bf16 && out_bf16) go<false>(a, t, p, static_cast<float *>(ws), st);
  else go<true>(a, t, p, static_cast<float *>(ws), st);
  return hipGetLastError();
}

}  // namespace q4

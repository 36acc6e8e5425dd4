// Attention of prompts: many query rows share a tile of keys (mathematics and
// operands: attention.hip, attn_device.hpp).
//
// A workgroup has 32 rows a wave of one key head, rows of all of its query heads
// side by side.  Keys and values of a step (64 keys, 32 past 128 columns) become
// halves once, on their way to LDS, where they lie as the matrix instructions'
// operands, 16 bytes a lane, 1 KB an instruction, so that neither writes nor
// reads conflict.  Operands come to registers four at a time, those of the next
// four instructions before these four.  Two buffers of LDS; a step's codes are
// loaded while the step before the last is multiplied; one barrier a step, which
// waits for LDS alone.
#include "attn_device.hpp"

namespace q4 {
namespace {

// WAVES waves, TILES times 32 keys a step.
template <int ND, bool TWO, int WAVES, int TILES>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4) void attention_tiled_kernel(AttnArgs a, Types types, int64_t slots,
                                                                                int64_t first) {
  constexpr int kRows = 32 * WAVES, kOps = 2 * ND;             // operands of 1 KB of one product and 32 keys
  constexpr int kLoads = (TILES * 2 * ND + WAVES - 1) / WAVES; // 16-byte loads of a lane a step
  constexpr int kSteps = 32 / TILES;                           // steps whose blocks the 64 lanes hold
  __shared__ uint4 key_ops[2][TILES][kOps][64], value_ops[2][TILES][kOps][64];
  __shared__ int2 blocks[2][2 * TILES];                        // scale bytes and first key of a step's blocks
  const int64_t id = first + blockIdx.x;
  // heads next to each other go to different XCDs, each with its keys in an L2 of its own; long rows first
  const int64_t head = id % a.pool.Hk, slot = slots - 1 - id / a.pool.Hk;
  const int64_t G = a.Hq / a.pool.Hk;
  const RowTile tile(a.seqs, slot, G, kRows);
  if (tile.i < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;
  const int D = static_cast<int>(a.pool.D), i = uniform(tile.i);
  const int64_t r0 = uniform(tile.r0), n = uniform(tile.rows), at_row = uniform(tile.s.row), at_pos = uniform(tile.s.first);
  const int64_t last = r0 + kRows < n ? r0 + kRows - 1 : n - 1;
  const KeyBlocks keys(at_pos + r0 / G, at_pos + last / G, a.window, a.sinks);
  // this wave's rows
  const int64_t wr = r0 + 32 * wave;
  const bool active = wr <= last;
  const int rows = !active ? 0 : last - wr < 31 ? static_cast<int>(last - wr) + 1 : 32;
  const int64_t r = wr + (c < rows ? c : rows - 1), t = r / G;
  const int64_t row = at_row + t, qh = head * G + (r - t * G);
  // lengths are int32, and so positions
  const int pos = static_cast<int>(at_pos + t);
  const int p0 = static_cast<int>(at_pos + wr / G), p1 = static_cast<int>(at_pos + (active ? wr + rows - 1 : wr) / G);
  const Sight sight(a.window, a.sinks);

  Query<ND, 2, TWO> q;
  q.load(a, types, active ? row * a.q_t + qh * a.q_h : 0, active, h);
  State<f32x16, ND, 2, TWO> st;

  // blocks of 64 keys' worth a lane, two rounds ahead: pages, then scales
  struct Info {
    int at, bytes, blk;
  };
  auto page_of = [&](int round) {
    const int v = 64 * round + lane;
    const int64_t p = v < keys.count ? keys.block(v) >> a.pool.page_blocks_log2 : a.pool.width;
    return p < a.pool.width ? a.pool.pages[i * a.pool.width + p] : -1;
  };
  auto info_of = [&](int round, int page) {
    const int v = 64 * round + lane;
    Info f = {0, 0xFFFF, keys.block(v)};     // a page that is not there: NaN
    if (v < keys.count && page >= 0 && page < a.pool.n_pages) {
      const int mask = (1 << a.pool.page_blocks_log2) - 1;
      f.at = static_cast<int>(((page * a.pool.Hk + head) << a.pool.page_blocks_log2) + (f.blk & mask));
      f.bytes = a.pool.ks[f.at] | a.pool.vs[f.at] << 8;
    }
    return f;
  };
  Info cur = info_of(0, page_of(0)), next = info_of(1, page_of(1));
  int page = page_of(2);

  // This wave's loads of a step: load u is of keys or values, of 32 columns of one
  // tile, which of two blocks by lane.  Columns past D, which the query has as 0 or
  // no result asks for, are the last ones again.
  uint4 raw[kLoads];
  int from[kLoads], to[kLoads];        // bytes from the block on; 16 bytes of LDS
  bool second[kLoads];
  const int8_t *base[kLoads];
  const int unit = kKvBlock * D;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int x = wave + WAVES * u, tl = x / (2 * ND), d = x / 2 % ND;
    to[u] = (tl * kOps + 2 * d) * 64 + lane;
    if (x & 1) {
      base[u] = a.pool.v;
      from[u] = min(32 * d + c, D - 1) * 16;
      second[u] = h;
    } else {
      // row c of the first product is key 16 (c / 4 mod 2) + 4 (c / 8) + c mod 4
      base[u] = a.pool.k;
      from[u] = min(2 * d + h, D / 16 - 1) * 256 + (4 * (c >> 3) + (c & 3)) * 16;
      second[u] = c & 4;
    }
  }
  auto load = [&](int s) {
    const int l = s % kSteps;
    if (l == 0 && s > 0) {
      cur = next;
      next = info_of(s / kSteps + 1, page);
      page = page_of(s / kSteps + 2);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int x = wave + WAVES * u, tl = x / (2 * ND);
      if (x >= TILES * 2 * ND) continue;
      const int b0 = __builtin_amdgcn_readlane(cur.at, 2 * TILES * l + 2 * tl);
      const int b1 = __builtin_amdgcn_readlane(cur.at, 2 * TILES * l + 2 * tl + 1);
      raw[u] = load16(base[u] + (static_cast<int64_t>(second[u] ? b1 : b0) * unit + from[u]));
    }
  };
  // the codes that load(s) brought; called before load(s + 1)
  auto store = [&](int s) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int x = wave + WAVES * u;
      if (x >= TILES * 2 * ND) continue;
      uint4 *p = (x & 1 ? &value_ops[s & 1][0][0][0] : &key_ops[s & 1][0][0][0]) + to[u];
      p[0] = codes_to_f16(raw[u].x, raw[u].y);
      p[64] = codes_to_f16(raw[u].z, raw[u].w);
    }
    if (wave == 0 && lane / (2 * TILES) == s % kSteps)
      blocks[s & 1][lane % (2 * TILES)] = make_int2(cur.bytes, cur.blk * kKvBlock);
  };
  constexpr int kAll = TILES * kOps, kGroup = 4, kGroups = (kAll + kGroup - 1) / kGroup;
  auto fetch_ops = [&](uint4 (&to)[kGroup], const uint4 (&ops)[TILES][kOps][64], int g) {
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (kGroup * g + j < kAll) to[j] = ops[(kGroup * g + j) / kOps][(kGroup * g + j) % kOps][lane];
  };
  auto compute = [&](int s) {
    int by[TILES], key[TILES];
    bool none = true, whole = true;    // of the step's keys that a row, or every row, sees
#pragma unroll
    for (int tl = 0; tl < TILES; ++tl) {
      const int2 m0 = blocks[s & 1][2 * tl], m1 = blocks[s & 1][2 * tl + 1];
      const int k0 = uniform(m0.y), k1 = uniform(m1.y);
      for (const int k : {k0, k1}) {
        none &= sight.none(p0, p1, k);
        whole &= sight.whole(p0, p1, k);
      }
      by[tl] = h ? m1.x : m0.x, key[tl] = h ? k1 : k0;
    }
    if (none) return;
    uint4 op[2][kGroup];
    f32x16 acc[TILES];
#pragma unroll
    for (int tl = 0; tl < TILES; ++tl) acc[tl] = f32x16{};
    fetch_ops(op[0], key_ops[s & 1], 0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) fetch_ops(op[(g + 1) & 1], key_ops[s & 1], g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const int o = kGroup * g + j, tl = o / kOps, d = o % kOps;
        if (o >= kAll) break;
        acc[tl] = mfma_f16_32x32x16(op[g & 1][j], q.hi[d], acc[tl]);
        if constexpr (TWO) acc[tl] = mfma_f16_32x32x16(op[g & 1][j], q.lo[d], acc[tl]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    fetch_ops(op[0], value_ops[s & 1], 0);
    typename decltype(st)::Keys w[TILES];
    if (whole) {
#pragma unroll
      for (int tl = 0; tl < TILES; ++tl)
        w[tl].template scores<false>(acc[tl], q.factor, by[tl] & 255, by[tl] >> 8, [](int) { return false; });
    } else {
#pragma unroll
      for (int tl = 0; tl < TILES; ++tl)
        w[tl].template scores<true>(acc[tl], q.factor, by[tl] & 255, by[tl] >> 8, [&](int j) {
          return sight.hides(pos, key[tl] + j);
        });
    }
    st.weights(w);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) fetch_ops(op[(g + 1) & 1], value_ops[s & 1], g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const int o = kGroup * g + j, tl = o / kOps, d = o % kOps / 2, u = o % 2;
        if (o >= kAll) break;
        st.y[d] = mfma_f16_32x32x16(op[g & 1][j], w[tl].p[u], st.y[d]);
        if constexpr (TWO) st.y[d] = mfma_f16_32x32x16(op[g & 1][j], w[tl].rest[u], st.y[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const int steps = (keys.count + 2 * TILES - 1) / (2 * TILES);
  if (steps > 0) {
    load(0);
    store(0);
    if (steps > 1) load(1);
    lds_barrier();
  }
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) store(s + 1);
    if (s + 2 < steps) load(s + 2);
    if (active) compute(s);
    lds_barrier();
  }
  const Quotient quotient(st.a, st.b, add_xor32(st.l), decltype(st)::kOffset);
  if (c >= rows) return;
  const int64_t out = (row * a.Hq + qh) * D;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const int col = 32 * d + 2 * j + 4 * h;
      if (col < D)
        store4(a.y, types.out_bf16, out + col, quotient(st.y[d][j]), quotient(st.y[d][j + 1]), quotient(st.y[d][j + 2]),
               quotient(st.y[d][j + 3]));
    }
}

template <int ND, bool TWO>
void go(const AttnArgs &a, const Types &t, hipStream_t st) {
  // 64 keys of more than 128 columns would be more than 64 KB in two buffers, and eight waves' registers too few
  constexpr int WAVES = ND <= 4 ? 8 : 4, TILES = ND <= 4 ? 2 : 1;
  const int64_t slots = tile_slots(a.seqs.T, a.seqs.N, a.Hq / a.pool.Hk, 32 * WAVES), all = slots * a.pool.Hk;
  const int64_t most = max_groups(64 * WAVES);
  for (int64_t first = 0; first < all; first += most)
    attention_tiled_kernel<ND, TWO, WAVES, TILES>
        <<<static_cast<unsigned>(all - first < most ? all - first : most), 64 * WAVES, 0, st>>>(a, t, slots, first);
}

template <bool TWO>
void pick(const AttnArgs &a, const Types &t, hipStream_t st) {
  switch ((a.pool.D + 31) / 32) {
    case 1: return go<1, TWO>(a, t, st);
    case 2: return go<2, TWO>(a, t, st);
    case 3: return go<3, TWO>(a, t, st);
    case 4: return go<4, TWO>(a, t, st);
    case 5: return go<5, TWO>(a, t, st);
    case 6: return go<6, TWO>(a, t, st);
    case 7: return go<7, TWO>(a, t, st);
    default: return go<8, TWO>(a, t, st);
  }
}

}  // namespace

hipError_t launch_attention_tiled(const AttnArgs &a, const Types &t, hipStream_t st) {
  t.in_bf16 && t.out_bf16 ? pick<false>(a, t, st) : pick<true>(a, t, st);
  return hipGetLastError();
}

}  // namespace q4

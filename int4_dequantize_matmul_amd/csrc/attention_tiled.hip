// Attention of prompts: many query rows share a tile of keys (mathematics and
// operands: attention.hip, attn_device.hpp).
//
// A workgroup has 256 rows of one key head, 32 a wave, rows of all of its query
// heads side by side.  Keys and values of a step of 64 keys become halves once, on
// their way to LDS, where they lie as the matrix instructions' operands, 16 bytes a
// lane, 1 KB an instruction, so that neither writes nor reads conflict.  An operand is on its way to registers seven instructions before
// the one that takes it.  One barrier a step, which waits for LDS alone; the second
// wave of a SIMD has it in the middle of its step, so that one wave has the
// exponentials of its scores while the other has the matrix instructions.  Two
// buffers each of keys and values, values a step behind; codes are loaded a step
// before they become halves, 1 KB of one block an instruction.
//
// Bound by the matrix instructions and their operands from LDS: a prompt of 8190
// tokens, 32 + 8 heads of 128, takes 600 to 625 us (900 TFLOP/s; a large library
// product 1155, 476 us); the instructions alone 271, with their operands 340, first
// loads and last stores of the workgroups 88.  Half a step apart against together:
// 597 and 657; two barriers a step 617 to 654, four waves a workgroup 660.
#include "attn_device.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 8, kTiles = 2;   // waves a workgroup; times 32 keys a step

template <int ND, bool TWO>
__global__ __launch_bounds__(64 * kWaves, kWaves / 4) void attention_tiled_kernel(AttnArgs a, Types types, uint32_t last_slot) {
  constexpr int kRows = 32 * kWaves, kOps = 2 * ND, kAll = kTiles * kOps;   // operands of 1 KB of a product
  constexpr int kBlocks = 2 * kTiles, kSteps = 64 / kBlocks;               // blocks a step; steps whose blocks 64 lanes hold
  constexpr int kUnits = kBlocks * ((ND + 1) / 2), kLoads = (kUnits + kWaves - 1) / kWaves;   // loads of a step, of a wave
  __shared__ uint4 key_ops[2][kTiles][kOps][64], value_ops[2][kTiles][kOps][64];
  __shared__ int2 blocks[2][kBlocks];                                     // scale bytes and first key of a step's blocks
  // heads next to each other go to different XCDs, each with its keys in an L2 of its own; long rows first
  const uint32_t Hk = static_cast<uint32_t>(a.pool.Hk), slot = last_slot - blockIdx.x / Hk;
  const int head = static_cast<int>(blockIdx.x % Hk);
  const uint32_t G = static_cast<uint32_t>(a.G);
  const RowTile<kRows> tile(a.seqs, slot, G);
  if (tile.s.i < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;
  const int D = static_cast<int>(a.pool.D);
  const int last = (tile.rows - tile.r0 > kRows ? tile.r0 + kRows : tile.rows) - 1;
  const Sight sight(a.window, a.sinks);
  const KeyBlocks keys(tile.s.first + tile.r0 / static_cast<int>(G), tile.s.first + last / static_cast<int>(G), sight,
                       a.pool);
  const int steps = (keys.count + kBlocks - 1) / kBlocks;

  // blocks of a round of kSteps steps, one a lane, two rounds ahead: pages, then scales
  const int32_t *pages = a.pool.pages + tile.s.i * a.pool.width;
  const int page_mask = (1 << a.pool.page_blocks_log2) - 1;
  struct Info {
    int at, bytes, blk;
  };
  auto page_of = [&](int round) {
    const int v = 64 * round + lane;
    const int64_t p = v < keys.count ? keys.block(v) >> a.pool.page_blocks_log2 : a.pool.width;
    return p < a.pool.width ? pages[p] : -1;
  };
  auto info_of = [&](int round, int page) {
    const int v = 64 * round + lane;
    Info f = {0, 0xFFFF, keys.block(v)};     // a page that is not there: NaN
    if (v < keys.count && page >= 0 && page < a.pool.n_pages) {
      f.at = ((page * static_cast<int>(Hk) + head) << a.pool.page_blocks_log2) + (f.blk & page_mask);
      f.bytes = a.pool.ks[f.at] | a.pool.vs[f.at] << 8;
    }
    return f;
  };
  const int page0 = page_of(0), page1 = page_of(1);
  int page = page_of(2);

  // this wave's rows; lengths are int32, and so positions
  const int wr = tile.r0 + 32 * wave;
  const bool active = wr <= last;
  const int rows = !active ? 0 : min(last - wr + 1, 32);
  const int r = wr + (c < rows ? c : max(rows - 1, 0)), t = static_cast<int>(static_cast<uint32_t>(r) / G);
  const int64_t row = tile.s.row + t, qh = head * static_cast<int>(G) + (r - t * static_cast<int>(G));
  const int pos = tile.s.first + t;
  const int p0 = uniform(tile.s.first + wr / static_cast<int>(G));
  const int p1 = uniform(tile.s.first + (active ? wr + rows - 1 : wr) / static_cast<int>(G));
  Query<ND, 2, TWO> q;
  q.load(a, types, active ? row * a.q_t + qh * a.q_h : 0, active, h);
  Info cur = info_of(0, page0), next = info_of(1, page1);

  // This wave's loads of a step: load u is 64 columns of one block.  Lane l has 16
  // columns of token l mod 16 of the keys, column l of the values.  Columns past D,
  // which the query has as 0 or no result asks for, are the last ones again.
  uint4 raw_k[kLoads], raw_v[kLoads];
  int from_k[kLoads], from_v[kLoads], to_k[kLoads], to_v[kLoads];   // bytes in the block; 16 bytes of LDS
  int of[kLoads];                                                   // the blocks of the values to load next
  const int64_t unit = kKvBlock * D;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int x = wave + kWaves * u, b = x % kBlocks, g = x / kBlocks, tl = b / 2, half = b % 2;
    // token 4 i + j of block h is row 8 i + 4 h + j of the first product
    const int token = lane & 15, chunk = 4 * g + (lane >> 4), col = 64 * g + lane;
    from_k[u] = min(chunk, D / 16 - 1) * 256 + token * 16;
    from_v[u] = min(col, D - 1) * 16;
    to_k[u] = (tl * kOps + chunk / 2 * 2) * 64 + 8 * (token >> 2) + 4 * half + (token & 3) + 32 * (chunk & 1);
    to_v[u] = (tl * kOps + col / 32 * 2) * 64 + (col & 31) + 32 * half;
    if (ND % 2 && chunk >= kOps) to_k[u] = -1;   // past the last 32 columns
    if (ND % 2 && col >= 32 * ND) to_v[u] = -1;
  }
  auto load_values = [&] {   // of the step whose keys were loaded last
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (wave + kWaves * u < kUnits) raw_v[u] = load16(a.pool.v + of[u] * unit + from_v[u]);
  };
  auto load_keys = [&](int s) {
    const int l = s % kSteps;
    if (l == 0 && s > 0) {
      cur = next;
      next = info_of(s / kSteps + 1, page);
      page = page_of(s / kSteps + 2);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (wave + kWaves * u >= kUnits) continue;
      of[u] = __builtin_amdgcn_readlane(cur.at, kBlocks * l + (wave + kWaves * u) % kBlocks);
      raw_k[u] = load16(a.pool.k + of[u] * unit + from_k[u]);
    }
  };
  auto store = [&](uint4 *ops, const int (&to)[kLoads], const uint4 (&raw)[kLoads]) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (wave + kWaves * u >= kUnits || to[u] < 0) continue;
      ops[to[u]] = codes_to_f16(raw[u].x, raw[u].y);
      ops[to[u] + 64] = codes_to_f16(raw[u].z, raw[u].w);
    }
  };
  // the keys that load_keys(s) brought; called before load_keys(s + 1)
  auto store_keys = [&](int s) {
    store(&key_ops[s & 1][0][0][0], to_k, raw_k);
    if (wave == 0 && lane / kBlocks == s % kSteps)
      blocks[s & 1][lane % kBlocks] = make_int2(cur.bytes, cur.blk * kKvBlock);
  };
  // In step s, when no wave reads them any more: the keys of s + 1 and the values of s.
  auto stage = [&](int s) {
    if (s + 1 < steps) store_keys(s + 1);
    if (s < steps) store(&value_ops[s & 1][0][0][0], to_v, raw_v);
    if (s + 1 < steps) load_values();
    if (s + 2 < steps) load_keys(s + 2);
  };

  // This wave's rows all see all of the keys of steps [inner, outer), of blocks from
  // the last row's window's first whole one to the first row's last, and nothing
  // from `end` on; in the other steps, sinks among them, each score is looked at.
  int inner = 0, outer = 0, end = -1;
  if (active) {
    if (p1 >= sight.window) inner = (static_cast<int>((static_cast<uint32_t>(p1 - sight.window) + 16) / kKvBlock) - keys.skip + kBlocks - 1) / kBlocks;
    if (p0 >= 0) outer = (static_cast<int>((static_cast<uint32_t>(p0) + 1) / kKvBlock) - keys.skip) / kBlocks;
    end = p1 < 0 ? 0 : min((p1 / kKvBlock + 1 - keys.skip + kBlocks - 1) / kBlocks, steps);
  }

  State<f32x16, ND, 2, TWO> st;
  constexpr int kRing = 8;
  uint4 ring[kRing];
  f32x16 acc[kTiles];
  typename decltype(st)::Keys w[kTiles];
#pragma unroll
  for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
    for (int u = 0; u < 2; ++u) w[tl].p[u] = w[tl].rest[u] = make_uint4(0, 0, 0, 0);
  int by[kTiles], key[kTiles];
  // The products of step s - 1 with its values, of step s with its keys.  The first
  // step has weights and values of 0 in front of it, and behind the last one scores
  // that nobody reads: one form of this loop, whose results stay where they are.
  auto multiply = [&](int s) {
    const uint4 *vo = &value_ops[(s - 1) & 1][0][0][lane], *ko = &key_ops[s & 1][0][0][lane];
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl) {
      const int2 m = blocks[s & 1][2 * tl + h];
      by[tl] = m.x, key[tl] = m.y;
      acc[tl] = f32x16{};
    }
    auto operand = [&](int o) { return o < kAll ? vo[64 * o] : ko[64 * (o - kAll)]; };
#pragma unroll
    for (int o = 0; o < kRing - 1 && o < 2 * kAll; ++o) ring[o] = operand(o);
#pragma unroll
    for (int o = 0; o < 2 * kAll; ++o) {
      if (o + kRing - 1 < 2 * kAll) ring[(o + kRing - 1) % kRing] = operand(o + kRing - 1);
      __builtin_amdgcn_sched_barrier(0);
      const uint4 x = ring[o % kRing];
      const int tl = o % kAll / kOps, d = o % kOps;
      if (o < kAll) {
        st.y[d / 2] = mfma_f16_32x32x16(x, w[tl].p[d % 2], st.y[d / 2]);
        if constexpr (TWO) st.y[d / 2] = mfma_f16_32x32x16(x, w[tl].rest[d % 2], st.y[d / 2]);
      } else {
        acc[tl] = mfma_f16_32x32x16(x, q.hi[d], acc[tl]);
        if constexpr (TWO) acc[tl] = mfma_f16_32x32x16(x, q.lo[d], acc[tl]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto weigh = [&](int s) {
    if (s >= inner && s < outer) {
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl)
        w[tl].template scores<false>(acc[tl], q.factor, by[tl] & 255, by[tl] >> 8, [](int) { return false; });
    } else {
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl)
        w[tl].template scores<true>(acc[tl], q.factor, by[tl] & 255, by[tl] >> 8, [&](int j) {
          return sight.hides(pos, key[tl] + j);
        });
    }
    st.weights(w);
  };

  if (steps > 0) {
    load_keys(0);
    load_values();
    store_keys(0);
    if (steps > 1) load_keys(1);
  }
  for (int x = threadIdx.x; x < kAll * 64; x += 64 * kWaves) (&value_ops[1][0][0][0])[x] = make_uint4(0, 0, 0, 0);
  lds_barrier();
  // Between two barriers, step s: K(s) and V(s - 1) are read, K(s + 1) and V(s) written.
  const bool second = wave >= kWaves / 2;
  for (int s = 0; s <= steps; ++s) {
    if (s <= end) multiply(s);
    stage(s);
    if (second) lds_barrier();
    if (s < end) weigh(s);
    if (!second) lds_barrier();
  }

  const Quotient quotient(st.d, add_xor32(st.l), decltype(st)::kOffset);
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
  const int64_t slots = tile_slots(a.seqs.T, a.seqs.N, a.G, 32 * kWaves), most = max_groups(64 * kWaves) / a.pool.Hk;
  for (int64_t left = slots; left > 0; left -= most)   // slots of a launch
    attention_tiled_kernel<ND, TWO><<<static_cast<unsigned>((left < most ? left : most) * a.pool.Hk), 64 * kWaves, 0, st>>>(
        a, t, static_cast<uint32_t>(left - 1));
}

}  // namespace

// Past 128 columns, with two halves past 64, a wave's registers would not do.
bool attention_tiled_ok(int64_t D, bool two) { return D <= (two ? 64 : 128); }

hipError_t launch_attention_tiled(const AttnArgs &a, const Types &t, hipStream_t st) {
  const int64_t nd = (a.pool.D + 31) / 32;
  if (t.in_bf16 && t.out_bf16) {
    if (nd == 1) go<1, false>(a, t, st);
    else if (nd == 2) go<2, false>(a, t, st);
    else if (nd == 3) go<3, false>(a, t, st);
    else go<4, false>(a, t, st);
  } else {
    if (nd == 1) go<1, true>(a, t, st);
    else go<2, true>(a, t, st);
  }
  return hipGetLastError();
}

}  // namespace q4

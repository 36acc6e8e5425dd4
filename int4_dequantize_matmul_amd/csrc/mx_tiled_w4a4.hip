// W4A4 in MX FP4 for many activation rows: LDS-tiled scaled matrix products.
//
//   y[m,n] = sum_b 2^(sx[m,b] + sw[n,b] - 254) sum_{k in b} cx[m,k] cw[n,k]
//
// The scaled 32 x 32 x 64 instruction takes the format as stored: a lane's
// operand is one block (16 bytes) and a byte of scale, so nothing is unpacked
// and the sums stay in f32.
//
// K goes in stages of 256 columns, 128 bytes of a row, through two places in
// LDS: a load that writes LDS costs what the rows it touches cost, in pieces
// of 128 bytes (19 clocks a KB, 28 in pieces of 64 bytes).  A stage is four
// instructions deep: in step q lane (r, h) takes block 4 h + q of row r, whose
// scale is byte q of a dword.
//
// Measured, operands met just before | from memory: 2048 x 13312 x 2048 38 us
// (2.9 PFLOP/s) | 45, 8192 x 2048 x 5632 50 us (3.8 PFLOP/s; the instruction alone
// 8.2) | 53.  In the second one a stage takes 3100 clocks of which the matrix
// instructions need 2400; the first loads, the stores and the launch take 12 us
// more.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "mx_plan.hpp"
#include "mx_tile.hpp"
#include "q4_lds_dma.hpp"

namespace q4 {
namespace {

struct TileArgs {
  const uint8_t *x, *sx, *w, *sw;
  void *y;
  int64_t M, N;
  int KB;
  int tiles_m, tiles_n;
};

// LDS of a group of waves: two stages of weight rows and then activation rows,
// and two buffers of their scales in slots of 16 bytes.  S16 (rows of scales
// that start on 16 bytes): a slot has the scales of two stages.  Otherwise the
// three dwords that a stage's 8 scales lie in, wherever they begin.
template <int BN, int BM>
struct Lds {
  static constexpr int rows = BN + BM, stage = rows * 128, s = 2 * stage, s_buf = rows * 16, bytes = s + 2 * s_buf;
};

// Tiles of 32 WM TM rows by 32 WN TN weight rows, by KG groups of NW waves,
// each with a part of K; in a group WN waves lie side by side along the weight
// rows; a wave has 32 TN weight rows by 32 TM rows.
template <int KG, int NW, int WN, int TN, int TM, bool S16, bool BOUT>
__global__ __launch_bounds__(64 * NW * KG, NW * KG <= 4 ? 2 : NW * KG / 4) void mx_tiled_w4a4(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem0[];
  constexpr int WM = NW / WN, BN = 32 * WN * TN, BM = 32 * WM * TM;
  using L = Lds<BN, BM>;

  const int KB = a.KB, pitch = KB * 16, all = (KB + 7) >> 3, tiles = a.tiles_m * a.tiles_n;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = KG > 1 ? wave % NW : wave, kg = KG > 1 ? wave / NW : 0;
  const int steps = KG > 1 ? (all + KG - 1) / KG : all, first = 8 * kg * steps;   // this group's stages; its first block
  uint8_t *smem = smem0 + kg * L::bytes;
  const int wn = wv / WM, wm = wv % WM;
  const int r = lane & 31, h = lane >> 5;
  const uint32_t lds0 = lds_addr(smem);

  const TileAt at = tile_at(xcd_run(static_cast<int>(blockIdx.x), tiles), a.tiles_m, a.tiles_n);
  const int64_t m0 = static_cast<int64_t>(at.m) * BM, n0 = static_cast<int64_t>(at.n) * BN;
  const int rows_m = min(static_cast<int>(a.M - m0), BM), rows_n = min(static_cast<int>(a.N - n0), BN);
  const __amdgpu_buffer_rsrc_t rs_w = rsrc(a.w + n0 * pitch, rows_n * pitch);
  const __amdgpu_buffer_rsrc_t rs_x = rsrc(a.x + m0 * pitch, rows_m * pitch);
  // whole dwords of scales: a dword with a byte of them may be read whole
  const uint8_t *sw0 = a.sw + n0 * KB, *sx0 = a.sx + m0 * KB;
  const int sw_odd = static_cast<int>(reinterpret_cast<uintptr_t>(sw0) & 3);
  const int sx_odd = static_cast<int>(reinterpret_cast<uintptr_t>(sx0) & 3);
  const __amdgpu_buffer_rsrc_t rs_sw = rsrc(sw0 - sw_odd, (sw_odd + rows_n * KB + 3) & ~3);
  const __amdgpu_buffer_rsrc_t rs_sx = rsrc(sx0 - sx_odd, (sx_odd + rows_m * KB + 3) & ~3);

  // Staging.  A load fills 8 LDS rows: lane i lands at row i / 8, position
  // i % 8, which holds chunk (i % 8) ^ (row / 2 % 8): 16 neighbouring rows then
  // have a chunk in the 16 different places that one clock reads.  LDS row i of the weights is row w_row32(i
  // % 32) of its 32.  Rows past the tile's end and chunks from KB on lie past
  // the buffer's range (or are sent there) and come as zeros, and so do whole
  // stages past the last one.
  // (An address worked out in vector registers is still the same in all lanes.)
  auto uniform = [](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); };
  // (The offsets are formed anew for each load: kept in registers they would
  // not leave room for the sums.)
  const int lrow = lane >> 3, even = (lane & 7) ^ (lrow >> 1);
  constexpr int nW = BN / 8 / NW, nX = BM / 8 / NW;   // loads of a wave in a stage
  static_assert(nW * 8 * NW == BN && nX * 8 * NW == BM, "whole loads");
  auto chunk = [&](int j) { return even ^ (4 * (j & 1)); };   // of a wave's load j
  int x_lane = lrow * pitch, w_lane = w_row32(lrow) * pitch;
  static_assert(nW % 2 == 0 && nX % 2 == 0, "a wave's loads begin at 16 rows");
  // LDS rows i .. i + 7 of the weights are rows w_at(i) + w_row32(0 .. 7)
  auto w_at = [](int i) { return (i & ~31) + 4 * ((i >> 3) & 3); };
  auto load_w = [&](int slot, int b0, int j) {
    const int i = 8 * (nW * wv + j);
    dma16(rs_w, uniform(lds0 + slot * L::stage + i * 128), b0 + chunk(j) < KB ? w_lane + w_at(i) * pitch + (b0 + chunk(j)) * 16 : kFar, 0);
  };
  auto load_x = [&](int slot, int b0, int j) {
    const int i = 8 * (nX * wv + j);
    dma16(rs_x, uniform(lds0 + slot * L::stage + (BN + i) * 128), b0 + chunk(j) < KB ? x_lane + i * pitch + (b0 + chunk(j)) * 16 : kFar, 0);
  };
  // Scales.  S16: a row a lane, 64 rows a load, every other stage.  Else lane i
  // has dword i % 4 of row i / 4.
  constexpr int nSw = S16 ? 1 : BN / 16 / NW, nSx = S16 ? 0 : BM / 16 / NW;
  static_assert(S16 ? L::rows == 64 * NW : nSw * 16 * NW == BN && nSx * 16 * NW == BM, "whole loads");
  auto w_row_at = [](int i) { return (i & ~31) + w_row32(i & 31); };
  int sw_lane, sx_lane;
  const __amdgpu_buffer_rsrc_t rs_s16 = 64 * wv < BN ? rs_sw : rs_sx;
  if constexpr (S16) {
    const bool w = 64 * wv < BN;
    sw_lane = (w ? w_row_at(64 * wv + lane) : 64 * wv - BN + lane) * KB;
    sx_lane = 0;
  } else {
    sw_lane = sw_odd + w_row32((lane >> 2) & 7) * KB + 4 * (lane >> 5) * KB;   // LDS rows 8 .. 15 come 4 rows on
    sx_lane = sx_odd + (lane >> 2) * KB;
  }
  auto load_sw = [&](int s, int b0, int j) {
    if constexpr (S16) {
      dma16(rs_s16, uniform(lds0 + L::s + ((s >> 1) & 1) * L::s_buf + wv * 1024), b0 < KB ? sw_lane + b0 : kFar, 0);
    } else {
      const int i = 16 * (nSw * wv + j), sub = 4 * (lane & 3);
      const int o = (b0 < KB) & (sub < 12) ? ((sw_lane + w_at(i) * KB + b0) & ~3) + sub : kFar;
      dma4(rs_sw, uniform(lds0 + L::s + (s & 1) * L::s_buf + i * 16), o, 0);
    }
  };
  auto load_sx = [&](int s, int b0, int j) {
    const int i = 16 * (nSx * wv + j), sub = 4 * (lane & 3);
    const int o = (b0 < KB) & (sub < 12) ? ((sx_lane + i * KB + b0) & ~3) + sub : kFar;
    dma4(rs_sx, uniform(lds0 + L::s + (s & 1) * L::s_buf + (BN + i) * 16), o, 0);
  };
  constexpr int nS = nSw + nSx, nAll = nS + nW + nX;
  auto load = [&](int slot, int s, int j) {   // load j of stage s; slot = s % 2
    const int b0 = first + 8 * s;
    if (j < nSw && !(S16 && slot)) load_sw(s, b0, j);
    else if (j < nSw) return;
    else if (j < nS) load_sx(s, b0, j - nSw);
    else if (j < nS + nW) load_w(slot, b0, j - nS);
    else load_x(slot, b0, j - nS - nW);
  };
  const std::integral_constant<int, 0> c0;
  const std::integral_constant<int, 1> c1;
  const std::integral_constant<int, 2> c2;
  const std::integral_constant<int, 3> c3;

  // Fragments of step q of a stage, and the scales of a stage.
  struct Frags {
    uint4 w[TN], x[TM];
  };
  struct Scales {
    uint32_t w[TN], x[TM];
  };
  const int w_base = (32 * TN * wn + r) * 128, x_base = (BN + 32 * TM * wm + r) * 128;
  auto read = [&](Frags &f, int slot, int q) {
    const uint8_t *st = smem + slot * L::stage + (((4 * h + q) ^ ((r >> 1) & 7)) << 4);
#pragma unroll
    for (int t = 0; t < TN; ++t) f.w[t] = load16(st + w_base + t * 4096);
#pragma unroll
    for (int t = 0; t < TM; ++t) f.x[t] = load16(st + x_base + t * 4096);
  };
  // A row's scales of the lane's four blocks; in the last stage the bytes past
  // the row's end are another row's, and a NaN among them would meet the zeros
  // there.
  uint32_t odd[TN + TM];
#pragma unroll
  for (int t = 0; t < TN; ++t) odd[t] = (sw_odd + w_row_at(32 * (TN * wn + t) + r) * KB) & 3;
#pragma unroll
  for (int t = 0; t < TM; ++t) odd[TN + t] = (sx_odd + (32 * (TM * wm + t) + r) * KB) & 3;
  auto read_scales = [&](Scales &f, int s) {
    const int left = KB - first - 8 * s - 4 * h;
    const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
    auto one = [&](int row, uint32_t o) {
      if constexpr (S16) {
        return *reinterpret_cast<const uint32_t *>(smem + L::s + ((s >> 1) & 1) * L::s_buf + row * 16 + 8 * (s & 1) + 4 * h);
      } else {
        const uint32_t *d = reinterpret_cast<const uint32_t *>(smem + L::s + (s & 1) * L::s_buf + row * 16 + 4 * h);
        return __builtin_amdgcn_alignbyte(d[1], d[0], o) & mask;
      }
    };
#pragma unroll
    for (int t = 0; t < TN; ++t) f.w[t] = one(32 * (TN * wn + t) + r, odd[t]);
#pragma unroll
    for (int t = 0; t < TM; ++t) f.x[t] = one(BN + 32 * (TM * wm + t) + r, odd[TN + t]);
  };

  f32x16 acc[TM][TN] = {};
  // Between the instructions go the loads lo .. hi - 1 of stage s.
  auto multiply = [&](const Frags &f, const Scales &sc, auto q_c, auto slot_c, int s, auto lo_c, auto hi_c) {
    constexpr int Q = decltype(q_c)::value, lo = decltype(lo_c)::value, n = decltype(hi_c)::value - lo;
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const int at = tm * TN + tn;
        acc[tm][tn] = mfma_mx_32x32x64<Q>(f.w[tn], f.x[tm], acc[tm][tn], sc.w[tn], sc.x[tm]);
#pragma unroll
        for (int j = at * n / (TM * TN); j < (at + 1) * n / (TM * TN); ++j) {
          __builtin_amdgcn_sched_barrier(0);
          load(decltype(slot_c)::value, s, lo + j);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
  };
  const std::integral_constant<int, 0> n0c;
  const std::integral_constant<int, nAll / 3> n1c;
  const std::integral_constant<int, 2 * nAll / 3> n2c;
  const std::integral_constant<int, nAll> n3c;

  // While one step is multiplied the next one's fragments are read.  The
  // barrier before a stage's last step says that the next stage has landed and
  // that this one has been read by every wave, so its place can take the stage
  // after the next.  Its loads go out in three parts, a step apart: all at
  // once they would hold the waves up, one after the other.
  Frags f0, f1;
  Scales sc0, sc1;
#pragma unroll
  for (int j = 0; j < nAll; ++j) load(0, 0, j);
#pragma unroll
  for (int j = 0; j < nAll / 3; ++j) load(1, 1, j);
  wait_vmcnt<0>();
  lds_barrier();
  read_scales(sc0, 0);
  read(f0, 0, 0);
  auto stage = [&](int s, auto slot_c, auto other_c, const Scales &sc, Scales &next) {
    constexpr int p = decltype(slot_c)::value;
    asm("" : "+v"(x_lane), "+v"(w_lane), "+v"(sx_lane), "+v"(sw_lane));
    read(f1, p, 1);
    multiply(f0, sc, c0, other_c, s + 1, n1c, n2c);
    read(f0, p, 2);
    multiply(f1, sc, c1, other_c, s + 1, n2c, n3c);
    read(f1, p, 3);
    multiply(f0, sc, c2, slot_c, 0, n0c, n0c);
    wait_vmcnt<0>();
    lds_barrier();
    read(f0, p ^ 1, 0);
    read_scales(next, s + 1);
    multiply(f1, sc, c3, slot_c, s + 2, n0c, n1c);
  };
  for (int s = 0; s < steps; s += 2) {
    stage(s, c0, c1, sc0, sc1);
    if (s + 1 < steps) stage(s + 1, c1, c0, sc1, sc0);
  }
  wait_vmcnt<0>();   // the loads past the end land before the LDS is used again

  // Stores: lane (c, h) has row c of each 32 activation rows.
  const int64_t m1 = m0 + 32 * TM * wm + r, n1 = n0 + 32 * TN * wn + 16 * h;
  if constexpr (KG > 1) {
    // the groups' sums, in their order; group i takes the tiles i, i + KG ..
    f32x16 *part = reinterpret_cast<f32x16 *>(smem0) + (wv * 64 + lane);
    constexpr int kPart = NW * 64;
    static_assert(TM * TN * kPart * 64 <= L::bytes, "the sums fit");
    lds_barrier();
#pragma unroll
    for (int t = 0; t < TM * TN; ++t) part[(kg * TM * TN + t) * kPart] = acc[t / TN][t % TN];
    lds_barrier();
    for (int t = kg; t < TM * TN; t += KG) {
      f32x16 sum = part[t * kPart];
#pragma unroll
      for (int i = 1; i < KG; ++i) sum += part[(i * TM * TN + t) * kPart];
      const int64_t m = m1 + 32 * (t / TN);
      if (m < a.M) store_16<BOUT>(a.y, m, n1 + 32 * (t % TN), a.N, sum);
    }
  } else if constexpr (BN == 256) {
    lds_barrier();
    store_lines<TM, TN, BOUT>(smem + wv * (64 * TM * TN * 32), a.y, a.M, a.N, m0 + 32 * TM * wm, n0 + 32 * TN * wn, acc);
  } else {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
      if (m1 + 32 * tm < a.M) {
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) store_16<BOUT>(a.y, m1 + 32 * tm, n1 + 32 * tn, a.N, acc[tm][tn]);
      }
  }
}

template <int KG, int NW, int WN, int TN, int TM, bool S16, bool BOUT>
hipError_t go(TileArgs a, hipStream_t st) {
  constexpr int BN = 32 * WN * TN, BM = 32 * (NW / WN) * TM, lds = KG * Lds<BN, BM>::bytes;
  a.tiles_m = static_cast<int>((a.M + BM - 1) / BM);
  a.tiles_n = static_cast<int>((a.N + BN - 1) / BN);
  const int tiles = a.tiles_m * a.tiles_n;
  const auto kernel = mx_tiled_w4a4<KG, NW, WN, TN, TM, S16, BOUT>;
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (set != hipSuccess) return set;
  kernel<<<static_cast<unsigned>(tiles), 64 * NW * KG, lds, st>>>(a);
  return hipGetLastError();
}

template <bool S16, bool BOUT>
hipError_t pick(const TileArgs &a, hipStream_t st) {
  constexpr bool large = S16 || BOUT;
  switch (mx_w4a4_tile(a.M, a.N, device_cu_count() > 0 ? device_cu_count() : 256, large)) {
    case MxW4A4Tile::k32x64: return go<4, 2, 2, 1, 1, false, BOUT>(a, st);
    case MxW4A4Tile::k64x64: return go<2, 4, 2, 1, 1, false, BOUT>(a, st);
    case MxW4A4Tile::k256x256:
      if constexpr (large) return go<1, 8, 2, 4, 2, S16, BOUT>(a, st);
      return hipErrorInvalidValue;   // not chosen
    default: return go<1, 4, 2, 2, 2, S16, BOUT>(a, st);
  }
}

}  // namespace

// Ranges of the tiles' buffers in 30 bits, tile counts in 31.
bool mx_tiled_w4a4_ok(int64_t M, int64_t N, int64_t K) {
  return K <= (int64_t(1) << 22) && ((M + 31) / 32) * ((N + 31) / 32) < (int64_t(1) << 30);
}

hipError_t launch_mx_tiled_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                                bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const TileArgs a = {xq, sx, wq, sw, y, M, N, static_cast<int>((K + 31) / 32), 0, 0};
  const auto at16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (a.KB % 16 == 0 && at16(sx) && at16(sw)) return y_bf16 ? pick<true, true>(a, st) : pick<true, false>(a, st);
  return y_bf16 ? pick<false, true>(a, st) : pick<false, false>(a, st);
}

}  // namespace q4

// bf16 activations times MX FP4 weights for many activation rows: LDS-tiled
// bf16 matrix products.
//
//   y[m,n] = sum_k x[m,k] cw[n,k] 2^(sw[n,k/32] - 127)
//
// The weights stay packed up to the registers: a lane takes 8 codes (a dword)
// and its block's scale to 8 bf16 values in four conversions, exactly.
//
// K goes in stages of 64 columns.  In a stage lane (r, g) holds columns
// 16 g .. 16 g + 15 of row r, 8 for each of two matrix instructions (which sum
// over whatever columns their lanes hold), all in block g / 2 of the stage's
// two.  Loads that write LDS bring activations three stages ahead, weights by
// pairs of stages and scales by pairs or (in the large tiles) by eight: what
// these loads cost is the rows they touch, not the bytes, so a row's bytes come
// many at a time.  Activation rows that do not start on 16 bytes go through
// registers.
//
// Measured: 2048 x 13312 x 2048 89 to 93 us (1.2 to 1.26 PFLOP/s; a library bf16
// product of that shape, weights unpacked before, 87), 2048 x 8192 x 4096 106 us
// (1.29).
// A stage of a workgroup takes 1900 clocks of which 1100 are its matrix
// instructions; two workgroups a CU fill some of the rest.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "mx_plan.hpp"
#include "mx_tile.hpp"
#include "q4_lds_dma.hpp"

namespace q4 {
namespace {

struct TileArgs {
  const uint16_t *x;
  const uint8_t *w, *sw;
  void *y;
  int64_t M, N;
  int K, KB;
  int tiles_m, tiles_n;
  int whole;   // workgroups with a whole tile; each later one has a quarter of one
};

// LDS of a group of waves: three stages of activation rows of 128 bytes; two
// pairs of stages of weight rows of 64 bytes; two buffers of the scales of a
// pair.  SB: the bytes of a row's scales that one lane loads: 4 (rows of scales
// that start on 4 bytes), 1 (any rows; slots of 4 bytes).
template <int BN, int BM, int SB>
struct Lds {
  static constexpr int x = 0, x_stage = BM * 128;
  static constexpr int w = x + 3 * x_stage, w_pair = BN * 64;
  static_assert(SB == 4 || SB == 1, "scales by the dword or by the byte");
  static constexpr int s = w + 2 * w_pair, s_row = SB == 4 ? 4 : 16, s_buf = BN * s_row;
  static constexpr int bytes = s + 2 * s_buf;
};

// The tile of rows m0 .. and weight rows n0 .. by KG groups of NW waves, each
// with a part of K; in a group WN waves lie side by side along the weight
// rows; a wave has 16 TN weight rows by 16 TM rows.
template <int KG, int NW, int WN, int TN, int TM, bool XAL, int SB, bool BOUT>
__device__ __forceinline__ void tile_body(const TileArgs &a, int64_t m0, int64_t n0) {
  extern __shared__ __align__(16) uint8_t smem0[];
  constexpr int WM = NW / WN, BN = 16 * WN * TN, BM = 16 * WM * TM;
  using L = Lds<BN, BM, SB>;
  // loads of a wave: activations in a stage, weights in a pair
  constexpr int nX = BM / 8 / NW, nW = BN / 16 / NW;
  static_assert(nX * 8 * NW == BM && nW * 16 * NW == BN, "whole loads");

  const int rows_m = min(static_cast<int>(a.M - m0), BM);
  const int rows_n = min(static_cast<int>(a.N - n0), BN);
  const int K = a.K, KB = a.KB, all = (K + 63) >> 6;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = KG > 1 ? wave % NW : wave, kg = KG > 1 ? wave / NW : 0;
  // this group's stages, a whole number of pairs
  const int steps = KG > 1 ? ((all + KG - 1) / KG + 1) & ~1 : all, first = kg * steps;
  uint8_t *smem = smem0 + kg * L::bytes;
  const int wn = wv / WM, wm = wv % WM;
  const int r = lane & 15, g = lane >> 4;

  const uint16_t *xt = a.x + m0 * K;
  const __amdgpu_buffer_rsrc_t rs_x = rsrc(xt, rows_m * 2 * K);
  const __amdgpu_buffer_rsrc_t rs_w = rsrc(a.w + n0 * KB * 16, rows_n * KB * 16);
  const __amdgpu_buffer_rsrc_t rs_s = rsrc(a.sw + n0 * KB, rows_n * KB);
  const uint32_t lds0 = lds_addr(smem);

  // Staging.  Rows past the tile's end and columns past K lie past the
  // buffer's range (or are sent there) and come as zeros, and so do whole
  // stages past the last one.
  // Activations: a load fills 8 LDS rows, lane i at row i / 8, position i % 8,
  // which holds chunk (i % 8) ^ (row / 2 % 8): 16 neighbouring rows then have a
  // chunk in the 16 different places that one clock reads.
  const int lrow = lane >> 3;
  auto chunk = [&](int j) { return (lane & 7) ^ (lrow >> 1) ^ (4 * ((nX * wv + j) & 1)); };   // of load j
  const int x_row0 = 8 * nX * wv + lrow;
  auto issue_x = [&](int slot, int s) {
#pragma unroll
    for (int j = 0; j < nX; ++j) {
      const int k = 64 * s + 8 * chunk(j);
      dma16(rs_x, lds0 + L::x + slot * L::x_stage + (nX * wv + j) * 1024, k < K ? ((x_row0 + 8 * j) * K + k) * 2 : kFar, 0);
    }
  };
  // Weights: a load fills 16 rows of the order w_row; lane i at row i / 4,
  // position i % 4, which holds block (i % 4) ^ (row / 4): 16 rows have a
  // block in 16 different places.
  auto row_of = [](int t, int i) { return 32 * (t >> 1) + w_row<BOUT>(t & 1, i); };
  const int c_w = (lane & 3) ^ ((lane >> 4) & 3);
  auto issue_w = [&](int d) {   // pair d of the group
    const int b = 2 * first + 4 * d + c_w;
#pragma unroll
    for (int j = 0; j < nW; ++j) {
      const int t = nW * wv + j;
      dma16(rs_w, lds0 + L::w + (d & 1) * L::w_pair + t * 1024, b < KB ? (row_of(t, lane >> 2) * KB + b) * 16 : kFar, 0);
    }
  };
  auto issue_s = [&](int d) {   // the scales of pair d
    const int b = 2 * first + 4 * d;
    const uint32_t to = lds0 + L::s + (d & 1) * L::s_buf;
    if constexpr (SB == 1) {
      // lane i: byte i % 4 of row i / 4
      const int i = b + (lane & 3);
#pragma unroll
      for (int j = 0; j < nW; ++j) {
        const int t = nW * wv + j;
        dma1(rs_s, to + t * 256, i < KB ? row_of(t, lane >> 2) * KB + i : kFar, 0);
      }
    } else if (wv < BN / 64) {   // a row a lane
      static_assert(BN / 64 <= NW, "a load a wave");
      const int o = b < KB ? row_of(4 * wv + g, r) * KB + b : kFar;
      dma4(rs_s, to + wv * 256, o, 0);
    }
  };
  // Activations through registers (XAL false); rows past the end are the last
  // one again.
  Run8<true> xr[XAL ? 1 : nX];
  auto fetch = [&](int s) {
#pragma unroll
    for (int j = 0; j < nX; ++j) {
      const int k = 64 * s + 8 * chunk(j);
      const int64_t i = static_cast<int64_t>(min(x_row0 + 8 * j, rows_m - 1)) * K + k;
      Run8<true> &v = xr[XAL ? 0 : j];
      if (64 * s + 64 <= K) {
        v.load(xt, i);
      } else {
        v.zero();
        if (k + 8 <= K) v.load(xt, i);
        else if (k < K) v.load_part(xt, i, K - k);
      }
    }
  };
  auto put = [&](int slot) {
#pragma unroll
    for (int j = 0; j < nX; ++j) {
      const uint32_t *v = xr[XAL ? 0 : j].v;
      *reinterpret_cast<uint4 *>(smem + L::x + slot * L::x_stage + (nX * wv + j) * 1024 + lane * 16) =
          make_uint4(v[0], v[1], v[2], v[3]);
    }
  };

  // Fragments: activations of half j of a stage, weights and scales of a stage.
  struct Weights {
    uint2 c[TN];
    uint32_t s[TN];
  };
  const int x_base = L::x + (16 * TM * wm + r) * 128;
  const int pos[2] = {((2 * g) ^ (r >> 1)) << 4, ((2 * g + 1) ^ (r >> 1)) << 4};
  auto read_x = [&](uint4 (&f)[TM], int slot, int j) {
#pragma unroll
    for (int t = 0; t < TM; ++t) f[t] = load16(smem + x_base + slot * L::x_stage + pos[j] + t * 2048);
  };
  auto read_w = [&](Weights &f, int s) {   // s: stage of the group
    const int blk = 2 * (s & 1) + (g >> 1);
    const uint8_t *w = smem + L::w + ((s >> 1) & 1) * L::w_pair + TN * wn * 1024 + r * 64 + ((blk ^ (r >> 2)) << 4) + 8 * (g & 1);
    const uint8_t *sc = smem + L::s + ((s >> 1) & 1) * L::s_buf + (TN * wn * 16 + r) * L::s_row +
                        (SB == 4 ? blk : 4 * blk);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      f.c[t] = *reinterpret_cast<const uint2 *>(w + t * 1024);
      f.s[t] = sc[t * 16 * L::s_row];
    }
  };
  f32x4 acc[TM][TN] = {};
  auto multiply = [&](const uint4 (&x)[TM], const Weights &w, int j) {
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      const uint4 wf = mx_decode8_bf16(j ? w.c[tn].y : w.c[tn].x, mx_scale(w.s[tn]));
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc[tm][tn] = mfma_bf16_16x16x32(wf, x[tm], acc[tm][tn]);
    }
  };

  // The barrier in the middle of stage s says that stage s + 1 has landed and
  // that stage s has been read; the second half of s is multiplied while the
  // first of s + 1 is read.  Stage s + 3 then takes the place of s and, after
  // odd stages, pair (s + 3) / 2 + ... the place of the pair that s ends.
  uint4 x0[TM], x1[TM];
  Weights w0, w1;
  issue_s(0);
  issue_s(1);
  issue_w(0);
  if constexpr (XAL) {
    issue_x(0, first);
    issue_x(1, first + 1);
    issue_x(2, first + 2);
    issue_w(1);
    wait_vmcnt<2 * nX + nW>();
  } else {
    issue_w(1);
    fetch(first);
    put(0);
    fetch(first + 1);
    put(1);
    fetch(first + 2);
    wait_vmcnt<0>();
  }
  lds_barrier();
  read_w(w0, 0);
  read_x(x0, 0, 0);
  int c = 0;   // s % 3
  auto step = [&](int s, auto odd_c, Weights &w, Weights &next) {
    constexpr bool ODD = decltype(odd_c)::value;
    const int c1 = c == 2 ? 0 : c + 1;
    read_x(x1, c, 1);
    multiply(x0, w, 0);
    if constexpr (XAL) {
      wait_vmcnt<ODD ? nX : nX + nW>();
    } else {
      wait_vmcnt<0>();
      put(c == 0 ? 2 : c - 1);   // stage s + 2
    }
    lds_barrier();
    if constexpr (ODD) issue_s((s >> 1) + 2);
    if constexpr (XAL) issue_x(c, first + s + 3);
    if constexpr (ODD) issue_w((s >> 1) + 2);
    if constexpr (!XAL) fetch(first + s + 3);
    read_w(next, s + 1);
    read_x(x0, c1, 0);
    multiply(x1, w, 1);
    c = c1;
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, std::false_type{}, w0, w1);
    if (s + 1 < steps) step(s + 1, std::true_type{}, w1, w0);
  }
  wait_vmcnt<0>();   // the loads past the end land before the LDS is used again

  if constexpr (KG > 1) {
    // the groups' sums, in their order; group i takes the 16 rows i, i + KG ..
    f32x4 *part = reinterpret_cast<f32x4 *>(smem0) + (wv * 64 + lane);
    constexpr int kPart = NW * 64;
    static_assert(TM * TN * kPart * 16 <= L::bytes, "the sums fit");
    lds_barrier();
#pragma unroll
    for (int t = 0; t < TM * TN; ++t) part[(kg * TM * TN + t) * kPart] = acc[t / TN][t % TN];
    lds_barrier();
    for (int tm = kg; tm < TM; tm += KG) {
      f32x4 sum[1][TN];
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        sum[0][tn] = part[(tm * TN + tn) * kPart];
#pragma unroll
        for (int i = 1; i < KG; ++i) sum[0][tn] += part[((i * TM + tm) * TN + tn) * kPart];
      }
      store_tile<TN, 1, BOUT>(a.y, a.M, a.N, m0 + 16 * (TM * wm + tm), n0 + 16 * TN * wn, sum);
    }
  } else {
    store_tile<TN, TM, BOUT>(a.y, a.M, a.N, m0 + 16 * TM * wm, n0 + 16 * TN * wn, acc);
  }
}

template <int KG, int NW, int WN, int TN, int TM, bool XAL, int SB, bool BOUT>
__global__ __launch_bounds__(64 * NW * KG, NW * KG == 4 ? 2 : NW * KG / 4) void mx_tiled_w4a16(TileArgs a) {
  constexpr int BN = 16 * WN * TN, BM = 16 * (NW / WN) * TM;
  const TileAt at = tile_at(xcd_run(static_cast<int>(blockIdx.x), a.whole), a.tiles_m, a.tiles_n);
  tile_body<KG, NW, WN, TN, TM, XAL, SB, BOUT>(a, static_cast<int64_t>(at.m) * BM, static_cast<int64_t>(at.n) * BN);
}

// Large products, 32 x 32 x 16 instructions, two workgroups a CU: two stages of
// activations, two pairs of stages of weights, one barrier a stage.
template <int BN, int BM, int SB>
struct LargeLds {
  static constexpr int x_stage = BM * 128, w = 2 * x_stage, w_pair = BN * 64;
  static constexpr int s = w + 2 * w_pair, s_buf = BN * SB, bytes = s + 2 * s_buf;
};

template <int TN, int TM, int SB, bool BOUT>
__device__ __forceinline__ void large_body(const TileArgs &a, int64_t m0, int64_t n0) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int BN = 128 * TN, BM = 32 * TM;
  using L = LargeLds<BN, BM, SB>;
  constexpr int nX = BM / 32, nW = BN / 64;   // loads of a wave: activations in a stage, weights in a pair
  static_assert(nX % 2 == 0, "a wave's loads begin at 16 rows");

  const int rows_m = min(static_cast<int>(a.M - m0), BM), rows_n = min(static_cast<int>(a.N - n0), BN);
  const int K = a.K, KB = a.KB, steps = (K + 63) >> 6;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;

  const __amdgpu_buffer_rsrc_t rs_x = rsrc(a.x + m0 * K, rows_m * 2 * K);
  const __amdgpu_buffer_rsrc_t rs_w = rsrc(a.w + n0 * KB * 16, rows_n * KB * 16);
  const __amdgpu_buffer_rsrc_t rs_s = rsrc(a.sw + n0 * KB, rows_n * KB);
  const uint32_t lds0 = lds_addr(smem);

  // LDS row i of the weights is row w_row32(i % 32) of its 32.  Activations:
  // lane i at row i / 8, position i % 8, which holds chunk (i % 8) ^ (row / 2 %
  // 8).  Weights: row i / 4, position i % 4, which holds block (i % 4) ^ (row /
  // 4 % 4).  Either way 16 rows have a chunk in the 16 different places that
  // one clock reads.
  const int c_x = (lane & 7) ^ (lane >> 4), x_row0 = 8 * nX * wv + (lane >> 3);   // chunk c_x in even loads
  const int c_w = (lane & 3) ^ (lane >> 4);
  auto issue_x = [&](int s) {
#pragma unroll
    for (int j = 0; j < nX; ++j) {
      const int k = 64 * s + 8 * (c_x ^ (4 * (j & 1)));
      dma16(rs_x, lds0 + (s & 1) * L::x_stage + (nX * wv + j) * 1024, k < K ? ((x_row0 + 8 * j) * K + k) * 2 : kFar, 0);
    }
  };
  auto issue_w = [&](int d) {   // pair d
    const int b = 4 * d + c_w;
#pragma unroll
    for (int j = 0; j < nW; ++j) {
      const int i = 16 * (nW * wv + j), row = (i & ~31) + w_row32((i & 31) + (lane >> 2));
      dma16(rs_w, lds0 + L::w + (d & 1) * L::w_pair + i * 64, b < KB ? (row * KB + b) * 16 : kFar, 0);
    }
  };
  auto issue_s = [&](int d) {   // the scales of pair d and (SB = 16) the three after it
    if (wv < BN / 64) {
      const int b = 4 * d, o = b < KB ? (64 * wv + 32 * h + w_row32(r)) * KB + b : kFar;
      const uint32_t to = lds0 + L::s + ((SB == 16 ? d >> 2 : d) & 1) * L::s_buf;
      if constexpr (SB == 16) dma16(rs_s, to + wv * 1024, o, 0);
      else dma4(rs_s, to + wv * 256, o, 0);
    }
  };

  // In instruction j of a stage's four lane (r, h) has columns 32 h + 8 j .. of
  // row r: a dword of its block h.
  f32x16 acc[TM][TN] = {};
  const int w_base = L::w + TN * wv * 2048 + r * 64, s_base = L::s + (32 * TN * wv + r) * SB;
  auto compute = [&](int s, auto odd_c) {
    constexpr int ODD = decltype(odd_c)::value;
    const int d = s >> 1, blk = 2 * ODD + h;
    const uint8_t *st = smem + ODD * L::x_stage + r * 128;
    const uint8_t *sw = smem + w_base + (d & 1) * L::w_pair + ((blk ^ ((r >> 2) & 3)) << 4);
    const uint8_t *sc = smem + s_base + (SB == 16 ? ((d >> 2) & 1) * L::s_buf + 4 * (d & 3) : (d & 1) * L::s_buf) + blk;
    uint32_t c[TN][4];
    float scale[TN];
    uint4 x[4][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const uint4 v = load16(sw + t * 2048);
      c[t][0] = v.x, c[t][1] = v.y, c[t][2] = v.z, c[t][3] = v.w;
      scale[t] = mx_scale(sc[t * 32 * SB]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < TM; ++t) x[j][t] = load16(st + (((4 * h + j) ^ ((r >> 1) & 7)) << 4) + t * 4096);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const uint4 wf = mx_decode8_bf16(c[tn][j], scale[tn]);
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) acc[tm][tn] = mfma_bf16_32x32x16(wf, x[j][tm], acc[tm][tn]);
      }
  };

  // The barrier before step s says that stage s has landed and that stage
  // s - 1 has been read, so its place can take stage s + 1; after even ones
  // pair s / 2 + 1 takes the place of the pair before s's.
  issue_s(0);
  issue_w(0);
  issue_x(0);
  for (int s = 0; s < steps; s += 2) {
    wait_vmcnt<0>();
    lds_barrier();
    const int d = s / 2 + 1;
    if (SB != 16 || (d & 3) == 0) issue_s(d);
    issue_x(s + 1);
    issue_w(d);
    compute(s, std::integral_constant<int, 0>{});
    if (s + 1 < steps) {
      wait_vmcnt<nW>();   // all but the weights of the next pair
      lds_barrier();
      issue_x(s + 2);
      compute(s + 1, std::integral_constant<int, 1>{});
    }
  }
  wait_vmcnt<0>();   // the loads past the end land before the LDS is handed on
  if constexpr (TN > 1) {
    static_assert(4 * 64 * TM * TN * 32 <= L::bytes, "the waves' results fit");
    lds_barrier();
    store_lines<TM, TN, BOUT>(smem + wv * (64 * TM * TN * 32), a.y, a.M, a.N, m0, n0 + 32 * TN * wv, acc);
  } else {
    // lane (c, h) has row c of each 32 activation rows
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
      if (m0 + 32 * tm + r < a.M) store_16<BOUT>(a.y, m0 + 32 * tm + r, n0 + 32 * wv + 16 * h, a.N, acc[tm][0]);
  }
}

// Whole tiles of 128 x 256, and the last ones in quarters.
template <int SB, bool BOUT>
__global__ __launch_bounds__(256, 2) void mx_large_w4a16(TileArgs a) {
  const int id = static_cast<int>(blockIdx.x);
  if (id < a.whole) {
    const TileAt at = tile_at(xcd_run(id, a.whole), a.tiles_m, a.tiles_n);
    large_body<2, 4, SB, BOUT>(a, 128 * static_cast<int64_t>(at.m), 256 * static_cast<int64_t>(at.n));
  } else {
    const int q = xcd_run(id - a.whole, static_cast<int>(gridDim.x) - a.whole);
    const TileAt at = tile_at(a.whole + (q >> 2), a.tiles_m, a.tiles_n);
    const int64_t m0 = 128 * static_cast<int64_t>(at.m) + 64 * (q & 1);
    const int64_t n0 = 256 * static_cast<int64_t>(at.n) + 128 * ((q >> 1) & 1);
    if (m0 >= a.M || n0 >= a.N) return;   // the whole workgroup
    large_body<1, 2, SB, BOUT>(a, m0, n0);
  }
}

template <auto Kernel, int Lds>
hipError_t launch(const TileArgs &a, int grid, int threads, hipStream_t st) {
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, Lds);
  if (set != hipSuccess) return set;
  Kernel<<<static_cast<unsigned>(grid), threads, Lds, st>>>(a);
  return hipGetLastError();
}

template <int KG, int NW, int WN, int TN, int TM, bool XAL, int SB, bool BOUT>
hipError_t go(TileArgs a, hipStream_t st) {
  constexpr int BN = 16 * WN * TN, BM = 16 * (NW / WN) * TM;
  a.tiles_m = static_cast<int>((a.M + BM - 1) / BM);
  a.tiles_n = static_cast<int>((a.N + BN - 1) / BN);
  a.whole = a.tiles_m * a.tiles_n;
  return launch<mx_tiled_w4a16<KG, NW, WN, TN, TM, XAL, SB, BOUT>, KG * Lds<BN, BM, SB>::bytes>(a, a.whole, 64 * NW * KG, st);
}

template <int SB, bool BOUT>
hipError_t go_large(TileArgs a, int cus, hipStream_t st) {
  a.tiles_m = static_cast<int>((a.M + 127) / 128);
  a.tiles_n = static_cast<int>((a.N + 255) / 256);
  const int tiles = a.tiles_m * a.tiles_n;
  a.whole = tiles / cus * cus;
  return launch<mx_large_w4a16<SB, BOUT>, LargeLds<256, 128, SB>::bytes>(a, a.whole + 4 * (tiles - a.whole), 256, st);
}

template <bool XAL, int SB, bool BOUT>
hipError_t pick(const TileArgs &a, hipStream_t st) {
  constexpr int SK = SB == 1 ? 1 : 4;   // of the tiles that do not take scales 16 at a time
  constexpr bool large = XAL && SB > 1;
  const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
  switch (mx_w4a16_tile(a.M, a.N, cus, large)) {
    case MxW4A16Tile::k32x64: return go<4, 4, 2, 2, 1, XAL, SK, BOUT>(a, st);
    case MxW4A16Tile::k64x64: return go<2, 4, 2, 2, 2, XAL, SK, BOUT>(a, st);
    case MxW4A16Tile::k64x128: return go<2, 4, 4, 2, 4, XAL, SK, BOUT>(a, st);
    case MxW4A16Tile::kLarge:
      if constexpr (large) return go_large<SB, BOUT>(a, cus, st);
      return hipErrorInvalidValue;   // not chosen
    default: return go<1, 4, 4, 2, 8, XAL, SK, BOUT>(a, st);
  }
}

}  // namespace

// Ranges of the tiles' buffers in 30 bits, tile counts in 31.
bool mx_tiled_w4a16_ok(int64_t M, int64_t N, int64_t K) {
  return K <= (int64_t(1) << 20) && ((M + 63) / 64) * ((N + 63) / 64) < (int64_t(1) << 28);
}

hipError_t launch_mx_tiled_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                 int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const TileArgs a = {x, wq, sw, y, M, N, static_cast<int>(K), static_cast<int>((K + 31) / 32), 0, 0, 0};
  const auto at = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const bool xal = K % 8 == 0 && at(x, 16);
  const int sb = a.KB % 16 == 0 && at(sw, 16) ? 16 : a.KB % 4 == 0 && at(sw, 4) ? 4 : 1;
  if (xal && sb == 16) return y_bf16 ? pick<true, 16, true>(a, st) : pick<true, 16, false>(a, st);
  if (xal && sb == 4) return y_bf16 ? pick<true, 4, true>(a, st) : pick<true, 4, false>(a, st);
  if (xal) return y_bf16 ? pick<true, 1, true>(a, st) : pick<true, 1, false>(a, st);
  // rows through registers: scales by the byte
  return y_bf16 ? pick<false, 1, true>(a, st) : pick<false, 1, false>(a, st);
}

}  // namespace q4

// bf16 activations times MX FP4 weights for many activation rows: LDS-tiled
// bf16 matrix products.
//
//   y[m,n] = sum_k x[m,k] cw[n,k] 2^(sw[n,k/32] - 127)
//
// The weights stay packed up to the registers: a lane takes 8 codes (a dword)
// and its block's scale to 8 bf16 values in four conversions, exactly.
// K goes in stages of 64 columns through a ring of three in LDS, requested
// two stages ahead by loads that write LDS; activation rows that do not start
// on 16 bytes go through registers instead, one stage ahead.  In a stage lane
// (r, g) holds columns 16 g .. 16 g + 15 of row r, 8 for each of two matrix
// instructions (which sum over whatever columns their lanes hold), all in
// block g / 2 of the stage's two.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "mx_tile.hpp"
#include "q4_lds_dma.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 3;

struct TileArgs {
  const uint16_t *x;
  const uint8_t *w, *sw;
  void *y;
  int64_t M, N;
  int K, KB;
  int tiles_m, tiles;
};

// LDS of a stage: activation rows of 128 bytes; weights by 16 rows, the first
// blocks of the 16 and then their second blocks; scales in slots of 4 bytes,
// a row's two in one (SAL: rows of scales that start on 2 bytes) or one each.
template <int TN, int TM, bool SAL>
constexpr int stage_bytes() {
  return 32 * TM * 128 + 32 * TN * 32 + 32 * TN * (SAL ? 4 : 8);
}

template <int TN, int TM, bool XAL, bool SAL, bool BOUT>
__global__ __launch_bounds__(kThreads, 2) void mx_tiled_w4a16(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int BN = 32 * TN, BM = 32 * TM;
  constexpr int kStage = stage_bytes<TN, TM, SAL>();
  constexpr int kW = BM * 128, kS = kW + BN * 32;
  constexpr int nW = TN >= 4 ? TN / 4 : 1;                       // weight loads of a wave in a stage
  constexpr int scale_loads = SAL ? TN / 2 : TN;                 // of the workgroup
  constexpr int nS = scale_loads >= 4 ? scale_loads / 4 : 1;     // of a wave

  const TileAt at = tile_at(a.tiles, a.tiles_m);
  const int64_t m0 = static_cast<int64_t>(at.m) * BM, n0 = static_cast<int64_t>(at.n) * BN;
  const int rows_m = static_cast<int>(min(a.M - m0, static_cast<int64_t>(BM)));
  const int rows_n = static_cast<int>(min(a.N - n0, static_cast<int64_t>(BN)));
  const int K = a.K, KB = a.KB, steps = (K + 63) >> 6;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv >> 1, wm = wv & 1;
  const int r = lane & 15, g = lane >> 4;

  const uint16_t *xt = a.x + m0 * K;
  const __amdgpu_buffer_rsrc_t rs_x = rsrc(xt, rows_m * 2 * K);
  const __amdgpu_buffer_rsrc_t rs_w = rsrc(a.w + n0 * KB * 16, rows_n * KB * 16);
  const __amdgpu_buffer_rsrc_t rs_s = rsrc(a.sw + n0 * KB, rows_n * KB);
  const uint32_t lds0 = lds_addr(smem);

  // Staging.  Activations: a wave's load fills 8 LDS rows, lane i at row
  // i / 8, position i % 8, which holds chunk (i % 8) ^ (row % 8): 8
  // neighbouring rows then have a chunk in 8 different places.  Rows past the
  // tile's end and columns past K lie past the buffer's range (or are sent
  // there) and come as zeros, and so do whole stages past the last one.
  const int lrow = lane >> 3, c_x = (lane & 7) ^ lrow;
  const int x_row0 = 8 * TM * wv + lrow;
  // Weights: lane i of load l has tile 2 l + i / 32, block i / 16 % 2, row
  // i % 16 of the tile.
  auto row_of = [&](int t, int i) { return 32 * (t >> 1) + w_row<BOUT>(t & 1, i); };
  const int w_half = (lane >> 4) & 1, w_off = row_of(lane >> 5, r) * KB;
  const int s_off = SAL ? row_of(lane >> 4, r) * KB : w_off + w_half;
  const int s_half = SAL ? 0 : w_half;
  auto issue = [&](int stage, int s) {
    const uint32_t st = lds0 + stage * kStage;
    if constexpr (XAL) {
      const int k = 64 * s + 8 * c_x;
      const int o = k < K ? (x_row0 * K + k) * 2 : kFar;
#pragma unroll
      for (int j = 0; j < TM; ++j) dma16(rs_x, st + (TM * wv + j) * 1024, k < K ? o + 16 * j * K : kFar, 0);
    }
    const bool in_w = 2 * s + w_half < KB, in_s = 2 * s + s_half < KB;
#pragma unroll
    for (int j = 0; j < nW; ++j) {
      const int l = TN >= 4 ? nW * wv + j : wv % TN;   // TN = 2: two waves bring the same rows
      dma16(rs_w, st + kW + l * 1024, in_w ? (w_off + 32 * l * KB + 2 * s + w_half) * 16 : kFar, 0);
    }
#pragma unroll
    for (int j = 0; j < nS; ++j) {
      const int l = scale_loads >= 4 ? nS * wv + j : wv % scale_loads;
      const int o = in_s ? s_off + (SAL ? 64 : 32) * l * KB + 2 * s : kFar;
      if constexpr (SAL) dma2(rs_s, st + kS + l * 256, o, 0);
      else dma1(rs_s, st + kS + l * 256, o, 0);
    }
  };
  // Activations through registers (XAL false).
  Run8<true> xr[XAL ? 1 : TM];
  auto fetch = [&](int s) {
    const int k = 64 * s + 8 * c_x;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int row = x_row0 + 8 * j;
      xr[XAL ? 0 : j].zero();
      if (row < rows_m) {
        const int64_t i = static_cast<int64_t>(row) * K + k;
        if (k + 8 <= K) xr[XAL ? 0 : j].load(xt, i);
        else if (k < K) xr[XAL ? 0 : j].load_part(xt, i, K - k);
      }
    }
  };
  auto put = [&](int stage) {
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const uint32_t *v = xr[XAL ? 0 : j].v;
      *reinterpret_cast<uint4 *>(smem + stage * kStage + (TM * wv + j) * 1024 + lane * 16) =
          make_uint4(v[0], v[1], v[2], v[3]);
    }
  };

  f32x4 acc[TM][TN] = {};
  const int x_base = (16 * TM * wm + r) * 128, w_base = kW + TN * wn * 512 + (g >> 1) * 256 + r * 16 + (g & 1) * 8;
  const int s_base = kS + (SAL ? (TN * wn * 16 + r) * 4 + (g >> 1) : TN * wn * 128 + (g >> 1) * 64 + r * 4);
  const int pos[2] = {((2 * g) ^ (r & 7)) << 4, ((2 * g + 1) ^ (r & 7)) << 4};
  auto compute = [&](int stage) {
    const uint8_t *st = smem + stage * kStage;
    uint2 c[TN];
    uint32_t sc[TN];
    uint4 xf[2][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      c[t] = *reinterpret_cast<const uint2 *>(st + w_base + t * 512);
      sc[t] = st[s_base + t * (SAL ? 64 : 128)];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < TM; ++t) xf[j][t] = load16(st + x_base + pos[j] + t * 2048);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        const uint4 wf = mx_decode8_bf16(j ? c[tn].y : c[tn].x, mx_scale(sc[tn]));
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) acc[tm][tn] = mfma_bf16_16x16x32(wf, xf[j][tm], acc[tm][tn]);
      }
  };

  // Stage s is read in step s; the barrier before it says that the stage has
  // landed and that the one read in step s - 1 is free.
  issue(0, 0);
  issue(1, 1);
  if constexpr (!XAL) {
    fetch(0);
    put(0);
    fetch(1);
  }
  for (int s = 0, c = 0; s < steps; ++s) {
    const int c1 = c == kStages - 1 ? 0 : c + 1, c2 = c1 == kStages - 1 ? 0 : c1 + 1;
    if constexpr (XAL) {
      wait_vmcnt<TM + nW + nS>();   // all but the loads of stage s + 1
    } else {
      wait_vmcnt<0>();
      put(c1);
    }
    lds_barrier();
    issue(c2, s + 2);
    if constexpr (!XAL) fetch(s + 2);
    compute(c);
    c = c1;
  }
  wait_vmcnt<0>();   // the loads past the end land before the LDS is handed on

  store_tile<TN, TM, BOUT>(a.y, a.M, a.N, m0 + 16 * TM * wm, n0 + 16 * TN * wn, acc);
}

template <int TN, int TM, bool XAL, bool SAL, bool BOUT>
hipError_t go(TileArgs a, hipStream_t st) {
  constexpr int lds = kStages * stage_bytes<TN, TM, SAL>();
  a.tiles_m = static_cast<int>((a.M + 32 * TM - 1) / (32 * TM));
  a.tiles = a.tiles_m * static_cast<int>((a.N + 32 * TN - 1) / (32 * TN));
  static const hipError_t set = hipFuncSetAttribute(
      reinterpret_cast<const void *>(mx_tiled_w4a16<TN, TM, XAL, SAL, BOUT>), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (set != hipSuccess) return set;
  mx_tiled_w4a16<TN, TM, XAL, SAL, BOUT><<<static_cast<unsigned>(a.tiles), kThreads, lds, st>>>(a);
  return hipGetLastError();
}

template <bool XAL, bool SAL, bool BOUT>
hipError_t pick(const TileArgs &a, hipStream_t st) {
  auto tiles = [&](int64_t bn, int64_t bm) { return ((a.N + bn - 1) / bn) * ((a.M + bm - 1) / bm); };
  if (tiles(256, 128) >= 256) return go<8, 4, XAL, SAL, BOUT>(a, st);
  if (tiles(128, 128) >= 256) return go<4, 4, XAL, SAL, BOUT>(a, st);
  return go<2, 2, XAL, SAL, BOUT>(a, st);
}

}  // namespace

// Ranges of the tiles' buffers in 30 bits, tile counts in 31.
bool mx_tiled_w4a16_ok(int64_t M, int64_t N, int64_t K) {
  return K <= (int64_t(1) << 21) && ((M + 63) / 64) * ((N + 63) / 64) < (int64_t(1) << 28);
}

hipError_t launch_mx_tiled_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                 int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const TileArgs a = {x, wq, sw, y, M, N, static_cast<int>(K), static_cast<int>((K + 31) / 32), 0, 0};
  const auto at = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const bool xal = K % 8 == 0 && at(x, 16), sal = a.KB % 2 == 0 && at(sw, 2);
  if (xal && sal) return y_bf16 ? pick<true, true, true>(a, st) : pick<true, true, false>(a, st);
  if (xal) return y_bf16 ? pick<true, false, true>(a, st) : pick<true, false, false>(a, st);
  // rows through registers: scales by the byte
  return y_bf16 ? pick<false, false, true>(a, st) : pick<false, false, false>(a, st);
}

}  // namespace q4

// W4A4 in MX FP4 for many activation rows: LDS-tiled scaled matrix products.
//
//   y[m,n] = sum_b 2^(sx[m,b] + sw[n,b] - 254) sum_{k in b} cx[m,k] cw[n,k]
//
// The scaled 16 x 16 x 128 instruction takes the format as stored: a lane's
// operand is one block (16 bytes) and a byte of scale, so nothing is unpacked
// and the sums stay in f32.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "mx_tile.hpp"
#include "q4_lds_dma.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kRow = 128;        // bytes of a row in a stage: 8 blocks, 256 columns

struct TileArgs {
  const uint8_t *x, *sx, *w, *sw;
  void *y;
  int64_t M, N;
  int KB;
  int tiles_m, tiles;
};

// LDS of a stage: weight rows, activation rows, and their scales: 8 bytes a
// row, or (rows whose scales do not start on a dword) 8 dwords of one byte.
template <int BN, int BM, bool AL>
constexpr int stage_bytes() {
  return (BN + BM) * (kRow + (AL ? 8 : 32));
}

// Chunk c of LDS row `row` sits at c ^ swz(row), which is c ^ (i % 8) for the
// row of lane i in either order: 8 neighbouring lanes read 8 different chunks.
template <bool BOUT>
__device__ __forceinline__ int w_swz(int row) {
  return BOUT ? (row & 3) | ((row >> 1) & 4) : row & 7;
}

// Waves 2 x 2, each 16 TN weight rows by 16 TM activation rows.
template <int TN, int TM, bool AL, bool BOUT>
__global__ __launch_bounds__(kThreads, TN * TM > 32 ? 1 : 2) void mx_tiled_w4a4(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int BN = 32 * TN, BM = 32 * TM;
  constexpr int kStage = stage_bytes<BN, BM, AL>();
  constexpr int kX = BN * kRow, kSW = (BN + BM) * kRow, kSX = kSW + BN * (AL ? 8 : 32);

  const TileAt at = tile_at(xcd_run(static_cast<int>(blockIdx.x), a.tiles), a.tiles_m, a.tiles / a.tiles_m);
  const int64_t m0 = static_cast<int64_t>(at.m) * BM, n0 = static_cast<int64_t>(at.n) * BN;
  const int rows_m = static_cast<int>(min(a.M - m0, static_cast<int64_t>(BM)));
  const int rows_n = static_cast<int>(min(a.N - n0, static_cast<int64_t>(BN)));
  const int KB = a.KB, pitch = KB * 16, steps = (KB + 7) >> 3;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv >> 1, wm = wv & 1;
  const int r = lane & 15, g = lane >> 4;

  const __amdgpu_buffer_rsrc_t rs_w = rsrc(a.w + n0 * pitch, rows_n * pitch);
  const __amdgpu_buffer_rsrc_t rs_x = rsrc(a.x + m0 * pitch, rows_m * pitch);
  const __amdgpu_buffer_rsrc_t rs_sw = rsrc(a.sw + n0 * KB, rows_n * KB);
  const __amdgpu_buffer_rsrc_t rs_sx = rsrc(a.sx + m0 * KB, rows_m * KB);
  const uint32_t lds0 = lds_addr(smem);

  // Staging.  A wave's load fills 8 LDS rows: lane i lands at row i / 8,
  // position i % 8.  Rows past the tile's end and chunks from KB on lie past
  // the buffer's range (or are sent there) and come as zeros, and so does the
  // whole step past the last one.
  const int lrow = lane >> 3, lpos = lane & 7;
  const int c_w[2] = {lpos ^ w_swz<BOUT>(lrow), lpos ^ w_swz<BOUT>(lrow + 8)}, c_x = lpos ^ (lrow & 7);
  const int p_w = (8 * TN * wv + lrow) * pitch, p_x = (8 * TM * wv + lrow) * pitch;
  const int s_b = AL ? 4 * (lane & 1) : lpos;
  auto issue = [&](int stage, int s) {
    const uint32_t st = lds0 + stage * kStage;
    const int b0 = 8 * s;
    const bool in_w[2] = {b0 + c_w[0] < KB, b0 + c_w[1] < KB}, in_x = b0 + c_x < KB, in_s = b0 + s_b < KB;
    const int o_w[2] = {p_w + (b0 + c_w[0]) * 16, p_w + (b0 + c_w[1]) * 16}, o_x = p_x + (b0 + c_x) * 16;
#pragma unroll
    for (int j = 0; j < TN; ++j)
      dma16(rs_w, st + (TN * wv + j) * 1024, in_w[j & 1] ? o_w[j & 1] + 8 * j * pitch : kFar, 0);
#pragma unroll
    for (int j = 0; j < TM; ++j) dma16(rs_x, st + kX + (TM * wv + j) * 1024, in_x ? o_x + 8 * j * pitch : kFar, 0);
    if constexpr (AL) {
      // lane i: dword i % 2 of row i / 2
#pragma unroll
      for (int q = 0; q < TN; q += 4) {
        const int l = TN < 4 ? wv % TN : q + wv;   // TN < 4: two waves bring the same rows
        dma4(rs_sw, st + kSW + l * 256, in_s ? (32 * l + (lane >> 1)) * KB + b0 + s_b : kFar, 0);
      }
#pragma unroll
      for (int q = 0; q < TM; q += 4) {
        const int l = TM < 4 ? wv % TM : q + wv;
        dma4(rs_sx, st + kSX + l * 256, in_s ? (32 * l + (lane >> 1)) * KB + b0 + s_b : kFar, 0);
      }
    } else {
      // lane i: byte i % 8 of row i / 8
#pragma unroll
      for (int j = 0; j < TN; ++j)
        dma1(rs_sw, st + kSW + (TN * wv + j) * 256, in_s ? (8 * (TN * wv + j) + lrow) * KB + b0 + s_b : kFar, 0);
#pragma unroll
      for (int j = 0; j < TM; ++j)
        dma1(rs_sx, st + kSX + (TM * wv + j) * 256, in_s ? (8 * (TM * wv + j) + lrow) * KB + b0 + s_b : kFar, 0);
    }
  };

  // Fragments.  Half j (0, 1) of a stage: lane group g takes block 2 g + j.
  struct Frags {
    uint4 w[TN], x[TM];
  };
  struct Scales {
    uint32_t w[TN][AL ? 1 : 2], x[TM][AL ? 1 : 2];
  };
  const int w_base = (16 * TN * wn + w_row<BOUT>(0, r)) * kRow, x_base = kX + (16 * TM * wm + r) * kRow;
  const int pos[2] = {((2 * g) ^ (r & 7)) << 4, ((2 * g + 1) ^ (r & 7)) << 4};
  auto read = [&](Frags &f, int stage, int j) {
    const uint8_t *st = smem + stage * kStage + pos[j];
#pragma unroll
    for (int t = 0; t < TN; ++t) f.w[t] = load16(st + w_base + (w_row<BOUT>(t, 0)) * kRow);
#pragma unroll
    for (int t = 0; t < TM; ++t) f.x[t] = load16(st + x_base + 16 * t * kRow);
  };
  auto read_scales = [&](Scales &s, int stage) {
    const uint8_t *st = smem + stage * kStage;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const int row = 16 * TN * wn + w_row<BOUT>(t, r);
      if constexpr (AL) {
        s.w[t][0] = *reinterpret_cast<const uint16_t *>(st + kSW + row * 8 + 2 * g);
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(st + kSW + row * 32 + 8 * g);
        s.w[t][0] = v.x, s.w[t][1] = v.y;
      }
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int row = 16 * TM * wm + 16 * t + r;
      if constexpr (AL) {
        s.x[t][0] = *reinterpret_cast<const uint16_t *>(st + kSX + row * 8 + 2 * g);
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(st + kSX + row * 32 + 8 * g);
        s.x[t][0] = v.x, s.x[t][1] = v.y;
      }
    }
  };

  f32x4 acc[TM][TN] = {};
  auto multiply = [&](const Frags &f, const Scales &s, auto half_c) {
    constexpr int J = decltype(half_c)::value;
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        if constexpr (AL) acc[tm][tn] = mfma_mx_16x16x128<J>(f.w[tn], f.x[tm], acc[tm][tn], s.w[tn][0], s.x[tm][0]);
        else acc[tm][tn] = mfma_mx_16x16x128<0>(f.w[tn], f.x[tm], acc[tm][tn], s.w[tn][J], s.x[tm][J]);
      }
  };
  // one LDS read between every few matrix instructions
  auto interleave = [&](int reads) {
    constexpr int per = TN * TM / (TN + TM) > 0 ? TN * TM / (TN + TM) : 1;
#pragma unroll
    for (int i = 0; i < reads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, per, 0);
    }
  };

  // Halves in turn: while one is multiplied the next one's fragments are
  // read.  The barrier between a stage's halves says that the next stage has
  // landed and that this one has been read by every wave, so its place can
  // take the stage after the next.
  Frags f0, f1;
  Scales sc;
  issue(0, 0);
  wait_vmcnt<0>();
  lds_barrier();
  issue(1, 1);
  read_scales(sc, 0);
  read(f0, 0, 0);
  for (int s = 0, c = 0; s < steps; ++s, c ^= 1) {
    read(f1, c, 1);
    multiply(f0, sc, std::integral_constant<int, 0>{});
    interleave(TN + TM);
    wait_vmcnt<0>();
    lds_barrier();
    issue(c, s + 2);
    Scales next;
    read(f0, c ^ 1, 0);
    read_scales(next, c ^ 1);
    multiply(f1, sc, std::integral_constant<int, 1>{});
    interleave(2 * (TN + TM));
    sc = next;
  }
  wait_vmcnt<0>();   // the loads past the end land before the LDS is handed on

  store_tile<TN, TM, BOUT>(a.y, a.M, a.N, m0 + 16 * TM * wm, n0 + 16 * TN * wn, acc);
}

template <int TN, int TM, bool AL, bool BOUT>
hipError_t go(TileArgs a, hipStream_t st) {
  constexpr int lds = 2 * stage_bytes<32 * TN, 32 * TM, AL>();
  a.tiles_m = static_cast<int>((a.M + 32 * TM - 1) / (32 * TM));
  a.tiles = a.tiles_m * static_cast<int>((a.N + 32 * TN - 1) / (32 * TN));
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void *>(mx_tiled_w4a4<TN, TM, AL, BOUT>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (set != hipSuccess) return set;
  mx_tiled_w4a4<TN, TM, AL, BOUT><<<static_cast<unsigned>(a.tiles), kThreads, lds, st>>>(a);
  return hipGetLastError();
}

template <bool AL, bool BOUT>
hipError_t pick(const TileArgs &a, hipStream_t st) {
  auto tiles = [&](int64_t bn, int64_t bm) { return ((a.N + bn - 1) / bn) * ((a.M + bm - 1) / bm); };
  if (tiles(256, 256) >= 192) return go<8, 8, AL, BOUT>(a, st);
  return go<4, 4, AL, BOUT>(a, st);
}

}  // namespace

// Ranges of the tiles' buffers in 30 bits, tile counts in 31.
bool mx_tiled_w4a4_ok(int64_t M, int64_t N, int64_t K) {
  return K <= (int64_t(1) << 22) && ((M + 127) / 128) * ((N + 127) / 128) < (int64_t(1) << 30);
}

hipError_t launch_mx_tiled_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                                bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const TileArgs a = {xq, sx, wq, sw, y, M, N, static_cast<int>((K + 31) / 32), 0, 0};
  const auto at4 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
  const bool al = a.KB % 4 == 0 && at4(sx) && at4(sw);
  if (al) return y_bf16 ? pick<true, true>(a, st) : pick<true, false>(a, st);
  return y_bf16 ? pick<false, true>(a, st) : pick<false, false>(a, st);
}

}  // namespace q4

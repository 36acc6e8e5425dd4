// Products with MX FP4 weights for few activation rows (and, block of rows by
// block of rows, for any number):
//   w4a4:  y[m,n] = sum_b 2^(sx[m,b] + sw[n,b] - 254) sum_{k in b} cx[m,k] cw[n,k]
//   w4a16: y[m,n] = sum_k x[m,k] cw[n,k] 2^(sw[n,k/32] - 127)
//
// Bound: the weights' bytes from memory (17 per block of 32), and the latency
// of one round of loads.  A workgroup has 16 weight rows and its four waves
// share out K in steps of 512 columns.  In a step lane (r, g) holds the four
// blocks 4 j + g (j = 0..3) of row r, so that a load's four lanes of a row read
// 64 bytes side by side, and the row's 16 scales, of which byte g of dword j is
// block 4 j + g's.  A matrix instruction sums over whatever columns its lanes
// hold, so the four calls on blocks 4 j + g cover the step once.  All loads of
// a step are under way before the first is used.  The waves' sums meet in LDS
// in wave order: a row's result does not depend on the batch.
//
// Measured, 13312 x 2048 weights (14.5 MB), one row, kernel trace, weights met
// just before | from memory: W4A4 quantized in the call 5.1 us | 6.2 (2.3 TB/s),
// W4A16 5.9 | 6.6.  In a graph of such calls, weights met before: W4A4 4.6,
// W4A16 5.0 and, with 16 rows, 7.8.  What is left over the weights' 2.8 us at a
// copy's rate is the launch and one round of loads from memory.
#include "kernels.hpp"
#include "mx_device.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;

struct GemvArgs {
  const void *x;       // w4a4: packed rows, or f32 / bf16 rows; w4a16: bf16 rows
  const uint8_t *sx;   // w4a4 packed rows
  const uint8_t *w, *sw;
  void *y;
  int64_t M, N, K;
  int KB;
  int64_t first;   // the launch's first block of 16 weight rows
};

// One lane's four blocks of a row, and the scale of each in byte 0 of s[j];
// blocks past KB are zeros under 2^-127.
struct Frag {
  uint4 c[4];
  uint32_t s[4];
};

template <bool STREAM>
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
  if constexpr (STREAM) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)));
  } else {
    return load16(p);
  }
}

// The row's blocks from b0 on (16 of them if whole).
template <bool STREAM>
__device__ __forceinline__ Frag load_frag(const uint8_t *row, const uint8_t *srow, int b0, int g, int KB, bool whole) {
  Frag f;
  if (whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.c[j] = load_codes<STREAM>(row + static_cast<int64_t>(b0 + 4 * j + g) * 16);
    const uint4 s = load_any<uint4>(srow + b0);
    f.s[0] = s.x >> (8 * g), f.s[1] = s.y >> (8 * g), f.s[2] = s.z >> (8 * g), f.s[3] = s.w >> (8 * g);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = b0 + 4 * j + g;
      f.c[j] = make_uint4(0, 0, 0, 0);
      f.s[j] = 0;
      if (b < KB) {
        f.c[j] = load_codes<STREAM>(row + static_cast<int64_t>(b) * 16);
        f.s[j] = srow[b];
      }
    }
  }
  return f;
}

// A step's blocks quantized here (the quantizer's recipe: same codes, same
// scale bytes), a row at a time by the whole wave: lane l forms the codes of
// columns 8 l .. 8 l + 7, and the lanes' blocks meet in LDS of the wave's own.
// (Each lane quantizing its own 128 columns, most of them of rows that are not
// there, took 3 us of a call with one row.)
constexpr int kCodeRow = 272;   // bytes of a row of codes: 16 rows begin 16 bytes apart, modulo 256
struct StepLds {
  uint8_t codes[16 * kCodeRow], scales[16 * 16];
};

// R rows at a time, without a branch among them: past the last one it is
// formed again, in a place that nothing reads.
template <bool BF16, int R>
__device__ __forceinline__ Frag quantize_step(const void *x, int64_t row0, int64_t k0, int64_t K, int rows, StepLds &lds) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t k = k0 + 8 * lane;
  for (int m = 0; m < rows; m += R) {
    Run8<BF16> v[R];
    if (k + 8 <= K) {
#pragma unroll
      for (int i = 0; i < R; ++i) v[i].load(x, row0 + min(m + i, rows - 1) * K + k);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) v[i].load_part(x, row0 + min(m + i, rows - 1) * K + k, static_cast<int>(K - k));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t byte = mx_scale_byte(quad_max(v[i].top()));
      const uint32_t code = byte == 255 ? 0u : v[i].encode(mx_scale(byte));
      *reinterpret_cast<uint32_t *>(lds.codes + (m + i) * kCodeRow + 4 * lane) = code;
      if ((lane & 3) == 0) lds.scales[(m + i) * 16 + (lane >> 2)] = static_cast<uint8_t>(byte);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  Frag f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.c[j] = make_uint4(0, 0, 0, 0);
    f.s[j] = 0;
    if (r < rows) {
      f.c[j] = load16(lds.codes + r * kCodeRow + (4 * j + g) * 16);
      f.s[j] = lds.scales[r * 16 + 4 * j + g];
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  return f;
}

// Sums of the waves in wave order, then the stores: wave t (and t + 4, ...)
// takes the row tile t.
template <int MT, bool BOUT>
__device__ __forceinline__ void join_and_store(const GemvArgs &a, f32x4 (&acc)[MT], int64_t m0, int64_t n0) {
  __shared__ f32x4 part[kWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave < MT) {
    f32x4 v = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[w][wave][lane];
    const int64_t m = m0 + 16 * wave + (lane & 15), n = n0 + 4 * (lane >> 4);
    if (m < a.M && n < a.N) store_y4<BOUT>(a.y, m, n, a.N, v);
  }
}

enum XType { kPacked = 0, kF32 = 1, kBf16 = 2 };

template <int MT, int XT, bool BOUT, int R>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_w4a4(GemvArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = 16 * (a.first + blockIdx.x), m0 = 16 * MT * static_cast<int64_t>(blockIdx.y);
  const int64_t n = min(n0 + r, a.N - 1);
  const uint8_t *wrow = a.w + n * a.KB * 16, *srow = a.sw + n * a.KB;
  const int steps = (a.KB + 15) / 16;
  f32x4 acc[MT] = {};
  for (int s = wave; s < steps; s += kWaves) {
    const int b0 = 16 * s;
    const bool whole = b0 + 16 <= a.KB;
    const Frag wf = load_frag<true>(wrow, srow, b0, g, a.KB, whole);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      Frag xf;
      if constexpr (XT == kPacked) {
        const int64_t m = min(m0 + 16 * t + r, a.M - 1);
        xf = load_frag<false>(static_cast<const uint8_t *>(a.x) + m * a.KB * 16, a.sx + m * a.KB, b0, g, a.KB, whole);
      } else {
        __shared__ __align__(16) StepLds lds[kWaves];
        const int64_t m = m0 + 16 * t;
        xf = quantize_step<XT == kBf16, R>(a.x, m * a.K, 32 * static_cast<int64_t>(b0), a.K,
                                        static_cast<int>(min(a.M - m, static_cast<int64_t>(16))), lds[wave]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t] = mfma_mx_16x16x128<0>(wf.c[j], xf.c[j], acc[t], wf.s[j], xf.s[j]);
    }
  }
  join_and_store<MT, BOUT>(a, acc, m0, n0);
}

// W4A16.  A step's activations come 16 bytes a lane, a row a load, and reach
// the lanes that multiply them through LDS of the wave's own: loaded as they
// are needed, 64 bytes apart, they took as long as the weights.  R: rows that
// there are places for.
constexpr int kRunRow = 1024 + 16;   // bytes of a row in LDS: 16 rows begin 16 bytes apart, modulo 256

template <bool BOUT, int R>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_w4a16(GemvArgs a) {
  extern __shared__ __align__(16) uint8_t runs0[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = 16 * (a.first + blockIdx.x), m0 = 16 * static_cast<int64_t>(blockIdx.y);
  const int64_t n = min(n0 + r, a.N - 1);
  const int rows = static_cast<int>(min(a.M - m0, static_cast<int64_t>(R)));
  const uint8_t *wrow = a.w + n * a.KB * 16, *srow = a.sw + n * a.KB;
  const int steps = (a.KB + 15) / 16;
  uint8_t *runs = runs0 + wave * R * kRunRow;
  const uint8_t *mine = runs + min(r, R - 1) * kRunRow + 64 * g;   // other lanes' columns of the result are not stored
  f32x4 acc[1] = {};
  for (int s = wave; s < steps; s += kWaves) {
    const int64_t k = 512 * static_cast<int64_t>(s) + 8 * lane;
    const Frag wf = load_frag<true>(wrow, srow, 16 * s, g, a.KB, 16 * s + 16 <= a.KB);
    Run8<true> x[R];
    if (k + 8 <= a.K) {
#pragma unroll
      for (int i = 0; i < R; ++i) x[i].load(a.x, (m0 + min(i, rows - 1)) * a.K + k);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) x[i].load_part(a.x, (m0 + min(i, rows - 1)) * a.K + k, static_cast<int>(a.K - k));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      *reinterpret_cast<uint4 *>(runs + i * kRunRow + 16 * lane) = make_uint4(x[i].v[0], x[i].v[1], x[i].v[2], x[i].v[3]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float sc = mx_scale(wf.s[j] & 255u);
      const uint32_t c[4] = {wf.c[j].x, wf.c[j].y, wf.c[j].z, wf.c[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[0] = mfma_bf16_16x16x32(mx_decode8_bf16(c[i], sc), load16(mine + 256 * j + 16 * i), acc[0]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  join_and_store<1, BOUT>(a, acc, m0, n0);
}

// The kernel over all blocks of weight rows, in as few launches as hold them.
template <int MT, class Kernel>
void run_blocks(Kernel kernel, GemvArgs a, int lds, hipStream_t st) {
  constexpr int64_t most = max_groups(64 * kWaves);
  const int64_t blocks = (a.N + 15) / 16;
  for (a.first = 0; a.first < blocks; a.first += most) {
    const int64_t n = blocks - a.first < most ? blocks - a.first : most;
    kernel<<<dim3(static_cast<unsigned>(n), static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT))), 64 * kWaves, lds,
             st>>>(a);
  }
}

// R: rows that the kernel quantizes at a time
template <int MT, int XT, int R = 1>
void run_w4a4(const GemvArgs &a, bool y_bf16, hipStream_t st) {
  run_blocks<MT>(y_bf16 ? mx_gemv_w4a4<MT, XT, true, R> : mx_gemv_w4a4<MT, XT, false, R>, a, 0, st);
}

// As few rows at a time as cover the call, up to 8 (us, N 13312 K 2048, bf16, at
// 1, 4 and 8 rows at a time): one row 4.6, 5.3, 6.3; 4 rows -, 5.2, 6.2; 8 rows
// -, 6.4, 6.2; 16 rows -, 8.8, 8.5.
template <int XT>
void run_w4a4_fused(const GemvArgs &a, bool y_bf16, hipStream_t st) {
  if (a.M == 1) run_w4a4<1, XT, 1>(a, y_bf16, st);
  else if (a.M <= 4) run_w4a4<1, XT, 4>(a, y_bf16, st);
  else run_w4a4<1, XT, 8>(a, y_bf16, st);
}

template <int R>
hipError_t run_w4a16(const GemvArgs &a, bool y_bf16, hipStream_t st) {
  constexpr int lds = kWaves * R * kRunRow;
  const auto kernel = y_bf16 ? mx_gemv_w4a16<true, R> : mx_gemv_w4a16<false, R>;
  if constexpr (lds > 60 * 1024) {   // beside the sums
    static const hipError_t set[2] = {
        hipFuncSetAttribute(reinterpret_cast<const void *>(mx_gemv_w4a16<false, R>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds),
        hipFuncSetAttribute(reinterpret_cast<const void *>(mx_gemv_w4a16<true, R>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds)};
    if (set[y_bf16] != hipSuccess) return set[y_bf16];
  }
  run_blocks<1>(kernel, a, lds, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemv_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                               bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {xq, sx, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32), 0};
  if (M <= 16) run_w4a4<1, kPacked>(a, y_bf16, st);
  else if (M <= 32) run_w4a4<2, kPacked>(a, y_bf16, st);
  else run_w4a4<4, kPacked>(a, y_bf16, st);
  return hipGetLastError();
}

hipError_t launch_mx_gemv_w4a4_fused(const void *x, bool x_bf16, const uint8_t *wq, const uint8_t *sw, void *y,
                                     bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {x, nullptr, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32), 0};
  if (x_bf16) run_w4a4_fused<kBf16>(a, y_bf16, st);
  else run_w4a4_fused<kF32>(a, y_bf16, st);
  return hipGetLastError();
}

hipError_t launch_mx_gemv_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {x, nullptr, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32), 0};
  // As few places as hold the rows (us, N 13312 K 2048, with 1, 4, 8 and 16):
  // one row 4.9, 5.3, 6.4, 7.9; 4 rows -, 5.3, 6.3, 7.8; 8 rows -, -, 6.3, 7.7.
  if (M == 1) return run_w4a16<1>(a, y_bf16, st);
  if (M <= 4) return run_w4a16<4>(a, y_bf16, st);
  if (M <= 8) return run_w4a16<8>(a, y_bf16, st);
  return run_w4a16<16>(a, y_bf16, st);
}

}  // namespace q4

// Products with MX FP4 weights for few activation rows (and, block of rows by
// block of rows, for any number):
//   w4a4:  y[m,n] = sum_b 2^(sx[m,b] + sw[n,b] - 254) sum_{k in b} cx[m,k] cw[n,k]
//   w4a16: y[m,n] = sum_k x[m,k] cw[n,k] 2^(sw[n,k/32] - 127)
//
// Bound: the weights' bytes from memory (17 per block of 32).  A workgroup
// has 16 weight rows and its four waves share out K in steps of 512 columns.
// In a step lane (r, g) holds the four blocks 4 g .. 4 g + 3 of row r: 64
// consecutive bytes of codes and one dword of scales, so the wave reads 256
// consecutive bytes of each row, and the matrix instruction picks the block's
// scale byte out of the dword.  A matrix instruction sums over whatever
// columns its lanes hold, so the four calls on blocks 4 g + j (j = 0..3) cover
// the step once.  The waves' sums meet in LDS in wave order: a row's result
// does not depend on the batch.
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
};

// One lane's four blocks of a row, and their scale bytes; blocks past KB are
// zeros under 2^-127.
struct Frag {
  uint4 c[4];
  uint32_t s;
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

template <bool STREAM>
__device__ __forceinline__ Frag load_frag(const uint8_t *row, const uint8_t *srow, int b0, int KB, bool whole) {
  Frag f;
  if (whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f.c[j] = load_codes<STREAM>(row + static_cast<int64_t>(b0 + j) * 16);
    f.s = load_any<uint32_t>(srow + b0);
  } else {
    f.s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.c[j] = make_uint4(0, 0, 0, 0);
      if (b0 + j < KB) {
        f.c[j] = load_codes<STREAM>(row + static_cast<int64_t>(b0 + j) * 16);
        f.s |= static_cast<uint32_t>(srow[b0 + j]) << (8 * j);
      }
    }
  }
  return f;
}

// The same four blocks quantized here from a float row (the quantizer's
// recipe: same codes, same scale bytes).
template <bool BF16>
__device__ __forceinline__ Frag quantize_frag(const void *x, int64_t row0, int b0, int64_t K) {
  Frag f;
  f.s = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    Run8<BF16> v[4];
    const int64_t k = 32 * static_cast<int64_t>(b0 + j);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ki = k + 8 * i;
      if (ki + 8 <= K) v[i].load(x, row0 + ki);
      else if (ki < K) v[i].load_part(x, row0 + ki, static_cast<int>(K - ki));
      else v[i].zero();
      top = max(top, v[i].top());
    }
    const uint32_t byte = mx_scale_byte(top);
    const float s = mx_scale(byte);
    f.c[j] = make_uint4(v[0].encode(s), v[1].encode(s), v[2].encode(s), v[3].encode(s));
    if (byte == 255) f.c[j] = make_uint4(0, 0, 0, 0);
    f.s |= byte << (8 * j);
  }
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

template <int MT, int XT, bool BOUT>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_w4a4(GemvArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = 16 * static_cast<int64_t>(blockIdx.x), m0 = 16 * MT * static_cast<int64_t>(blockIdx.y);
  const int64_t n = min(n0 + r, a.N - 1);
  const uint8_t *wrow = a.w + n * a.KB * 16, *srow = a.sw + n * a.KB;
  const int steps = (a.KB + 15) / 16;
  f32x4 acc[MT] = {};
  for (int s = wave; s < steps; s += kWaves) {
    const int b0 = 16 * s + 4 * g;
    const bool whole = 16 * s + 16 <= a.KB;
    const Frag wf = load_frag<true>(wrow, srow, b0, a.KB, whole);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t m = min(m0 + 16 * t + r, a.M - 1);
      Frag xf;
      if constexpr (XT == kPacked)
        xf = load_frag<false>(static_cast<const uint8_t *>(a.x) + m * a.KB * 16, a.sx + m * a.KB, b0, a.KB, whole);
      else
        xf = quantize_frag<XT == kBf16>(a.x, m * a.K, b0, a.K);
      acc[t] = mfma_mx_16x16x128<0>(wf.c[0], xf.c[0], acc[t], wf.s, xf.s);
      acc[t] = mfma_mx_16x16x128<1>(wf.c[1], xf.c[1], acc[t], wf.s, xf.s);
      acc[t] = mfma_mx_16x16x128<2>(wf.c[2], xf.c[2], acc[t], wf.s, xf.s);
      acc[t] = mfma_mx_16x16x128<3>(wf.c[3], xf.c[3], acc[t], wf.s, xf.s);
    }
  }
  join_and_store<MT, BOUT>(a, acc, m0, n0);
}

template <int MT, bool BOUT>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_w4a16(GemvArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = 16 * static_cast<int64_t>(blockIdx.x), m0 = 16 * MT * static_cast<int64_t>(blockIdx.y);
  const int64_t n = min(n0 + r, a.N - 1);
  const uint8_t *wrow = a.w + n * a.KB * 16, *srow = a.sw + n * a.KB;
  const int steps = (a.KB + 15) / 16;
  f32x4 acc[MT] = {};
  for (int s = wave; s < steps; s += kWaves) {
    const int b0 = 16 * s + 4 * g;
    const bool whole = 512 * static_cast<int64_t>(s) + 512 <= a.K;
    const Frag wf = load_frag<true>(wrow, srow, b0, a.KB, whole);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float sc = mx_scale((wf.s >> (8 * j)) & 255u);
      const uint32_t c[4] = {wf.c[j].x, wf.c[j].y, wf.c[j].z, wf.c[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 wv = mx_decode8_bf16(c[i], sc);
        const int64_t k = 32 * static_cast<int64_t>(b0 + j) + 8 * i;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int64_t m = min(m0 + 16 * t + r, a.M - 1);
          Run8<true> xv;
          if (whole || k + 8 <= a.K) xv.load(a.x, m * a.K + k);
          else if (k < a.K) xv.load_part(a.x, m * a.K + k, static_cast<int>(a.K - k));
          else xv.zero();
          acc[t] = mfma_bf16_16x16x32(wv, make_uint4(xv.v[0], xv.v[1], xv.v[2], xv.v[3]), acc[t]);
        }
      }
    }
  }
  join_and_store<MT, BOUT>(a, acc, m0, n0);
}

template <int MT>
dim3 grid_of(const GemvArgs &a) {
  return dim3(static_cast<unsigned>((a.N + 15) / 16), static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT)));
}

template <int MT, int XT>
void run_w4a4(const GemvArgs &a, bool y_bf16, hipStream_t st) {
  if (y_bf16) mx_gemv_w4a4<MT, XT, true><<<grid_of<MT>(a), 64 * kWaves, 0, st>>>(a);
  else mx_gemv_w4a4<MT, XT, false><<<grid_of<MT>(a), 64 * kWaves, 0, st>>>(a);
}

template <int MT>
void run_w4a16(const GemvArgs &a, bool y_bf16, hipStream_t st) {
  if (y_bf16) mx_gemv_w4a16<MT, true><<<grid_of<MT>(a), 64 * kWaves, 0, st>>>(a);
  else mx_gemv_w4a16<MT, false><<<grid_of<MT>(a), 64 * kWaves, 0, st>>>(a);
}

}  // namespace

hipError_t launch_mx_gemv_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                               bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {xq, sx, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32)};
  if (M <= 16) run_w4a4<1, kPacked>(a, y_bf16, st);
  else if (M <= 32) run_w4a4<2, kPacked>(a, y_bf16, st);
  else run_w4a4<4, kPacked>(a, y_bf16, st);
  return hipGetLastError();
}

hipError_t launch_mx_gemv_w4a4_fused(const void *x, bool x_bf16, const uint8_t *wq, const uint8_t *sw, void *y,
                                     bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {x, nullptr, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32)};
  if (x_bf16) run_w4a4<1, kBf16>(a, y_bf16, st);
  else run_w4a4<1, kF32>(a, y_bf16, st);
  return hipGetLastError();
}

hipError_t launch_mx_gemv_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                int64_t M, int64_t N, int64_t K, hipStream_t st) {
  const GemvArgs a = {x, nullptr, wq, sw, y, M, N, K, static_cast<int>((K + 31) / 32)};
  if (M <= 16) run_w4a16<1>(a, y_bf16, st);
  else if (M <= 32) run_w4a16<2>(a, y_bf16, st);
  else run_w4a16<4>(a, y_bf16, st);
  return hipGetLastError();
}

}  // namespace q4

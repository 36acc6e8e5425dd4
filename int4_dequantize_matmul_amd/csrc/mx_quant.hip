// Rows of f32 or bf16 -> MX FP4 blocks, and back.
//
// Per block of 32 columns: top = max |x|, e = max(floor(log2 top) - 2, -127),
// scale byte e + 127, code = x 2^-e rounded to the nearest E2M1 value (ties
// to even, beyond 6 to 6); back: code 2^e.  Every step is exact or rounded
// once, so the codes do not depend on the kernel that forms them.
//
// Bound: memory.  Four lanes hold a block, 8 columns each (one 16-byte load
// of bf16, two of f32), so a wave reads and writes consecutive bytes; the
// block's maximum is two quad moves.  Where K is whole blocks all rows are one
// long run of blocks and no lane is idle; otherwise each row is cut by itself
// and its last, short run is read element by element.
//
// Measured, from memory | input met just before: 8192 x 5632 bf16 to codes 24 to
// 26 us (117 MB, 4.5 to 4.9 TB/s; a copy of 1 GiB runs at 5.2) | 19.7; 2048 x 5632
// 8.7 | 7.0 us there and 6.6 | 6.9 back; 2048 x 1023 f32, rows cut one by one,
// 5.0 | 4.0 and 4.8 | 4.9 us.
#include "kernels.hpp"
#include "mx_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerWg = kThreads / 4;

template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx_quantize(const void *__restrict__ x, int64_t K, int64_t KB,
                                                        int64_t chunks, int64_t total,
                                                        uint8_t *__restrict__ packed, uint8_t *__restrict__ scales) {
  for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int64_t row = chunks == total ? 0 : c / chunks;
    const int64_t b = (c - row * chunks) * kBlocksPerWg + (threadIdx.x >> 2);
    if (b >= KB) continue;   // the four lanes of a block alike
    const int sub = threadIdx.x & 3;
    const int64_t k = 32 * b + 8 * sub;
    Run8<BF16> v;
    if (k + 8 <= K) v.load(x, row * K + k);
    else if (k < K) v.load_part(x, row * K + k, static_cast<int>(K - k));
    else v.zero();
    const uint32_t byte = mx_scale_byte(quad_max(v.top()));
    const uint32_t code = byte == 255 ? 0u : v.encode(mx_scale(byte));
    const int64_t at = row * KB + b;
    reinterpret_cast<uint32_t *>(packed)[4 * at + sub] = code;
    if (sub == 0) scales[at] = static_cast<uint8_t>(byte);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx_dequantize(const uint8_t *__restrict__ packed,
                                                          const uint8_t *__restrict__ scales, int64_t K, int64_t KB,
                                                          int64_t chunks, int64_t total, void *__restrict__ y) {
  for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int64_t row = chunks == total ? 0 : c / chunks;
    const int64_t b = (c - row * chunks) * kBlocksPerWg + (threadIdx.x >> 2);
    if (b >= KB) continue;
    const int sub = threadIdx.x & 3;
    const int64_t k = 32 * b + 8 * sub, at = row * KB + b, o = row * K + k;
    if (k >= K) continue;
    const uint32_t code = reinterpret_cast<const uint32_t *>(packed)[4 * at + sub];
    const float s = mx_scale(scales[at]);
    if constexpr (BF16) {
      const uint4 v = mx_decode8_bf16(code, s);
      uint16_t *p = static_cast<uint16_t *>(y) + o;
      if (k + 8 <= K) {
        store_any(p, v);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (k + j < K) p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
      }
    } else {
      const f32x2 a = mx_decode2_f32<0>(code, s), b2 = mx_decode2_f32<1>(code, s), d = mx_decode2_f32<2>(code, s),
                  e = mx_decode2_f32<3>(code, s);
      const float w[8] = {a[0], a[1], b2[0], b2[1], d[0], d[1], e[0], e[1]};
      float *p = static_cast<float *>(y) + o;
      if (k + 8 <= K) {
        store_any(p, make_float4(w[0], w[1], w[2], w[3]));
        store_any(p + 4, make_float4(w[4], w[5], w[6], w[7]));
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (k + j < K) p[j] = w[j];
      }
    }
  }
}

// Rows of whole blocks are one run of M KB blocks.
struct Split {
  int64_t K, KB, chunks, total;
  unsigned grid;
  Split(int64_t M, int64_t K_) : K(K_), KB((K_ + 31) / 32) {
    if (K % 32 == 0) {
      K *= M;
      KB *= M;
      M = 1;
    }
    chunks = (KB + kBlocksPerWg - 1) / kBlocksPerWg;
    total = M * chunks;
    grid = static_cast<unsigned>(total < (int64_t(1) << 22) ? total : (int64_t(1) << 22));
  }
};

}  // namespace

hipError_t launch_mx_quantize(const void *x, bool x_bf16, int64_t M, int64_t K, uint8_t *packed, uint8_t *scales,
                              hipStream_t st) {
  const Split s(M, K);
  if (x_bf16) mx_quantize<true><<<s.grid, kThreads, 0, st>>>(x, s.K, s.KB, s.chunks, s.total, packed, scales);
  else mx_quantize<false><<<s.grid, kThreads, 0, st>>>(x, s.K, s.KB, s.chunks, s.total, packed, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *packed, const uint8_t *scales, int64_t M, int64_t K, void *y,
                                bool y_bf16, hipStream_t st) {
  const Split s(M, K);
  if (y_bf16) mx_dequantize<true><<<s.grid, kThreads, 0, st>>>(packed, scales, s.K, s.KB, s.chunks, s.total, y);
  else mx_dequantize<false><<<s.grid, kThreads, 0, st>>>(packed, scales, s.K, s.KB, s.chunks, s.total, y);
  return hipGetLastError();
}

}  // namespace q4

// MX FP4 on gfx950: blocks of 32 E2M1 codes (16 bytes, low nibble = even
// column) under one E8M0 scale byte b, which stands for 2^(b - 127); b = 255
// is NaN.  The chip's conversion and matrix instructions take this format as
// it is stored: a conversion's scale operand is read as an exponent field
// (b << 23), 255 included, and a matrix instruction's scale operand is the
// byte.  Both were checked against the format's definition over every code,
// every scale byte and every bf16 input.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "q4_device.hpp"

namespace q4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Loads of any alignment (rows of an odd K start at any element).
template <class T>
__device__ __forceinline__ T load_any(const void *p) {
  T v;
  memcpy(&v, p, sizeof v);
  return v;
}
template <class T>
__device__ __forceinline__ void store_any(void *p, T v) {
  memcpy(p, &v, sizeof v);
}

// The scale operand of a conversion for scale byte b.
__device__ __forceinline__ float mx_scale(uint32_t b) { return __uint_as_float(b << 23); }

// Scale byte of a block whose largest magnitude has the bits top (sign
// clear): floor(log2 top) - 2 + 127, the 2 being E2M1's largest exponent.
// The exponent field of top is floor(log2 top) + 127, so this is that field
// less 2, not below 0 (2^-127, also for zeros and subnormals).  A block with
// a NaN or an infinity gets 255, so it decodes to NaN instead of to a
// plausible number.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}

// The largest of four neighbouring lanes' values, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
}

// Two float32 values -> two codes in byte SEL of d: v / 2^(b - 127), rounded
// to the nearest code, ties to even, beyond 6 to 6.
template <int SEL>
__device__ __forceinline__ uint32_t mx_encode2(uint32_t d, float lo, float hi, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo, hi, scale, SEL);
}
// The same of a pair of bf16 values.
template <int SEL>
__device__ __forceinline__ uint32_t mx_encode2(uint32_t d, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2, pair), scale, SEL);
}

// Byte SEL of d (two codes) -> a pair of bf16 values, exactly.
template <int SEL>
__device__ __forceinline__ uint32_t mx_decode2_bf16(uint32_t d, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, SEL));
}
template <int SEL>
__device__ __forceinline__ f32x2 mx_decode2_f32(uint32_t d, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, SEL);
}

// Eight codes (a dword) -> eight bf16 values.
__device__ __forceinline__ uint4 mx_decode8_bf16(uint32_t d, float scale) {
  return make_uint4(mx_decode2_bf16<0>(d, scale), mx_decode2_bf16<1>(d, scale), mx_decode2_bf16<2>(d, scale),
                    mx_decode2_bf16<3>(d, scale));
}

// A run of 8 activations as it is loaded: four bf16 pairs, or 8 floats.
template <bool BF16>
struct Run8;
template <>
struct Run8<true> {
  uint32_t v[4];
  __device__ __forceinline__ void load(const void *x, int64_t i) {
    const uint4 t = load_any<uint4>(static_cast<const uint16_t *>(x) + i);
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  }
  // the first n (< 8, may be <= 0) elements, zeros after them
  __device__ __forceinline__ void load_part(const void *x, int64_t i, int n) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = 2 * j < n ? p[2 * j] : 0u, hi = 2 * j + 1 < n ? p[2 * j + 1] : 0u;
      v[j] = lo | (hi << 16);
    }
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = v[2] = v[3] = 0; }
  // the largest magnitude's float32 bits (bf16 bits order as their float32)
  __device__ __forceinline__ uint32_t top() const {
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi = max(hi, v[j] & 0x7FFFFFFFu);
      lo = max(lo, v[j] & 0x7FFFu);
    }
    return max(hi & 0xFFFF0000u, lo << 16);
  }
  __device__ __forceinline__ uint32_t encode(float s) const {
    return mx_encode2<3>(mx_encode2<2>(mx_encode2<1>(mx_encode2<0>(0u, v[0], s), v[1], s), v[2], s), v[3], s);
  }
};
template <>
struct Run8<false> {
  float v[8];
  __device__ __forceinline__ void load(const void *x, int64_t i) {
    const float *p = static_cast<const float *>(x) + i;
    const float4 a = load_any<float4>(p), b = load_any<float4>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void load_part(const void *x, int64_t i, int n) {
    const float *p = static_cast<const float *>(x) + i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.0f;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return t;
  }
  __device__ __forceinline__ uint32_t encode(float s) const {
    return mx_encode2<3>(
        mx_encode2<2>(mx_encode2<1>(mx_encode2<0>(0u, v[0], v[1], s), v[2], v[3], s), v[4], v[5], s), v[6], v[7], s);
  }
};

// acc += A B over the 128 columns that a wave's lanes hold: lane (r, g) has
// the 32 columns of block g for row r of A and of B, and the byte J of sa and
// sb is that block's scale.  Result register i of lane (c, q) is the element
// of A's row 4 q + i and B's row c.
template <int J>
__device__ __forceinline__ f32x4 mfma_mx_16x16x128(uint4 a, uint4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w)};
  const i32x8 bv = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, J, static_cast<int>(sa), J,
                                                          static_cast<int>(sb));
}

// The same with 32 rows and 64 columns: lane (r, h) has 32 columns of row r,
// a block; result register 4 a + b of lane (c, h) is the element of A's row
// 8 a + 4 h + b and B's row c.  On this chip it does the work of four of the
// above in the time of two of them.
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <int J>
__device__ __forceinline__ f32x16 mfma_mx_32x32x64(uint4 a, uint4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w)};
  const i32x8 bv = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, J, static_cast<int>(sa), J,
                                                         static_cast<int>(sb));
}

// acc += A B over 16 columns of 32 rows: lane (r, h) has 8 columns of row r;
// results as above.
__device__ __forceinline__ f32x16 mfma_bf16_32x32x16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// float32 -> bf16 pairs, round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// Four results of one row, columns n .. n + 3 of an N-column output.
template <bool BF16>
__device__ __forceinline__ void store_y4(void *y, int64_t m, int64_t n, int64_t N, f32x4 v) {
  if constexpr (BF16) {
    uint16_t *p = static_cast<uint16_t *>(y) + m * N + n;
    const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    if (n + 4 <= N) {
      store_any(p, w);
    } else {
      if (n < N) p[0] = static_cast<uint16_t>(w.x);
      if (n + 1 < N) p[1] = static_cast<uint16_t>(w.x >> 16);
      if (n + 2 < N) p[2] = static_cast<uint16_t>(w.y);
    }
  } else {
    float *p = static_cast<float *>(y) + m * N + n;
    if (n + 4 <= N) {
      store_any(p, v);
    } else {
      if (n < N) p[0] = v[0];
      if (n + 1 < N) p[1] = v[1];
      if (n + 2 < N) p[2] = v[2];
    }
  }
}

}  // namespace q4

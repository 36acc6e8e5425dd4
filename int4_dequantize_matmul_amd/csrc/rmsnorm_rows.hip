// Rows in front of int8 linears in one pass: the residual's addition, the
// root-mean-square norm and the int8 codes of the result with their scale.
//   h = x + r,  u = h g,  y = u / sqrt(mean(h^2) + eps)
//   code = rint(127 y / max|y|) = rint(127 u / max|u|),  scale = max|y| / 127
// The root cancels out of the codes, so they need nothing that is summed: they
// are the nearest ones of the exact quotients (ties to even, up to a sum x + r
// past 53 bits), on every route.  h and products go in f32; an element whose
// f32 quotient, off by at most 6 roundings of 2^-24, lies next to a border is
// divided again in f64, as is the maximum formed.  No square meets more than 20
// roundings of the sum, which goes by runs of 8 columns, lanes and waves (runs of a
// row that is read again are added in f64), so a scale is within 12 steps of 2^-24.
// Where eps does not make up for squares that f32 loses (they end at steps of 2^-149),
// rows that have such are summed once more, times 2^100.
//
// Bound: memory; x and r are read, the sum and the codes written once.  A row
// stays in the registers of one to 16 waves, 8 columns a lane at a time; rows of
// more than 16384 columns are read three times.  8192 rows of 2048 with residual:
// bf16 28 us (4.2 TB/s), f32 35 us (6.2 TB/s, partly from the last-level cache).
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"

namespace q4 {
namespace {

// Below this a sum of squares, with eps for each, may lack what f32 lost: at most 2^30 times 2^-149.
constexpr float kSmall = 0x1p-90f;

template <bool BF16>
__device__ __forceinline__ float at(const Run8<BF16> &r, int j) {
  if constexpr (BF16) return __uint_as_float(j & 1 ? r.v[j / 2] & 0xFFFF0000u : r.v[j / 2] << 16);
  else return r.v[j];
}

// The 8 columns from c on of a row of K, zeros past its end.
template <bool BF16>
__device__ __forceinline__ void fetch(Run8<BF16> &v, const void *p, int64_t row, int64_t c, int64_t K) {
  if (c + 8 <= K) v.load(p, row + c);
  else if (c < K) v.load_part(p, row + c, static_cast<int>(K - c));
  else v.zero();
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int W>
__device__ __forceinline__ void join(float &ss, uint32_t &top, float *sums, uint32_t *tops) {
  // magnitudes order as their bits; NaN and infinity come last
  ss = add_xor32(add_xor16(dpp_row_sum_f32<16>(ss)));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = ss, tops[threadIdx.x >> 6] = top;
    __syncthreads();
    float s[W];
    top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = sums[i], top = max(top, tops[i]);
#pragma unroll
    for (int n = W / 2; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) s[i] += s[i + n];
    ss = s[0];
  }
}

// The largest of the lanes' numbers, most of which are 0.
template <int W>
__device__ __forceinline__ double join(double m, double *tops) {
  unsigned long long left = __ballot(m > 0.0);
  const uint64_t b = __builtin_bit_cast(uint64_t, m);
  m = 0.0;
  while (left) {
    const int l = __builtin_ctzll(left);
    left &= left - 1;
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), l);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), l);
    m = fmax(m, __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo));
  }
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
    __syncthreads();
    m = tops[0];
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmax(m, tops[i]);
  }
  return m;
}

// W waves a row; RUNS times 8 columns a lane in registers, or 0 for rows that
// are read again; SMALL: eps may leave squares that f32 loses to count (a kernel of
// its own, since the second sum takes 8 registers: 8192 rows of 2048 in bf16 29 us, not 28).
template <bool BF16, int W, int RUNS, bool SMALL>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rmsnorm_rows_kernel(NormArgs a, int64_t first) {
  __shared__ float sums[W];
  __shared__ uint32_t tops[W];
  __shared__ double tops64[W];
  const int64_t m = first + (W == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6) : int64_t(blockIdx.x));
  if (m >= a.M) return;   // a whole wave; only where no wave waits for another
  const int64_t K = a.K, row = m * K;
  const int tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  constexpr int step = 64 * W * 8;

  constexpr int N = RUNS ? RUNS : 1;
  Run8<BF16> x[N], r[N];
  float g[N][8];
  auto load = [&](int i, int64_t c) {
    fetch(x[i], a.x, row, c, K);
    if (a.r) fetch(r[i], a.r, row, c, K);
    else r[i].zero();
    if (!a.g) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = 1.0f;
    } else if (a.g_bf16) {
      Run8<true> t;
      fetch(t, a.g, 0, c, K);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = at(t, j);
    } else {
      Run8<false> t;
      fetch(t, a.g, 0, c, K);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = at(t, j);
    }
  };
  // f over the lane's runs, loaded before where they stay in registers
  auto each = [&](auto f) {
    if constexpr (RUNS > 0) {
#pragma unroll
      for (int i = 0; i < RUNS; ++i) f(i, int64_t(i) * step + tid * 8);
    } else {
      for (int64_t c = tid * 8; c < K; c += step) load(0, c), f(0, c);
    }
  };
  auto product = [&](int i, int j) { return (at(x[i], j) + at(r[i], j)) * g[i][j]; };
  auto product64 = [&](int i, int j) {
    return (static_cast<double>(at(x[i], j)) + static_cast<double>(at(r[i], j))) * static_cast<double>(g[i][j]);
  };
  if constexpr (RUNS > 0) {
#pragma unroll
    for (int i = 0; i < RUNS; ++i) load(i, int64_t(i) * step + tid * 8);
  }

  std::conditional_t<RUNS == 0, double, float> lane_ss = 0;
  uint32_t top = 0;
  each([&](int i, int64_t) {
    float run = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float h = at(x[i], j) + at(r[i], j);
      run = fmaf(h, h, run);
      top = max(top, magnitude(h * g[i][j]));
    }
    lane_ss += run;
  });
  float ss = static_cast<float>(lane_ss);
  join<W>(ss, top, sums, tops);
  bool scaled = false;
  if constexpr (SMALL) {
    scaled = fmaf(static_cast<float>(K), a.eps, ss) < kSmall;   // the same in every wave
    if (scaled) {
      if constexpr (W > 1) __syncthreads();   // all have read the sums
      lane_ss = 0;
      each([&](int i, int64_t) {
        float run = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = (at(x[i], j) + at(r[i], j)) * 0x1p100f;
          run = fmaf(h, h, run);
        }
        lane_ss += run;
      });
      ss = static_cast<float>(lane_ss);
      join<W>(ss, top, sums, tops);
    }
    // sums and products are formed again, not kept in registers (an instruction it is not)
    if constexpr (RUNS > 0) {
#pragma unroll
      for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int j = 0; j < (BF16 ? 4 : 8); ++j) asm("" : "+v"(x[i].v[j]));
    }
  }
  const bool bad = top >= 0x7F800000u || !(ss < __builtin_inff());

  // max|u| in f64, from the elements whose f32 product is within its roundings of the largest (of all where that is
  // next to nothing: products below the range of f32 are not 0)
  double m64 = 0.0;
  const uint32_t near_top = top > 8 ? top - 8 : 0;
  each([&](int i, int64_t) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (magnitude(product(i, j)) >= near_top) m64 = fmax(m64, fabs(product64(i, j)));
  });
  m64 = join<W>(m64, tops64);
  if (tid == 0) {
    const double mean = (scaled ? ss * 0x1p-200 : static_cast<double>(ss)) * a.inv_K + static_cast<double>(a.eps);
    const double root = mean < __builtin_inf() ? inverse_root(mean) : 0.0;
    a.sx[m] = bad ? __builtin_nanf("") : m64 == 0.0 ? 0.0f : static_cast<float>(m64 * root * (1.0 / 127.0));
  }

  const float f = __uint_as_float(top);
  const bool small = f < 0x1p-100f;   // subnormal products, or 127 / f past the range
  const float k127 = small ? 0.0f : 127.0f / f;
  each([&](int i, int64_t c) {
    if (c >= K) return;
    const int n = K - c < 8 ? static_cast<int>(K - c) : 8;
    if (a.sum) {
      float h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = at(x[i], j) + at(r[i], j);
      if constexpr (BF16) {
        uint16_t *p = static_cast<uint16_t *>(a.sum) + row + c;
        const uint4 w = make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]),
                                   pack_bf16(h[6], h[7]));
        if (n == 8) {
          store_any(p, w);
        } else {
          const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(d[j / 2] >> (16 * (j & 1)));
        }
      } else {
        float *p = static_cast<float *>(a.sum) + row + c;
        if (n == 8) {
          store_any(p, make_float4(h[0], h[1], h[2], h[3]));
          store_any(p + 4, make_float4(h[4], h[5], h[6], h[7]));
        } else {
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = h[j];
        }
      }
    }
    int code[8];
    bool near = small;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = product(i, j) * k127, q = rintf(t);
      near |= fabsf(t - q) > 0.4998f;
      code[j] = static_cast<int>(q);
    }
    if (bad || m64 == 0.0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) code[j] = 0;
    } else if (near) {
#pragma unroll
      for (int j = 0; j < 8; ++j) code[j] = static_cast<int>(rint(127.0 * product64(i, j) / m64));
    }
    uint32_t d[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j / 4] |= (static_cast<uint32_t>(code[j]) & 0xFFu) << (8 * (j & 3));
    int8_t *p = a.xq + row + c;
    if (n == 8) {
      store_any(p, make_uint2(d[0], d[1]));
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) p[j] = static_cast<int8_t>(d[j / 4] >> (8 * (j & 3)));
    }
  });
}

template <bool BF16, int W, int RUNS, bool SMALL>
void go(const NormArgs &a, hipStream_t st) {
  constexpr int threads = W == 1 ? 256 : 64 * W, rows = W == 1 ? 4 : 1;
  const int64_t most = rows * max_groups(threads);
  for (int64_t first = 0; first < a.M; first += most) {   // rows of a launch
    const int64_t n = a.M - first < most ? a.M - first : most;
    rmsnorm_rows_kernel<BF16, W, RUNS, SMALL><<<static_cast<unsigned>((n + rows - 1) / rows), threads, 0, st>>>(a, first);
  }
}

// As few runs of 8 columns a lane as 1024 lanes allow: each takes about 50 registers,
// so more of them leave too few waves (bf16, 8192 rows of 2048 with residual: four
// waves of one run 28 us, one wave of four 36; 4096 of 5632: four waves of three runs
// 39, of four 52, eight waves of two 43; 2048 of 13312: 16 waves of two 58, four that
// read their rows again 60; one row of 13312 6.5 against 14).
template <bool BF16, bool SMALL>
void pick(const NormArgs &a, hipStream_t st) {
  const int64_t runs = (a.K + 7) / 8;
  if (runs <= 64) go<BF16, 1, 1, SMALL>(a, st);
  else if (runs <= 128) go<BF16, 2, 1, SMALL>(a, st);
  else if (runs <= 256) go<BF16, 4, 1, SMALL>(a, st);
  else if (runs <= 512) go<BF16, 4, 2, SMALL>(a, st);
  else if (runs <= 768) go<BF16, 4, 3, SMALL>(a, st);
  else if (runs <= 1024) go<BF16, 8, 2, SMALL>(a, st);
  else if (runs <= 2048) go<BF16, 16, 2, SMALL>(a, st);
  else go<BF16, 16, 0, SMALL>(a, st);
}

}  // namespace

hipError_t launch_rmsnorm_rows(const NormArgs &a, bool bf16, hipStream_t st) {
  const bool small = static_cast<double>(a.K) * a.eps < 2 * kSmall;
  if (bf16) small ? pick<true, true>(a, st) : pick<true, false>(a, st);
  else small ? pick<false, true>(a, st) : pick<false, false>(a, st);
  return hipGetLastError();
}

}  // namespace q4

// Queries and keys of a decoder layer in one pass: each head's row of D
// numbers is divided by its root mean square, multiplied by a gain, and its
// first R columns are rotated by the token's angles:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos - b sin, b cos + a sin) for the R / 2 pairs (a, b)
// with pair i made of columns i and i + R/2 (halves) or 2 i and 2 i + 1
// (neighbours).  Sums and products in f32, one rounding at the store.
//
// Bound: memory; every number is read and written once.  A head's row stays
// in the registers of a group of L lanes (L a power of two): a lane has the
// columns of whole pairs, so the rotation crosses no lanes, and the square
// sum takes log2 L moves.  In units of V columns (up to 16 bytes, as R and
// D allow it): halves,
// a unit is V columns of the first half with the V opposite ones; neighbours,
// V columns that hold V / 2 pairs; past R a unit is V plain columns.  Rows of
// more than 64 units take turns over them, and read their row a second time
// for the result.
//
// Measured, from memory | input met just before: 8190 tokens of 32 + 8 heads of
// 128 in bf16 41 us (172 MB, 4.2 TB/s) | 32; one token 4.4 | 3.2 us.  Where only 1
// or 2 columns a unit are possible the number of loads bounds it: 4096 tokens of
// 40 heads of 130 88 us (1 TB/s).
#include "kernels.hpp"
#include "mx_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;

// V numbers from element i on, at any address.
template <bool BF16, int V>
__device__ __forceinline__ void load_v(const void *p, int64_t i, float (&o)[V]) {
  if constexpr (BF16) {
    const uint16_t *q = static_cast<const uint16_t *>(p) + i;
    if constexpr (V == 1) {
      o[0] = bf16_to_f32(q[0]);
    } else {
      typedef uint32_t W __attribute__((ext_vector_type(V / 2)));
      const W w = load_any<W>(q);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        o[2 * j] = __uint_as_float(w[j] << 16);
        o[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
    const float *q = static_cast<const float *>(p) + i;
    constexpr int P = V < 4 ? V : 4;   // 16 bytes a load at most
    typedef float W __attribute__((ext_vector_type(P)));
#pragma unroll
    for (int j = 0; j < V; j += P) {
      const W w = load_any<W>(q + j);
#pragma unroll
      for (int l = 0; l < P; ++l) o[j + l] = w[l];
    }
  }
}

template <bool BF16, int V>
__device__ __forceinline__ void store_v(void *p, int64_t i, const float (&o)[V]) {
  if constexpr (BF16) {
    uint16_t *q = static_cast<uint16_t *>(p) + i;
    if constexpr (V == 1) {
      q[0] = static_cast<uint16_t>(pack_bf16(o[0], 0.0f));
    } else {
      typedef uint32_t W __attribute__((ext_vector_type(V / 2)));
      W w;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) w[j] = pack_bf16(o[2 * j], o[2 * j + 1]);
      store_any(q, w);
    }
  } else {
    float *q = static_cast<float *>(p) + i;
    constexpr int P = V < 4 ? V : 4;
    typedef float W __attribute__((ext_vector_type(P)));
#pragma unroll
    for (int j = 0; j < V; j += P) {
      W w;
#pragma unroll
      for (int l = 0; l < P; ++l) w[l] = o[j + l];
      store_any(q + j, w);
    }
  }
}

template <int V>
__device__ __forceinline__ void load_gain(const void *w, bool bf16, int i, float (&o)[V]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 1.0f;
  } else if (bf16) {
    load_v<true, V>(w, i, o);
  } else {
    load_v<false, V>(w, i, o);
  }
}

// Units of a row: PU of rotated columns, then the plain ones.
template <int V, bool NEIGHBOURS>
struct Unit {
  bool rotated;
  int c0, c1;   // first columns of its V (and, in halves, its other V) columns
  int p0;       // its first pair
  __device__ __forceinline__ Unit(int u, int R) {
    const int pu = NEIGHBOURS ? R / V : R / (2 * V);
    rotated = u < pu;
    if (NEIGHBOURS) {
      c0 = u * V;
      c1 = 0;
      p0 = c0 / 2;
    } else {
      p0 = u * V;
      c0 = rotated ? p0 : R + (u - pu) * V;
      c1 = p0 + R / 2;
    }
  }
};

// EARLY: a unit a lane at most, and everything that the row needs under way
// before its square sum (4096 tokens of 40 heads of 256, neighbours: 56 -> 38 us);
// not for two times 8 columns a lane, whose registers would leave too few waves
// (8190 tokens of 40 heads of 128, halves: 39 against 32).
template <bool IB, bool OB, int V, bool NEIGHBOURS, bool EARLY>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(QkArgs a, int L, int units, uint32_t first) {
  const uint32_t id = first + blockIdx.x * static_cast<uint32_t>(kThreads / L) + threadIdx.x / L;
  const int sub = threadIdx.x & (L - 1);
  const uint32_t H = static_cast<uint32_t>(a.Hq + a.Hk);
  const bool live = id < static_cast<uint32_t>(a.T) * H;
  // dead groups go through the moves below with the others
  const uint32_t t = live ? id / H : 0, h = live ? id - t * H : 0;
  const bool key = h >= static_cast<uint32_t>(a.Hq);
  const int64_t hh = key ? h - a.Hq : h;
  const void *x = key ? a.k : a.q;
  const int64_t xi = key ? t * a.k_t + hh * a.k_h : t * a.q_t + hh * a.q_h;
  const void *w = key ? a.wk : a.wq;
  void *y = key ? a.ko : a.qo;
  const int64_t yi = (static_cast<int64_t>(t) * (key ? a.Hk : a.Hq) + hh) * a.D;
  const int D = static_cast<int>(a.D), R = static_cast<int>(a.R);
  bool known;   // an unknown position gives NaN, not a wild read
  const float *cs;
  auto locate = [&] {
    const int64_t pos = a.pos[t];
    known = pos >= 0 && pos < a.P;
    cs = a.table + (known ? pos : 0) * R;
  };

  constexpr int P = NEIGHBOURS ? V / 2 : V;   // pairs of a unit
  float v0[V], v1[V], g0[V], g1[V], c[P], s[P];
  float ss = 0.0f;
  auto fetch = [&](const Unit<V, NEIGHBOURS> &u) {
    load_v<IB, V>(x, xi + u.c0, v0);
    if (!NEIGHBOURS && u.rotated) load_v<IB, V>(x, xi + u.c1, v1);
  };
  auto fetch_rest = [&](const Unit<V, NEIGHBOURS> &u) {
    load_gain<V>(w, a.w_bf16, u.c0, g0);
    if (u.rotated) {
      if constexpr (!NEIGHBOURS) load_gain<V>(w, a.w_bf16, u.c1, g1);
      load_v<false, P>(cs, u.p0, c);
      load_v<false, P>(cs, R / 2 + u.p0, s);
    }
  };
  auto square = [&](const Unit<V, NEIGHBOURS> &u) {
#pragma unroll
    for (int j = 0; j < V; ++j) ss = fmaf(v0[j], v0[j], ss);
    if (!NEIGHBOURS && u.rotated) {
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v1[j], v1[j], ss);
    }
  };
  auto finish = [&](const Unit<V, NEIGHBOURS> &u, float rms) {
#pragma unroll
    for (int j = 0; j < V; ++j) v0[j] = v0[j] * rms * g0[j];
    if (u.rotated) {
      if (!known) {
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = __builtin_nanf("");
      }
      if constexpr (NEIGHBOURS) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float p = v0[2 * j], q = v0[2 * j + 1];
          v0[2 * j] = p * c[j] - q * s[j];
          v0[2 * j + 1] = q * c[j] + p * s[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float p = v0[j], q = v1[j] * rms * g1[j];
          v0[j] = p * c[j] - q * s[j];
          v1[j] = q * c[j] + p * s[j];
        }
        store_v<OB, V>(y, yi + u.c1, v1);
      }
    }
    store_v<OB, V>(y, yi + u.c0, v0);
  };

  if constexpr (EARLY) {
    if (live && sub < units) {
      const Unit<V, NEIGHBOURS> u(sub, R);
      locate();
      fetch(u);
      fetch_rest(u);
      square(u);
    }
  } else if (live) {
    for (int i = sub; i < units; i += L) {
      const Unit<V, NEIGHBOURS> u(i, R);
      fetch(u);
      square(u);
    }
  }
  for (int d = 1; d < L; d <<= 1) ss += __shfl_xor(ss, d);
  if (!live) return;
  const float rms = 1.0f / sqrtf(ss / static_cast<float>(D) + a.eps);
  if constexpr (EARLY) {
    if (sub < units) finish(Unit<V, NEIGHBOURS>(sub, R), rms);
  } else {
    locate();
    for (int i = sub; i < units; i += L) {
      const Unit<V, NEIGHBOURS> u(i, R);
      if (units > L) fetch(u);   // otherwise still in registers
      fetch_rest(u);
      finish(u, rms);
    }
  }
}

template <bool IB, bool OB, int V, bool NB>
void go(const QkArgs &a, hipStream_t st) {
  const int64_t units = NB ? a.D / V : a.R / (2 * V) + (a.D - a.R) / V;
  int L = 1;
  while (L < units && L < 64) L *= 2;
  const auto kernel = (NB || V < 8) && units <= L ? qk_norm_rope_kernel<IB, OB, V, NB, NB || V < 8>
                                                  : qk_norm_rope_kernel<IB, OB, V, NB, false>;
  const int64_t rows = a.T * (a.Hq + a.Hk), per = kThreads / L, most = per * max_groups(kThreads);
  for (int64_t first = 0; first < rows; first += most) {   // rows of heads of a launch
    const int64_t n = rows - first < most ? rows - first : most;
    kernel<<<static_cast<unsigned>((n + per - 1) / per), kThreads, 0, st>>>(a, L, static_cast<int>(units),
                                                                            static_cast<uint32_t>(first));
  }
}

template <bool IB, bool OB, bool NB>
void pick(const QkArgs &a, hipStream_t st) {
  // as many columns a unit, up to 16 bytes of the wider type, as divide the
  // halves (or the pairs' columns) and the rest; rows may start anywhere
  constexpr int most = IB && OB ? 8 : 4;
  const int64_t n = (NB ? a.R : a.R / 2) | (a.D - a.R);
  if (most == 8 && n % 8 == 0) go<IB, OB, most, NB>(a, st);
  else if (n % 4 == 0) go<IB, OB, 4, NB>(a, st);
  else if (NB || n % 2 == 0) go<IB, OB, 2, NB>(a, st);   // R and D are even
  else go<IB, OB, NB ? 2 : 1, NB>(a, st);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs &a, bool in_bf16, bool out_bf16, bool neighbours, hipStream_t st) {
  if (in_bf16 && out_bf16) neighbours ? pick<true, true, true>(a, st) : pick<true, true, false>(a, st);
  else if (in_bf16) neighbours ? pick<true, false, true>(a, st) : pick<true, false, false>(a, st);
  else if (out_bf16) neighbours ? pick<false, true, true>(a, st) : pick<false, true, false>(a, st);
  else neighbours ? pick<false, false, true>(a, st) : pick<false, false, false>(a, st);
  return hipGetLastError();
}

}  // namespace q4

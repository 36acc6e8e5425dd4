// Keys and values into the paged 8-bit cache, and out of it again.
//
// Append: a row of a key head is normalised (if asked for) and its first R
// columns are rotated by its position's angles, as in qk_norm_rope.hip; then
// the rows of a block of 16 tokens share the scale 2^e, the smallest power of
// two with max|x| <= 127 2^e, and a code is x / 2^e rounded to the nearest, ties
// to even.  Where the block has tokens already, e only grows, and their codes
// are rounded again, c -> rint(c 2^(old - new)): as steps at least double, what
// such roundings add up to stays below one step of the last scale.  Key rows are
// computed in f64, so that a code and the scale depend on no sum's order;
// scaling by a power of two is exact.  Query rows, rounded to 24 or 8 bits, go
// in f32.
//
// Bound: memory.  A block has one owner, a workgroup of 16 tokens by 16 lanes
// (8 columns a lane, twice past 128), so nothing is shared between workgroups
// and a block's scale is written by who writes its codes; keys and values are
// two workgroups.  Values are turned in LDS to their layout, 16 tokens a column.
#include "kv_device.hpp"

namespace q4 {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&o)[8]) {
  Run8<BF16> t;
  t.load(p, i);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BF16) o[j] = __uint_as_float(j & 1 ? t.v[j / 2] & 0xFFFF0000u : t.v[j / 2] << 16);
    else o[j] = t.v[j];
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, const float (&o)[8]) {
  if constexpr (BF16)
    store_any(static_cast<uint16_t *>(p) + i, make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                         pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])));
  else {
    float *q = static_cast<float *>(p) + i;
    store_any(q, make_float4(o[0], o[1], o[2], o[3]));
    store_any(q + 4, make_float4(o[4], o[5], o[6], o[7]));
  }
}

// Orders this wave's LDS writes before its later LDS reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One head's row by 16 lanes: lane j has the columns 8 j .. and 8 (j + 16) ...
// Norm and rotation; turn: D numbers of LDS of the row's own.  All lanes of the
// wave come here; rows that are not live read nothing.
template <class real, bool BF16>
__device__ __forceinline__ void head_row(const AppendArgs &a, const void *x, int64_t xi, const void *gain, int64_t pos,
                                         bool live, real (&y)[2][8], real *turn) {
  const int lane = threadIdx.x & 15, D = static_cast<int>(a.pool.D), R = static_cast<int>(a.R);
  real ss = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = 8 * (lane + 16 * u);
    float t[8] = {};
    if (live && c < D) load8<BF16>(x, xi + c, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[u][j] = t[j];
      ss += y[u][j] * y[u][j];
    }
  }
  if (a.norm) {
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) ss += __shfl_xor(ss, d);
    const real rms = 1 / sqrt(ss / D + static_cast<real>(a.eps));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      if (c >= D) break;
      float g[8];
      if (!gain) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 1.0f;
      } else if (a.g_bf16) {
        load8<true>(gain, c, g);
      } else {
        load8<false>(gain, c, g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[u][j] = y[u][j] * rms * static_cast<real>(g[j]);
    }
  }
  if (!a.table) return;
  const bool known = pos >= 0 && pos < a.P;   // an unknown position gives NaN, not a wild read
  const float *cs = a.table + (known ? pos : 0) * R, *sn = cs + R / 2;
  if (a.neighbours) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if (c + j >= R) break;
        const real co = known ? cs[(c + j) / 2] : __builtin_nanf(""), si = sn[(c + j) / 2];
        const real p = y[u][j], q = y[u][j + 1];
        y[u][j] = p * co - q * si;
        y[u][j + 1] = q * co + p * si;
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      if (c < D) {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn[c + j] = y[u][j];
      }
    }
    wave_sync();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = 8 * (lane + 16 * u) + j;
        if (c >= R) break;
        const bool low = c < R / 2;
        const int p = low ? c : c - R / 2;
        const real co = known ? cs[p] : __builtin_nanf(""), si = sn[p];
        const real other = turn[low ? c + R / 2 : p];
        y[u][j] = low ? y[u][j] * co - other * si : y[u][j] * co + other * si;
      }
    }
  }
}

// The scale byte of a block whose largest magnitude is t, finite: the smallest
// e + 127 >= 0 with t <= 127 2^e.  127 is 1.984375 2^6.
__device__ __forceinline__ int scale_byte(double t) {
  const uint64_t b = __builtin_bit_cast(uint64_t, t);
  const int e = static_cast<int>(b >> 52) - 1023 - 6;
  const bool over = (b & 0xFFFFFFFFFFFFFull) > 0xFC00000000000ull;   // 0.984375 of a mantissa
  const int b8 = max(e + (over ? 1 : 0) + 127, 0);
  return min(b8, 255);
}

// Four codes -> the same at a scale 2^shift times as large.
__device__ __forceinline__ uint32_t coarser(uint32_t w, int shift) {
  const float f = ldexpf(1.0f, -min(shift, 126));
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = static_cast<int8_t>(w >> (8 * j));
    o |= (static_cast<uint32_t>(static_cast<int>(rintf(static_cast<float>(c) * f))) & 0xFFu) << (8 * j);
  }
  return o;
}

// Workgroups of a launch: slots x heads x {keys, values}, then 16 query rows each.
template <bool BF16, bool OB>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a, uint32_t blocks, uint32_t first) {
  extern __shared__ double lds[];
  __shared__ double tops[kThreads / 64];
  const uint32_t id = first + blockIdx.x;
  const int lane = threadIdx.x & 15, slot16 = threadIdx.x >> 4;
  const int D = static_cast<int>(a.pool.D);

  if (id >= blocks) {   // queries
    const uint32_t r = (id - blocks) * 16 + slot16, Hq = static_cast<uint32_t>(a.Hq);
    const int64_t t = r / Hq, h = r % Hq;
    const bool in = t < a.seqs.T;
    const Sequence s = find_sequence<16>(a.seqs, in ? static_cast<uint32_t>(t) : 0, [&](uint32_t start, int) { return start; });
    const bool live = in && s.i >= 0 && t - s.row < s.n;   // not behind the last sequence
    const int64_t pos = live ? s.first + (t - s.row) : -1;
    float y[2][8];
    head_row<float, BF16>(a, a.q, t * a.q_t + h * a.q_h, a.gq, pos, live, y, reinterpret_cast<float *>(lds) + slot16 * D);
    if (!live) return;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      if (c < D) store8<OB>(a.qo, (t * a.Hq + h) * D + c, y[u]);
    }
    return;
  }

  const bool values = id & 1;
  const uint32_t Hk = static_cast<uint32_t>(a.pool.Hk), h = (id >> 1) % Hk;
  const BlockOf w(a.seqs, (id >> 1) / Hk);
  const Sequence &s = w.s;
  if (s.i < 0) return;
  const int64_t at = block_at(a.pool, s.i, w.b, h);
  if (at < 0) return;                    // no such page: the tokens are dropped
  const int begin = w.b * kKvBlock, had = max(max(s.first, 0) - begin, 0), have = min(s.len - begin, kKvBlock);
  int8_t *codes = (values ? a.pool.v : a.pool.k) + at * kKvBlock * D;
  uint8_t *scale = (values ? a.pool.vs : a.pool.ks) + at;

  const bool live = slot16 >= had && slot16 < have;
  const int64_t row = static_cast<int64_t>(s.row) + begin + slot16 - s.first;
  double y[2][8];
  if (values) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      float t[8] = {};
      if (live && c < D) load8<BF16>(a.v, row * a.v_t + h * a.v_h + c, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[u][j] = t[j];
    }
  } else {
    head_row<double, BF16>(a, a.k, row * a.k_t + h * a.k_h, a.gk, begin + slot16, live, y, lds + slot16 * D);
  }

  const int old = had ? *scale : 0;       // before the barrier: the first thread writes it behind that
  double top = 0.0;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double v = live ? fabs(y[u][j]) : 0.0;
      top = v <= top ? top : v;          // NaN goes on as NaN: it is not <= anything ...
      if (!(v < __builtin_inf())) top = __builtin_inf();   // ... and counts as infinity
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmax(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) top = fmax(top, tops[i]);
  const int need = top < __builtin_inf() ? scale_byte(top) : 255;
  const int byte = had ? max(old, need) : need;
  const int shift = byte == 255 ? 0 : byte - old;   // of the codes that the block has

  // codes of this lane's columns, 8 bytes a run
  uint2 c8[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t d[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = byte == 255 ? 0 : static_cast<int>(rint(ldexp(y[u][j], 127 - byte)));
      d[j / 4] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (j & 3));
    }
    c8[u] = make_uint2(d[0], d[1]);
  }
  if (!values) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      if (c >= D) break;
      uint2 *p = reinterpret_cast<uint2 *>(codes + (c / 16) * 256 + slot16 * 16 + (c & 8));
      if (live) *p = c8[u];
      else if (slot16 < had && shift > 0) {
        const uint2 t = *p;
        *p = make_uint2(coarser(t.x, shift), coarser(t.y, shift));
      }
    }
  } else {
    // columns side by side per token -> tokens side by side per column
    uint8_t *turn = reinterpret_cast<uint8_t *>(lds);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 8 * (lane + 16 * u);
      if (c >= D) break;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        turn[(c + j) * 16 + slot16] = static_cast<uint8_t>((j < 4 ? c8[u].x : c8[u].y) >> (8 * (j & 3)));
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c < D) {
      uint4 v = *reinterpret_cast<const uint4 *>(turn + c * 16);
      uint4 *p = reinterpret_cast<uint4 *>(codes + c * 16);
      if (had) {
        const uint4 t = *p;
        const uint32_t o[4] = {t.x, t.y, t.z, t.w};
        uint32_t n[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = had - 4 * j;     // bytes of this word that the block has
          const uint32_t mask = k <= 0 ? 0u : k >= 4 ? ~0u : (1u << (8 * k)) - 1;
          n[j] = (n[j] & ~mask) | ((shift > 0 ? coarser(o[j], shift) : o[j]) & mask);
        }
        v = make_uint4(n[0], n[1], n[2], n[3]);
      }
      *p = v;
    }
  }
  if (threadIdx.x == 0) *scale = static_cast<uint8_t>(byte);
}

// A block of one head, keys or values, as bf16 or f32 rows.
template <bool OB>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvPool pool, KvSeqs seqs, void *ko, void *vo, uint32_t first) {
  __shared__ uint8_t turn[256 * 16];
  const uint32_t id = first + blockIdx.x;
  const bool values = id & 1;
  const uint32_t Hk = static_cast<uint32_t>(pool.Hk), h = (id >> 1) % Hk;
  const BlockOf w(seqs, (id >> 1) / Hk);
  const Sequence &s = w.s;
  if (s.i < 0) return;
  const int lane = threadIdx.x & 15, slot16 = threadIdx.x >> 4, D = static_cast<int>(pool.D);
  const int64_t at = block_at(pool, s.i, w.b, h), pos = static_cast<int64_t>(w.b) * kKvBlock + slot16;
  const bool known = at >= 0;            // no such page: NaN
  const int8_t *codes = (values ? pool.v : pool.k) + (known ? at : 0) * kKvBlock * D;
  const int byte = known ? (values ? pool.vs : pool.ks)[at] : 255;
  const bool live = pos >= s.first && pos < s.len;
  const int64_t row = s.row + (pos - s.first);
  if (values) {
    const int c = threadIdx.x;
    if (c < D && known) *reinterpret_cast<uint4 *>(turn + c * 16) = load16(codes + c * 16);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = 8 * (lane + 16 * u);
    if (c >= D || !live) break;
    float y[8];
    uint2 t = make_uint2(0, 0);
    if (!values && known) t = *reinterpret_cast<const uint2 *>(codes + (c / 16) * 256 + slot16 * 16 + (c & 8));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int8_t q = values ? static_cast<int8_t>(turn[(c + j) * 16 + slot16])
                              : static_cast<int8_t>((j < 4 ? t.x : t.y) >> (8 * (j & 3)));
      y[j] = byte == 255 ? __builtin_nanf("") : ldexpf(static_cast<float>(q), byte - 127);
    }
    store8<OB>(values ? vo : ko, (row * pool.Hk + h) * D + c, y);
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, bool bf16, bool out_bf16, hipStream_t st) {
  const int64_t blocks = block_slots(a.seqs.T, a.seqs.N) * a.pool.Hk * 2;
  const int64_t all = blocks + (a.q ? (a.seqs.T * a.Hq + 15) / 16 : 0), most = max_groups(kThreads);
  const size_t lds = 16 * a.pool.D * sizeof(double);
  const auto kernel = bf16 ? (out_bf16 ? kv_append_kernel<true, true> : kv_append_kernel<true, false>)
                           : (out_bf16 ? kv_append_kernel<false, true> : kv_append_kernel<false, false>);
  for (int64_t first = 0; first < all; first += most)
    kernel<<<static_cast<unsigned>(all - first < most ? all - first : most), kThreads, lds, st>>>(
        a, static_cast<uint32_t>(blocks), static_cast<uint32_t>(first));
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvPool &pool, const KvSeqs &seqs, void *ko, void *vo, bool out_bf16, hipStream_t st) {
  const int64_t all = block_slots(seqs.T, seqs.N) * pool.Hk * 2, most = max_groups(kThreads);
  const auto kernel = out_bf16 ? kv_read_kernel<true> : kv_read_kernel<false>;
  for (int64_t first = 0; first < all; first += most)
    kernel<<<static_cast<unsigned>(all - first < most ? all - first : most), kThreads, 0, st>>>(
        pool, seqs, ko, vo, static_cast<uint32_t>(first));
  return hipGetLastError();
}

}  // namespace q4

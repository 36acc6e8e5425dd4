// Internal launchers of libq4's kernels.  Callers (q4_api.hip) have already
// validated every argument; the launchers only choose grid shapes and
// enqueue on the given stream.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

// Is the current device gfx950?  (Cached per device; the API checks it
// before every launch.)
bool device_is_gfx950();

// Workgroups of `threads` threads that one launch can have along x: a grid axis
// holds fewer than 2^32 threads.  The runtime does not refuse more, it starts
// their number modulo 2^32 and reports success.
constexpr int64_t max_groups(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

// Weight rows that one launch of a streaming or matrix-core decode kernel can
// have: 16 to 256 threads (4 to 64).  The general kernels serve more.
constexpr int64_t kDecodeMaxN = 16 * max_groups(256);

// Stored-nibble encodings, as in q4_enc.
enum Enc : int { kTwos = 0, kExcess8 = 1 };

// y[0..n) = 0 for float outputs, written by a kernel (no memset node, so a
// captured graph replays it like any other kernel).
hipError_t launch_zero(void *p, size_t bytes, hipStream_t st);

// Activation rows -> int8 codes + f32 scales (canonical Q8 recipe).
hipError_t launch_quantize_rows(const void *x, bool x_bf16, int64_t M, int64_t K, int8_t *xq,
                                float *sx, hipStream_t st);

// General kernels: any shape the API accepts, byte-granular loads.
// Float activations (W4A32: f32 x, f16 scales; W4A16: bf16 x, bf16 scales).
// zp (optional, W4A16 and grouped W4A8): uint8 zero points [N, K/G]; then
// a weight is s * (u - z) with u the stored nibble, and enc is not used.
hipError_t launch_generic_float(const void *x, bool x_bf16, const uint8_t *wq, const uint16_t *s,
                                bool s_bf16, float *yf, uint16_t *yb, int64_t M, int64_t N,
                                int64_t K, int64_t G, int enc, hipStream_t st,
                                const uint8_t *zp = nullptr);
// Integer activations (W4A8 per channel / grouped, W8A8).
hipError_t launch_generic_int(const int8_t *xq, const float *sx, const void *w, bool w_int8,
                              const float *sw, float *y, int64_t M, int64_t N, int64_t K,
                              int64_t G, int enc, hipStream_t st, const uint8_t *zp = nullptr);

// int8 weights, one f32 scale per row, f32 or bf16 activations (W8A32 /
// W8A16): y = s[n] * sum_k x q; yf and / or yb (bf16 RNE) written.
hipError_t launch_generic_w8_float(const void *x, bool x_bf16, const int8_t *wq, const float *s, float *yf,
                                   uint16_t *yb, int64_t M, int64_t N, int64_t K, hipStream_t st);
bool gemv_stream_w8_ok(const void *x, const void *wq, int64_t M, int64_t K);
hipError_t launch_gemv_stream_w8(const void *x, bool x_bf16, const int8_t *wq, const float *s, float *yf,
                                 uint16_t *yb, int64_t M, int64_t N, int64_t K, hipStream_t st);

// W4A32 on the vector ALUs: f32 x, f16 group scales, G a multiple of 32,
// 16-byte aligned x and wq; every M (workgroups of 1 or 2 activation rows).
bool gemv_stream_w4a32_ok(const void *x, const void *wq, int64_t M, int64_t K, int64_t G);
hipError_t launch_gemv_stream_w4a32(const float *x, const uint8_t *wq, const uint16_t *s, float *y, int64_t M,
                                    int64_t N, int64_t K, int64_t G, int enc, hipStream_t st);

// Decode GEMV on MFMA (M in blocks of 16).  *_ok says whether the fast
// kernel serves a shape / alignment; the launcher must only be called then.
bool gemv_w4a16_ok(const void *x, const void *wq, int64_t K, int64_t G, int64_t N = 16);
hipError_t launch_gemv_w4a16(const uint16_t *x, const uint8_t *wq, const uint16_t *s, float *yf,
                             uint16_t *yb, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                             hipStream_t st, const uint8_t *zp = nullptr);
// Decode GEMV for W4A16 on the matrix cores (M <= 16, G a multiple of 128).
bool gemv_mc_w4a16_ok(const void *x, const void *wq, int64_t M, int64_t K, int64_t G);
hipError_t launch_gemv_mc_w4a16(const uint16_t *x, const uint8_t *wq, const uint16_t *s, float *yf,
                                uint16_t *yb, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                                hipStream_t st);
// Decode GEMV for W4A16 on the vector ALUs (M <= 16, K and G multiples of 32).
bool gemv_stream_w4a16_ok(const void *x, const void *wq, int64_t M, int64_t K, int64_t G);
hipError_t launch_gemv_stream_w4a16(const uint16_t *x, const uint8_t *wq, const uint16_t *s, float *yf,
                                    uint16_t *yb, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                                    hipStream_t st, const uint8_t *zp = nullptr);
// Decode GEMV for per-channel W4A8 on the vector ALUs (M <= 16, ceil(K/2) a
// multiple of 16).  xt: 0 = int8 codes with scales sx, 1 = f32 x, 2 = bf16 x
// (quantized inside with the Q8 recipe; sx unused).
bool gemv_chan_w4a8_ok(const void *wq, int64_t M, int64_t K);
hipError_t launch_gemv_chan_w4a8(const void *x, int xt, const float *sx, const uint8_t *wq,
                                 const float *sw, float *y, int64_t M, int64_t N, int64_t K, int enc,
                                 hipStream_t st);
// The same kernel over several independent problems in one launch (float
// x quantized inside, excess-8 weights, one M <= 16 for all).  The caller
// lists only problems with N > 0 and K > 0 that gemv_chan_w4a8_ok accepts,
// at most gemv_chan_w4a8_multi_max() of them, whose tiles of 16 weight rows
// (gemv_chan_w4a8_multi_tiles(N) each) sum to at most 2^24 - 1.
struct ChanProblem {
  const void *x;
  const uint8_t *wq;
  const float *sw;
  float *y;
  int64_t N, K;
};
int64_t gemv_chan_w4a8_multi_max();
int64_t gemv_chan_w4a8_multi_tiles(int64_t N);
hipError_t launch_gemv_chan_w4a8_multi(const ChanProblem *pr, int count, int64_t M, bool x_bf16,
                                       hipStream_t st);
bool gemv_w4a8_ok(const void *wq, int64_t K, int64_t G, int64_t N = 16);
hipError_t launch_gemv_w4a8(const int8_t *xq, const float *sx, const uint8_t *wq, const float *sw,
                            float *y, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                            hipStream_t st, const uint8_t *zp = nullptr);
// Dynamic W4A8 in one launch: f32 or bf16 activation rows quantized inside
// the MFMA GEMV (a small activation matrix).
bool gemv_w4a8_fused_ok(const void *wq, int64_t M, int64_t K, int64_t G, bool x_bf16);
hipError_t launch_gemv_w4a8_fused(const void *x, bool x_bf16, const uint8_t *wq, const float *sw, float *y,
                                  int64_t M, int64_t N, int64_t K, int64_t G, int enc, hipStream_t st,
                                  const uint8_t *zp = nullptr);
bool gemv_w8a8_ok(const void *wq, int64_t K, int64_t N = 16);
hipError_t launch_gemv_w8a8(const int8_t *xq, const float *sx, const int8_t *wq, const float *sw,
                            float *y, int64_t M, int64_t N, int64_t K, hipStream_t st);

// Prefill: LDS-tiled MFMA GEMM (M >= 17).
int device_cu_count();   // compute units of the current device, 0 if unknown
void tiled_w4a8_pieces(int64_t M, int64_t N, int cus, int *full, int *split, int64_t *tiles);
void tiled_w4a16_pieces(int64_t M, int64_t N, int cus, int *full, int64_t *pieces);
bool tiled_w4a8_ok(const void *xq, const void *wq, int64_t M, int64_t N, int64_t K, int64_t G);
hipError_t launch_tiled_w4a8(const int8_t *xq, const float *sx, const uint8_t *wq, const float *sw,
                             float *y, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                             hipStream_t st, const uint8_t *zp = nullptr);
bool tiled_w4a16_ok(const void *x, const void *wq, int64_t M, int64_t N, int64_t K, int64_t G);
hipError_t launch_tiled_w4a16(const uint16_t *x, const uint8_t *wq, const uint16_t *s, float *yf,
                              uint16_t *yb, int64_t M, int64_t N, int64_t K, int64_t G, int enc,
                              hipStream_t st, const uint8_t *zp = nullptr);

// MX FP4 (blocks of 32 E2M1 codes under one E8M0 byte).  packed and wq, xq
// are 16-byte aligned, rows of 16 ceil(K/32) bytes; scales rows of ceil(K/32).
hipError_t launch_mx_quantize(const void *x, bool x_bf16, int64_t M, int64_t K, uint8_t *packed, uint8_t *scales,
                              hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t *packed, const uint8_t *scales, int64_t M, int64_t K, void *y,
                                bool y_bf16, hipStream_t st);
// Products by blocks of 16 weight rows; any M up to 16 * 65535, K > 0.  The
// fused form quantizes f32 or bf16 rows itself.
hipError_t launch_mx_gemv_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                               bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st);
hipError_t launch_mx_gemv_w4a4_fused(const void *x, bool x_bf16, const uint8_t *wq, const uint8_t *sw, void *y,
                                     bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st);
hipError_t launch_mx_gemv_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                int64_t M, int64_t N, int64_t K, hipStream_t st);
// LDS-tiled products, any shape that mx_tiled_*_ok takes.
bool mx_tiled_w4a4_ok(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_tiled_w4a4(const uint8_t *xq, const uint8_t *sx, const uint8_t *wq, const uint8_t *sw, void *y,
                                bool y_bf16, int64_t M, int64_t N, int64_t K, hipStream_t st);
bool mx_tiled_w4a16_ok(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_tiled_w4a16(const uint16_t *x, const uint8_t *wq, const uint8_t *sw, void *y, bool y_bf16,
                                 int64_t M, int64_t N, int64_t K, hipStream_t st);

// Norm of each query and key head with the rotation of its first R columns.
// Strides in elements; wq, wk (gains) and the keys may be null (then Hk == 0).
struct QkArgs {
  const void *q, *k;
  int64_t q_t, q_h, k_t, k_h;   // strides of a token and of a head
  const void *wq, *wk;
  bool w_bf16;
  const int64_t *pos;           // [T]
  const float *table;           // [P, R]: R/2 cosines, then R/2 sines
  void *qo, *ko;                // [T, Hq, D], [T, Hk, D]
  int64_t T, Hq, Hk, D, R, P;
  float eps;
};
hipError_t launch_qk_norm_rope(const QkArgs &a, bool in_bf16, bool out_bf16, bool neighbours, hipStream_t st);

// Rows x + r, normalised and quantised to int8 with an f32 scale a row.  r, g and
// sum may be null; x, r and sum have one type.
struct NormArgs {
  const void *x, *r, *g;
  bool g_bf16;
  void *sum;
  int8_t *xq;
  float *sx;
  int64_t M, K;
  double inv_K;
  float eps;
};
hipError_t launch_rmsnorm_rows(const NormArgs &a, bool bf16, hipStream_t st);

// The paged 8-bit cache (layout: kv_device.hpp) and the rows of a call: row
// starts[i] + t of sequence i is its token lengths[i] - (starts[i + 1] -
// starts[i]) + t.
struct KvPool {
  int8_t *k, *v;
  uint8_t *ks, *vs;
  const int32_t *pages;         // [N, width]
  int64_t n_pages, width, Hk, D;
  int page_blocks_log2;         // blocks of 16 tokens a page
};
struct KvSeqs {
  const int32_t *starts;        // [N + 1]
  const int32_t *lengths;       // [N]
  int64_t N, T;                 // sequences, rows that the row arrays have
};
// Keys and values into the cache, keys (and queries into qo) normalised and
// rotated on the way.  Strides in elements; q, gains and the table may be null.
struct AppendArgs {
  KvPool pool;
  KvSeqs seqs;
  const void *q, *k, *v;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h;
  const void *gq, *gk;
  bool g_bf16;
  const float *table;           // [P, R], or null: no rotation
  int64_t P, R;
  bool neighbours, norm;
  float eps;
  void *qo;                     // [T, Hq, D]
  int64_t Hq;
};
hipError_t launch_kv_append(const AppendArgs &a, bool bf16, bool out_bf16, hipStream_t st);
// ko, vo: [T, Hk, D]
hipError_t launch_kv_read(const KvPool &pool, const KvSeqs &seqs, void *ko, void *vo, bool out_bf16, hipStream_t st);

// Attention of the rows of a call over the cache.  q strided, y [T, Hq, D].
struct AttnArgs {
  KvPool pool;
  KvSeqs seqs;
  const void *q;
  int64_t q_t, q_h;
  void *y;
  int64_t Hq, G;                // query heads, and of a key head
  float scale;
  int64_t window, sinks;        // window 0: none
};
// The routes that attention_plan knows (values of q4_path); any other means few rows.
constexpr int kPathAuto = 0, kPathTiled = 3;
// How a call is shared out; from sizes alone, so that the workspace is known
// before.  two: queries or results in f32.
struct AttnPlan {
  bool tiled;      // LDS-tiled kernel for many rows a sequence, else waves that share out the keys
  int splits;      // workgroups that share out a sequence's keys
  size_t ws;       // bytes of workspace
};
AttnPlan attention_plan(int64_t T, int64_t N, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len, int64_t window,
                        int64_t sinks, bool two, int path);
hipError_t launch_attention(const AttnArgs &a, const AttnPlan &p, bool bf16, bool out_bf16, void *ws, hipStream_t st);

}  // namespace q4

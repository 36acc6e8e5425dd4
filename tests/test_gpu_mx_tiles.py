"""Every tile of the many-row MX FP4 products against the float64 oracle, in
both result types, on shapes that tests/test_mx_tile_shapes.py shows to reach
it.

A product of n terms in f32 is off by at most n + 8 roundings (half a step,
2^-24, each) of the sum of the terms' magnitudes, and never by more than the
1e-5 of that sum which the library's float products keep; a bf16 result by half
a bf16 step (2^-8) of itself more.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.mx as X
from tests import mx_tile_shapes as S
from tests.gpu_util import DEV, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _tiles():
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
    q4.q4_set_path("tiled")
    yield
    q4.q4_set_path("auto")


def codes(rng, rows, K, lo, hi):
    """Random codes (0 past column K) and scale bytes lo .. hi."""
    B = X.blocks(K)
    c = rng.integers(0, 256, (rows, 16 * B), dtype=np.uint8)
    c[:, (K + 1) // 2:] = 0
    if K % 2:
        c[:, K // 2] &= 15
    return c, rng.integers(lo, hi + 1, (rows, B), dtype=np.uint8)


def check(y, ref, mag, K, what):
    got = host(y)
    bf16 = y.dtype == torch.bfloat16
    got = (F.bf16_bits_to_f32(got) if bf16 else got).astype(np.float64)
    tol = min(1e-5, (K + 8) * 2.0 ** -24) * mag + 1e-44
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


def product(x, w):
    """x W^T and |x| |W|^T in float64 (on the GPU: a library product of plain matrices)."""
    x, w = (torch.from_numpy(a).to(DEV) for a in (x, w))
    return tuple(torch.matmul(a, b.t().contiguous()).cpu().numpy() for a, b in ((x, w), (x.abs(), w.abs())))


@pytest.mark.parametrize("tile,M,N,K", list(S.cases_w4a4()))
def test_w4a4_tiles(tile, M, N, K):
    rng = np.random.default_rng(M + N + K)
    xq, sx = codes(rng, M, K, 120, 130)
    wq, sw = codes(rng, N, K, 110, 122)
    ref, mag = product(X.dequantize_rows(xq, sx, K), X.dequantize_rows(wq, sw, K))
    args = [dev(a) for a in (xq, sx, wq, sw)]
    for yt in ("f32", "bf16"):
        check(q4.q4_linear_w4a4_mx(*args, yt), ref, mag, K, (tile, yt))
        assert q4.q4_last_path() == "tiled"


@pytest.mark.parametrize("tile,M,N,K", list(S.cases_w4a16()))
def test_w4a16_tiles(tile, M, N, K):
    rng = np.random.default_rng(M + N + K)
    x = F.f32_to_bf16_bits((rng.standard_normal((M, K)) * np.exp2(rng.integers(-4, 5, K))).astype(np.float32))
    wq, sw = codes(rng, N, K, 110, 122)
    ref, mag = product(F.bf16_bits_to_f32(x).astype(np.float64), X.dequantize_rows(wq, sw, K))
    args = [dev(a) for a in (x, wq, sw)]
    for yt in ("f32", "bf16"):
        check(q4.q4_linear_w4a16_mx(*args, yt), ref, mag, K, (tile, yt))
        assert q4.q4_last_path() == "tiled"


@pytest.mark.parametrize("tile,M,N", [(t, *s[0]) for t, s in S.W4A4.items()])
def test_w4a4_tiles_column_and_block(tile, M, N):
    """One-hot activation rows read single weights: exact, with every block's own scale."""
    for K in (1536, 1504):
        rng = np.random.default_rng(K)
        wq, sw = codes(rng, N, K, 100, 140)
        w = X.dequantize_rows(wq, sw, K).astype(np.float32)
        at = (np.arange(M) * 769 + 5) % K
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), at] = 1
        xq, sx = q4.q4_mx_quantize_rows(dev(x))
        y = host(q4.q4_linear_w4a4_mx(xq, sx, dev(wq), dev(sw), "f32"))
        assert np.array_equal(y, w[:, at].T), (tile, K)


@pytest.mark.parametrize("tile,M,N", [(t, *s[0]) for t, s in S.W4A16.items()])
def test_w4a16_tiles_column_and_block(tile, M, N):
    for K in (1536, 1408) if tile == "kLarge" else (1536, 1408, 1432, 1429):
        rng = np.random.default_rng(K)
        wq, sw = codes(rng, N, K, 100, 140)
        w = X.dequantize_rows(wq, sw, K).astype(np.float32)
        at = (np.arange(M) * 769 + 5) % K
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), at] = 1
        y = host(q4.q4_linear_w4a16_mx(dev(F.f32_to_bf16_bits(x)), dev(wq), dev(sw), "f32"))
        assert np.array_equal(y, w[:, at].T), (tile, K)


@pytest.mark.parametrize("op,tile,M,N", [(op, t, *s[0]) for op, d in (("w4a4", S.W4A4), ("w4a16", S.W4A16))
                                         for t, s in d.items()])
def test_tiles_keep_nan_in_its_row_and_column(op, tile, M, N):
    """Blocks of scale 255 at the edges of tiles, the last block of K among them."""
    for K in (1536, 1408):
        rng = np.random.default_rng(N)
        wq, sw = codes(rng, N, K, 110, 122)
        B = X.blocks(K)
        cols = sorted({0, 31, 63, 255, N // 2, N - 1})
        rows = sorted({1, 31, 62, M - 1})
        for i, n in enumerate(cols):
            sw[n, (B - 1, 0, B // 2)[i % 3]] = 255
        x = rng.standard_normal((M, K)).astype(np.float32)
        for i, m in enumerate(rows):
            x[m, (K - 1, 0, K // 2)[i % 3]] = np.nan
        xb = dev(x).bfloat16()
        if op == "w4a4":
            y = q4.q4_linear_w4a4_mx(*q4.q4_mx_quantize_rows(xb), dev(wq), dev(sw), "f32")
        else:
            y = q4.q4_linear_w4a16_mx(xb, dev(wq), dev(sw), "f32")
        want = np.zeros((M, N), bool)
        want[rows] = True
        want[:, cols] = True
        assert np.array_equal(np.isnan(host(y)), want), (op, tile, K)

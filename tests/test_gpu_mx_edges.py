"""MX FP4 at the ends of its range, and on streams that are not the default one.

Tolerances as in tests/test_gpu_mx.py; a float32 sum below 2^-126 keeps 2^-149
steps, so each of its n + 8 roundings adds up to 2^-150.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.mx as X
from tests.gpu_util import DEV, assert_bitwise, dev, host

pytestmark = pytest.mark.gpu

# few rows; the small tiles; the large ones, whole and cut
SHAPES = [("gemv", 3, 40, 96), ("gemv", 1, 70, 1100), ("tiled", 3, 40, 96), ("tiled", 300, 200, 512),
          ("tiled", 1290, 6401, 512)]


@pytest.fixture(autouse=True)
def _auto_path():
    yield
    q4.q4_set_path("auto")


def codes(rng, rows, K, lo, hi):
    B = X.blocks(K)
    c = rng.integers(0, 256, (rows, 16 * B), dtype=np.uint8)
    c[:, (K + 1) // 2:] = 0
    return c, rng.integers(lo, hi + 1, (rows, B), dtype=np.uint8)


def values(t):
    return t.double().cpu().numpy()


def close(y, ref, mag, K):
    assert np.all(np.abs(values(y) - ref) <= min(1e-5, (K + 8) * 2.0 ** -24) * mag + (K + 8) * 2.0 ** -150)


def test_quantize_every_finite_bf16():
    """All 65280 of them, 31 at a time under each of some block maxima."""
    b = np.arange(65536, dtype=np.uint16)
    b = b[np.isfinite(F.bf16_bits_to_f32(b))]
    assert len(b) == 65280
    b = np.concatenate([b, b[:-len(b) % 31]]).reshape(-1, 31)
    for top in (0x0000, 0x0001, 0x0080, 0x00FF, 0x3F80, 0x40DF, 0x7F7F):
        x = np.concatenate([b, np.full((len(b), 1), top, np.uint16)], 1)
        c, s = q4.q4_mx_quantize_rows(dev(x))
        cr, sr = X.quantize_rows(F.bf16_bits_to_f32(x))
        assert_bitwise(host(s), sr, f"scales under {top:#x}")
        assert_bitwise(host(c), cr, f"codes under {top:#x}")


@pytest.mark.parametrize("path,M,N,K", SHAPES)
def test_w4a16_weights_below_the_smallest_normal_bf16(path, M, N, K):
    """Scale bytes 0, 1 and 2: weights from 2^-128 on, subnormal in bf16, are not lost."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(M + K)
    wq, sw = codes(rng, N, K, 0, 2)
    x = (torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(K)) * 2.0 ** 100).bfloat16()
    close(q4.q4_linear_w4a16_mx(x, dev(wq), dev(sw), "f32"), *X.linear_w4a16(values(x), wq, sw), K)


@pytest.mark.parametrize("path,M,N,K", SHAPES)
def test_w4a16_activations_and_sums_below_the_smallest_normal(path, M, N, K):
    q4.q4_set_path(path)
    rng = np.random.default_rng(M + K + 1)
    # subnormal activations
    x = torch.from_numpy(rng.integers(1, 128, (M, K)).astype(np.int16)).to(DEV).view(torch.bfloat16)
    wq, sw = codes(rng, N, K, 230, 236)
    close(q4.q4_linear_w4a16_mx(x, dev(wq), dev(sw), "f32"), *X.linear_w4a16(values(x), wq, sw), K)
    # subnormal sums
    x = (torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(K)) * 2.0 ** -20).bfloat16()
    wq, sw = codes(rng, N, K, 10, 15)
    close(q4.q4_linear_w4a16_mx(x, dev(wq), dev(sw), "f32"), *X.linear_w4a16(values(x), wq, sw), K)


@pytest.mark.parametrize("path,M,N,K", SHAPES)
def test_w4a4_sums_below_the_smallest_normal(path, M, N, K):
    q4.q4_set_path(path)
    rng = np.random.default_rng(M + K + 2)
    xq, sx = codes(rng, M, K, 0, 3)
    wq, sw = codes(rng, N, K, 110, 115)
    close(q4.q4_linear_w4a4_mx(dev(xq), dev(sx), dev(wq), dev(sw), "f32"), *X.linear_w4a4(xq, sx, wq, sw), K)


@pytest.mark.parametrize("path,M,N,K", SHAPES)
def test_w4a16_weights_past_bf16_are_infinite(path, M, N, K):
    """2^128 and more, which a scale byte of 253 or 254 can stand for (the quantizer gives none above 252)."""
    q4.q4_set_path(path)
    wq = np.zeros((N, 16 * X.blocks(K)), np.uint8)
    sw = np.full((N, X.blocks(K)), 127, np.uint8)
    wq[::2, 3] = 0x05            # column 6: 3 in every other row, 6 in the others
    wq[1::2, 3] = 0x07
    sw[:, 0] = 253
    x = torch.full((M, K), 2.0 ** -100, device=DEV).bfloat16()
    y = values(q4.q4_linear_w4a16_mx(x, dev(wq), dev(sw), "f32"))
    assert np.all(y[:, ::2] == 3 * 2.0 ** 26) and np.all(np.isposinf(y[:, 1::2]))


# ---- streams -----------------------------------------------------------------

def late(t, value):
    """t becomes `value` after some milliseconds of work on the current stream."""
    a = torch.full((4096, 4096), 2.0 ** -12, device=DEV)
    for _ in range(8):
        a = torch.mm(a, a)          # every element stays 2^-12
    t.copy_(value * (a[0, 0] * 4096).to(value.dtype))


@pytest.mark.parametrize("M,N,K", [(1, 200, 640), (70, 200, 640), (300, 8200, 512)])
def test_calls_follow_the_current_stream(M, N, K):
    """Inputs that two side streams write late, each with its own, outputs allocated in the calls."""
    wq, sw = X.quantize_rows(np.random.default_rng(K).standard_normal((N, K)).astype(np.float32))
    w, s = dev(wq), dev(sw)
    D = 64
    cs = torch.randn(M, D, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    pos = torch.arange(M, device=DEV)
    gain = torch.ones(D, device=DEV, dtype=torch.bfloat16)
    want = [torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(i)).bfloat16() for i in range(2)]
    xs = [torch.zeros_like(t) for t in want]
    streams = [torch.cuda.Stream() for _ in want]
    out = []
    torch.cuda.synchronize()
    for st, x, v in zip(streams, xs, want):
        with torch.cuda.stream(st):
            late(x, v)
            h = x[:, :4 * D].view(M, 4, D)
            xq, sx = q4.q4_mx_quantize_rows(x)
            out.append([xq, sx, q4.q4_mx_dequantize_rows(xq, sx, K), q4.q4_linear_w4a4_mx(xq, sx, w, s, "f32"),
                        q4.q4_linear_w4a4_mx_dynamic(x, w, s, "f32"), q4.q4_linear_w4a16_mx(x, w, s, "f32"),
                        q4.q4_qk_norm_rope(h, h, gain, gain, pos, cs, dtype="f32")[1],
                        q4.q4_qk_norm_rope(h, None, None, None, pos, cs, dtype="f32")[0]])
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    angles = values(cs)
    for v, (xq, sx, back, y44, y44d, y416, k, q) in zip(want, out):
        x = values(v)
        cr, sr = X.quantize_rows(x)
        assert_bitwise(host(xq), cr)
        assert_bitwise(host(sx), sr)
        assert_bitwise(host(back), X.dequantize_rows(cr, sr, K).astype(np.float32))
        ref, mag = X.linear_w4a4(cr, sr, wq, sw)
        close(y44, ref, mag, K)
        close(y44d, ref, mag, K)
        close(y416, *X.linear_w4a16(x, wq, sw), K)
        ref, mag = X.qk_norm_rope(x[:, :4 * D].reshape(M, 4, D), None, angles[:, :D // 2], angles[:, D // 2:], 1e-6, True)
        for t in (k, q):
            assert np.all(np.abs(values(t) - ref) <= (D / 2 + 16) * 2.0 ** -24 * mag)


def test_given_workspaces():
    """Host memory and strided views are refused; a longer one of another type serves."""
    x = torch.randn(40, 64, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    c, s = q4.q4_mx_quantize_rows(x[:8])
    need = q4.q4_w4a4_mx_dynamic_workspace(40, 64)
    for ws in (torch.empty(need, dtype=torch.uint8), np.empty(need, np.uint8), need):
        with pytest.raises(TypeError):
            q4.q4_linear_w4a4_mx_dynamic(x, c, s, ws=ws)
    with pytest.raises(ValueError):
        q4.q4_linear_w4a4_mx_dynamic(x, c, s, ws=torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2])
    y = q4.q4_linear_w4a4_mx_dynamic(x, c, s, "f32", ws=torch.empty(need, dtype=torch.float32, device=DEV))
    assert_bitwise(host(y), host(q4.q4_linear_w4a4_mx_dynamic(x, c, s, "f32")))

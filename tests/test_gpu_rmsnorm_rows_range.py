"""Scales of q8_rmsnorm_rows over the whole range of rows: within 1e-6 of the
float64 oracle's (a square meets at most 19 roundings of the sum and twice its own
number's, each half a step of 2^-23, and the root halves them: 10.5 of 2^-24, with
the result's own 12, 7.2e-7), codes bit for bit."""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.serving as S
from tests.gpu_util import DEV, assert_bitwise, dev, host
from tests.test_gpu_rmsnorm_rows import TORCH, f64

pytestmark = pytest.mark.gpu
WIDTHS = [40, 757, 1000, 2048, 4000, 6000, 8000, 16000, 16392]   # one to 16 waves, in registers and read again


def check(x, gain, residual, eps, what):
    codes, scales, _ = q4.q8_rmsnorm_rows(x, gain, residual, eps)
    ref, sref, _ = S.rmsnorm_rows(f64(x), f64(residual), f64(gain), np.float64(np.float32(eps)))
    assert_bitwise(host(codes), ref, what)
    got = host(scales).astype(np.float64)
    # f32 ends at steps of 2^-149
    assert np.all(np.abs(got - sref) <= 1e-6 * np.abs(sref) + 2.0 ** -149), (what, got[:4], sref[:4])


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("K", WIDTHS)
def test_small_and_large_rows_without_eps(K, xt):
    """Squares far below the range of f32, and as near its end as the sum may come."""
    rng = np.random.default_rng(K)
    for power in (-120, -100, -80, -75, -70, -66, -60, 0, 50, 55):
        x, r = (dev((rng.standard_normal((3, K)) * 2.0 ** power).astype(np.float32)).to(TORCH[xt]) for _ in range(2))
        g = dev((1 + 0.2 * rng.standard_normal(K)).astype(np.float32))
        check(x, g, r, 0.0, f"2^{power}")
        check(x, None, None, 1e-30, f"2^{power} with a small eps")


@pytest.mark.parametrize("K", WIDTHS)
def test_products_below_the_range(K):
    """Rows times gains that are 0 or subnormal in f32: not rows of zeros."""
    rng = np.random.default_rng(K)
    x = dev((rng.standard_normal((2, K)) * 2.0 ** -90).astype(np.float32))
    for power in (-75, -58, -50):
        g = dev((rng.standard_normal(K) * 2.0 ** power).astype(np.float32))
        check(x, g, None, 0.0, f"gain 2^{power}")


@pytest.mark.parametrize("K", WIDTHS)
def test_rows_of_zeros_without_eps(K):
    x = torch.zeros(2, K, device=DEV)
    x[1, K // 2] = 3.0
    g = torch.ones(K, device=DEV)
    g[K // 2] = 0.0                        # the second row's only number meets a gain of 0
    for gain in (None, g):
        codes, scales, _ = q4.q8_rmsnorm_rows(x, gain, None, 0.0)
        ref, sref, _ = S.rmsnorm_rows(f64(x), None, f64(gain), 0.0)
        assert_bitwise(host(codes), ref, "codes")
        assert np.all(np.abs(host(scales) - sref) <= 1e-6 * sref)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2 ** 14, 2 ** 17, 2 ** 20, 2 ** 24])
def test_long_rows(K, xt):
    """Constant rows, whose roundings all go one way."""
    x = torch.full((1, K), 1.3, device=DEV).to(TORCH[xt])
    x[0, 5] = 2.6
    check(x, None, None, 1e-6, "constant")


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(2, 16392), (2, 20001), (300, 16400)])
def test_sum_in_place_of_rows_that_are_read_again(M, K, xt):
    gen = torch.Generator(DEV).manual_seed(2)
    x, r = (torch.randn(M, K, device=DEV, generator=gen).to(TORCH[xt]) for _ in range(2))
    want = [host(t) for t in q4.q8_rmsnorm_rows(x, None, r, 1e-6)]
    for place in ("residual", "x"):
        a, b = x.clone(), r.clone()
        got = q4.q8_rmsnorm_rows(a, None, b, 1e-6, total=b if place == "residual" else a)
        assert got[2].data_ptr() == (b if place == "residual" else a).data_ptr()
        for g, w in zip(got, want):
            assert_bitwise(host(g), w, place)


@pytest.mark.parametrize("K", WIDTHS)
def test_codes_next_to_borders_at_every_width(K):
    """Quotients that are ties and their neighbours, over and over; the largest is 127."""
    half = (np.arange(-126, 126) + 0.5).astype(np.float32)
    up, down = (np.nextafter(half, np.float32(s)) for s in (1e9, -1e9))
    x = np.resize(np.concatenate([[np.float32(127)], half, up, down]), (1, K))
    for s in (1.0, 2.0 ** -110, 2.0 ** 40, 3.0):
        check(dev((x * np.float32(s)).astype(np.float32)), None, None, 1e-6, f"times {s}")

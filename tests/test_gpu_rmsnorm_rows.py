"""Rows to int8 with norm and residual on the GPU against the float64 oracle.

Codes are those of the oracle, bit for bit, on every route: both divide the same
float64 numbers where an f32 quotient lies next to a border.  A scale carries the
square sum's chain (at most K / 2 + 16 roundings of half a step, 2^-24) and a
handful more; the sum is the f32 sum, rounded once.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.linear as L
import oracle.serving as S
from tests.gpu_util import DEV, assert_bitwise, dev, host

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def check(x, gain, residual, eps, what, total=None):
    r64, x64 = f64(residual), f64(x)
    got = q4.q8_rmsnorm_rows(x, gain, residual, eps, total)
    codes, scales, h = (None if t is None else host(t) for t in got)
    ref, sref, _ = S.rmsnorm_rows(x64, r64, f64(gain), eps)
    assert_bitwise(codes, ref, what)
    K = x.shape[1]
    tol = (K / 2 + 16) * 2.0 ** -24 * np.abs(sref) + 2.0 ** -149
    bad = np.argwhere(~((np.abs(scales - sref) <= tol) | (np.isnan(scales) & np.isnan(sref))))
    assert bad.size == 0, (what, bad[:3].tolist())
    if residual is None:
        assert h is None
    else:
        want = x64.astype(np.float32) + r64.astype(np.float32)
        assert_bitwise(h, F.f32_to_bf16_bits(want) if x.dtype == torch.bfloat16 else want, what + " sum")
    return got


# rows of one to 16 waves, in registers and read again; whole and partial runs of 8
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 511), (7, 512), (1, 520), (2, 1023), (3, 2048),
                                 (2, 2049), (1, 4095), (2, 5632), (1, 8191), (2, 8192), (2, 8200), (1, 13312), (2, 16384), (1, 20001), (130, 64)])
def test_parity(M, K, xt):
    rng = np.random.default_rng(M + K)
    x, r = (dev(rng.standard_normal((M, K)).astype(np.float32)).to(TORCH[xt]) for _ in range(2))
    g = dev((1 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    check(x, g, r, 1e-6, "all")
    check(x, g.bfloat16(), None, 1e-5, "no residual")
    check(x, None, r, 0.0, "no gain")


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [64, 520, 1000, 1024, 1500, 2048])
def test_many_rows(K, xt):
    """More rows than run at a time."""
    gen = torch.Generator(DEV).manual_seed(K)
    x, r = (torch.randn(2050, K, device=DEV, generator=gen).to(TORCH[xt]) for _ in range(2))
    g = (1 + 0.1 * torch.randn(K, device=DEV, generator=gen)).to(TORCH[xt])
    check(x, g, r, 1e-6, "rows")


def test_codes_next_to_borders():
    """Rows whose quotients are ties and their neighbours: the largest is 127, the others n + 1/2 and a step of it."""
    half = np.arange(-126, 126) + 0.5
    up, down = (np.nextafter(half.astype(np.float32), np.float32(s)) for s in (1e9, -1e9))
    x = np.concatenate([half.astype(np.float32), up, down, [np.float32(127)]])[None]
    for s in (1.0, 2.0 ** -110, 2.0 ** 40, 3.0):
        check(dev((x * np.float32(s)).astype(np.float32)), None, None, 1e-6, f"times {s}")
    b = dev(np.concatenate([half, [127.0]])[None].astype(np.float32)).bfloat16()     # exact in bf16
    check(b, None, b * 0.5, 1e-6, "bf16 ties")


def test_zero_rows_and_non_finite_values():
    x = torch.randn(7, 40, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 39] = float("nan")
    x[3, 0] = float("-inf")
    x[4] *= 1e-30                        # the square sum is 0
    codes, scales, _ = check(x, None, None, 1e-6, "rows")
    assert not host(codes)[[0, 1, 2, 3]].any() and np.isnan(host(scales)[[1, 2, 3]]).all() and host(scales)[0] == 0
    g = torch.ones(40, device=DEV)
    g[5] = float("nan")
    codes, scales, _ = q4.q8_rmsnorm_rows(x, g, None, 1e-6)
    assert np.isnan(host(scales)).all() and not host(codes).any()
    x[5] = 1e25                          # the square sum passes the range of f32
    codes, scales, total = q4.q8_rmsnorm_rows(x, None, x, 1e-6)
    assert np.isnan(host(scales)[5]) and not host(codes)[5].any()
    assert_bitwise(host(total)[5], host(x)[5] * np.float32(2), "the sum is written all the same")


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(3, 100), (2, 2048), (2060, 700), (2, 9000)])
def test_sum_in_place(M, K, xt):
    gen = torch.Generator(DEV).manual_seed(2)
    x, r = (torch.randn(M, K, device=DEV, generator=gen).to(TORCH[xt]) for _ in range(2))
    want = [host(t) for t in q4.q8_rmsnorm_rows(x, None, r, 1e-6)]
    for place in ("residual", "x"):
        a, b = x.clone(), r.clone()
        got = q4.q8_rmsnorm_rows(a, None, b, 1e-6, total=b if place == "residual" else a)
        assert got[2].data_ptr() == (b if place == "residual" else a).data_ptr()
        for g, w in zip(got, want):
            assert_bitwise(host(g), w, place)


def test_rows_at_any_address():
    buf = torch.randn(4000, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).bfloat16()
    for off in (1, 3, 8):
        check(buf[off:off + 3 * 333].view(3, 333), buf[off + 1:off + 334], buf[2000 + off:2000 + off + 999].view(3, 333),
              1e-6, f"from {off}")


def test_feeds_the_int8_linears():
    """Norm, then the W4A8 product of its codes: as the oracle's product of the same codes, bit for bit."""
    rng = np.random.default_rng(4)
    x, r = (dev(rng.standard_normal((5, 256)).astype(np.float32)).bfloat16() for _ in range(2))
    W = rng.standard_normal((96, 256), dtype=np.float32)
    packed, sw = q4.q4_quantize_matrix(W)
    codes, scales, _ = q4.q8_rmsnorm_rows(x, None, r)
    y = q4.q4_linear_w4a8(codes, scales, dev(packed), dev(sw))
    assert_bitwise(host(y), L.linear_w4a8(host(codes), host(scales), packed, sw, 0, F.EXCESS8), "product")


def test_refused():
    x = torch.zeros(3, 16, device=DEV)
    for bad in (lambda: q4.q8_rmsnorm_rows(x.t()), lambda: q4.q8_rmsnorm_rows(x, torch.ones(15, device=DEV)),
                lambda: q4.q8_rmsnorm_rows(x, None, x[:2]), lambda: q4.q8_rmsnorm_rows(x, total=x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q8_rmsnorm_rows(x.half()), lambda: q4.q8_rmsnorm_rows(x, None, x.bfloat16()),
                lambda: q4.q8_rmsnorm_rows(x, torch.ones(16, device=DEV).half())):
        with pytest.raises(TypeError):
            bad()
    buf = torch.zeros(64, device=DEV)
    for bad in (lambda: q4.q8_rmsnorm_rows(x, eps=-1.0), lambda: q4.q8_rmsnorm_rows(x, eps=float("nan")),
                lambda: q4.q8_rmsnorm_rows(buf[:48].view(3, 16), None, x, total=buf[8:56].view(3, 16))):
        with pytest.raises(q4.Q4Error) as e:
            bad()
        assert e.value.status == q4.EINVAL
    codes, scales, none = q4.q8_rmsnorm_rows(torch.zeros(0, 16, device=DEV))
    assert codes.shape == (0, 16) and scales.shape == (0,) and none is None
    codes, scales, _ = q4.q8_rmsnorm_rows(torch.zeros(3, 0, device=DEV))
    assert codes.shape == (3, 0) and not host(scales).any()


def test_graph_replays():
    x, r = (torch.zeros(3, 2048, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q4.q8_rmsnorm_rows(x, None, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q4.q8_rmsnorm_rows(x, None, r)
    for seed in range(4):
        gen = torch.Generator(DEV).manual_seed(seed)
        x.copy_(torch.randn(x.shape, device=DEV, generator=gen))
        r.copy_(torch.randn(x.shape, device=DEV, generator=gen))
        graph.replay()
        got = [host(o) for o in out]
        for a, b in zip(got, q4.q8_rmsnorm_rows(x, None, r)):
            assert_bitwise(a, host(b), f"replay {seed}")


def test_both_paths_of_the_binding_agree(monkeypatch):
    x = torch.randn(3, 100, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    a = q4.q8_rmsnorm_rows(x, x[0], x)
    monkeypatch.setattr(q4, "_DIRECT", q4._NoDirect())
    for t, u in zip(a, q4.q8_rmsnorm_rows(x, x[0], x)):
        assert_bitwise(host(t), host(u), "paths")

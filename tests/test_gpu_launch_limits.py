"""Calls whose launch would have more threads along an axis than a grid can
(2^32): rows of heads and weight rows past that go out in several launches.

The inputs are zeros but for the rows that are compared: the first, the last,
and those around the launches' borders (2^24 workgroups of 256 threads).
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.mx as X
from tests.gpu_util import DEV, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,xt,pairs", [(66, torch.bfloat16, "halves"), (256, torch.float32, "neighbours")])
def test_head_rows_past_a_grid(D, xt, pairs):
    """2^26 + 64 rows of heads, a wave each."""
    H, T, R, P = 64, (1 << 20) + 1, D, 7
    rng = np.random.default_rng(D)
    x = torch.from_numpy(rng.standard_normal((H, D)).astype(np.float32)).to(DEV).to(xt)
    q = x[None].expand(T, H, D)                 # every token has the same heads, at its own position
    pos = torch.arange(T, device=DEV) % P
    cs = rng.standard_normal((P, R)).astype(np.float32)
    y, _ = q4.q4_qk_norm_rope(q, None, None, None, pos, torch.from_numpy(cs).to(DEV), 1e-6, pairs, "bf16")
    small, _ = q4.q4_qk_norm_rope(q[:P], None, None, None, pos[:P], torch.from_numpy(cs).to(DEV), 1e-6, pairs, "bf16")
    ref, mag = X.qk_norm_rope(x.double().cpu().numpy()[None].repeat(P, 0), None, cs[:, :R // 2].astype(np.float64),
                              cs[:, R // 2:].astype(np.float64), 1e-6, pairs == "halves")
    tol = (D / 2 + 16) * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    assert np.all(np.abs(small.double().cpu().numpy() - ref) <= tol)
    whole = T // P * P
    assert (y[:whole].view(-1, P, H, D) == small).all() and (y[whole:] == small[:T - whole]).all()


@pytest.mark.parametrize("op", ["w4a4", "w4a4_dynamic", "w4a16"])
def test_weight_rows_past_a_grid(op):
    """2^28 + 40 weight rows of one block, 16 to a workgroup."""
    N, K, M = (1 << 28) + 40, 32, 2
    at = np.array([0, 1, 17, (1 << 27) + 3, (1 << 28) - 17, (1 << 28) - 16, (1 << 28) - 15, (1 << 28) - 1, 1 << 28,
                   (1 << 28) + 15, (1 << 28) + 16, N - 1])
    rng = np.random.default_rng(11)
    wq, sw = X.quantize_rows(rng.standard_normal((len(at), K)))
    i = torch.from_numpy(at).to(DEV)
    w = torch.zeros((N, 16), dtype=torch.uint8, device=DEV)
    s = torch.full((N, 1), 127, dtype=torch.uint8, device=DEV)
    w[i], s[i] = torch.from_numpy(wq).to(DEV), torch.from_numpy(sw).to(DEV)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DEV).bfloat16()
    v = x.double().cpu().numpy()
    if op == "w4a16":
        y = q4.q4_linear_w4a16_mx(x, w, s, "f32")
        ref, mag = X.linear_w4a16(v, wq, sw)
    else:
        xq, sx = q4.q4_mx_quantize_rows(x)
        y = q4.q4_linear_w4a4_mx(xq, sx, w, s, "f32") if op == "w4a4" else q4.q4_linear_w4a4_mx_dynamic(x, w, s, "f32")
        ref, mag = X.linear_w4a4(*X.quantize_rows(v), wq, sw)
    assert np.all(np.abs(host(y[:, i]) - ref) <= (K + 8) * 2.0 ** -24 * mag)
    y[:, i] = 0
    assert not y.any()


@pytest.fixture
def _auto_path():
    yield
    q4.q4_set_path("auto")


@pytest.mark.parametrize("K,xt", [(8, torch.float32), (8, torch.bfloat16), (3, torch.float32)])
def test_int8_rows_past_a_grid(K, xt):
    """2^24 + 1000 activation rows, a workgroup each."""
    P, M = 11, (1 << 24) + 1000
    gen = torch.Generator(DEV).manual_seed(K)
    x = torch.randn(P, K, device=DEV, generator=gen).to(xt)
    q, s = q4.q8_quantize_rows(x)
    whole = M // P * P
    qm, sm = q4.q8_quantize_rows(x[torch.arange(M, device=DEV) % P])
    assert (qm[:whole].view(-1, P, K) == q).all() and (qm[whole:] == q[:M - whole]).all()
    assert (sm[:whole].view(-1, P) == s).all() and (sm[whole:] == s[:M - whole]).all()


def test_zeros_past_a_grid():
    """A result of 2^36 bytes and more that is all zeros (no columns to sum)."""
    M, N = 16400, 1 << 20
    z = torch.zeros((N, 0), dtype=torch.uint8, device=DEV)
    y = torch.full((M, N), float("nan"), device=DEV)
    q4.q4_linear_w4a4_mx(z[:M], z[:M], z, z, "f32", y=y)
    for part in y.split(1024):
        assert (part == 0).all()


@pytest.mark.parametrize("N,path", [((1 << 26) + 21, "generic"), ((1 << 28) + 21, "auto")])
@pytest.mark.parametrize("op", ["w4a32", "w4a16", "w4a16_zp", "w4a8", "w4a8_grouped", "w4a8_dynamic", "w8a8", "w8a16"])
def test_int4_and_int8_weight_rows_past_a_grid(op, N, path, _auto_path):
    """Weight rows past a launch of the general kernels (2^26) and past one of
    the decode kernels (2^28): 13 rows over and over, so the results repeat."""
    P, M = 13, 1
    K, G = (32, 32) if path == "auto" else (8, 4)
    if op in ("w4a8_grouped", "w4a16_zp"):
        G = K
    rng = np.random.default_rng(K + len(op))
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DEV)
    wide = 1 if op.startswith("w8") else 2
    w = torch.from_numpy(rng.integers(0, 256, (P, K // wide), dtype=np.uint8)).to(DEV)
    s = torch.from_numpy(rng.uniform(0.5, 2, (P, K // G)).astype(np.float32)).to(DEV)
    z = torch.from_numpy(rng.integers(0, 16, (P, K // G), dtype=np.uint8)).to(DEV)
    xq, sx = q4.q8_quantize_rows(x)

    def call(n):
        # (not by an index: torch's own launch for so many rows wraps as well)
        wn, sn, zn = (t.repeat(-(-n // P), 1)[:n] for t in (w, s, z))
        if op == "w4a32":
            return q4.q4_linear_w4a32(x, wn, sn.half(), G)
        if op == "w4a16":
            return q4.q4_linear_w4a16(x.bfloat16(), wn, sn.bfloat16(), G)[0]
        if op == "w4a16_zp":
            return q4.q4_linear_w4a16_zp(x.bfloat16(), wn, sn.bfloat16(), zn, G)[0]
        if op == "w4a8":
            return q4.q4_linear_w4a8(xq, sx, wn, sn[:, 0].contiguous(), 0)
        if op == "w4a8_grouped":
            return q4.q4_linear_w4a8(xq, sx, wn, sn, G)
        if op == "w4a8_dynamic":
            return q4.q4_linear_w4a8_dynamic(x, wn, sn[:, 0].contiguous(), 0)
        if op == "w8a8":
            return q4.q8_linear_w8a8(xq, sx, wn.view(torch.int8), sn[:, 0].contiguous())
        return q4.q8_linear_w8a16(x.bfloat16(), wn.view(torch.int8), sn[:, 0].contiguous())[0]

    q4.q4_set_path("generic")   # the kernels that serve what is past the decode kernels' launches
    small = call(P)
    q4.q4_set_path(path)
    y = call(N)
    assert y.shape == (M, N)
    whole = N // P * P
    assert (y[:, :whole].view(M, -1, P) == small[:, None]).all() and (y[:, whole:] == small[:, :N - whole]).all()

"""Head norms with rotation on the GPU against the float64 oracle.

An f32 result carries at most D / 2 + 16 roundings (the square sum's chain, the
root, the quotient, three products and a sum) of half a step (2^-24) of the
magnitudes that it is the sum of; a bf16 one half a bf16 step (2^-8) of itself
more.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.mx as X
from tests.gpu_util import DEV, assert_bitwise, dev, host

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def table(P, R, base=10000.0):
    a = np.arange(P)[:, None] * base ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(y, x, gain, cs, pos, eps, pairs, what):
    D, R = x.shape[2], cs.shape[1]
    rows = cs.astype(np.float64)[pos]
    ref, mag = X.qk_norm_rope(f64(x), None if gain is None else f64(gain), rows[:, :R // 2], rows[:, R // 2:], eps,
                              pairs == "halves")
    tol = (D / 2 + 16) * 2.0 ** -24 * mag + 1e-44
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    bad = np.argwhere(~(np.abs(f64(y) - ref) <= tol))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist())


CASES = [(1, 1, 1, 2, 2), (1, 16, 16, 128, 128), (3, 7, 1, 80, 32), (5, 4, 2, 64, 64), (61, 3, 3, 96, 96),
         (2, 5, 5, 250, 250), (17, 8, 2, 256, 64), (4, 2, 1, 34, 6), (2, 3, 2, 512, 512), (1, 2, 1, 1030, 1030),
         (130, 32, 8, 128, 128), (9, 6, 2, 72, 16), (3, 2, 2, 130, 2)]


@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", CASES)
def test_parity(T, Hq, Hk, D, R, pairs, xt, yt):
    """Slices of a fused projection, as they lie."""
    rng = np.random.default_rng(T + Hq + D + R)
    P, eps = 333, 1e-6
    qkv = dev(rng.standard_normal((T, (Hq + 2 * Hk) * D)).astype(np.float32)).to(TORCH[xt])
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    gt = xt if (T + Hq) % 2 else yt
    gq, gk = (dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(TORCH[gt]) for _ in range(2))
    pos = rng.integers(0, P, T)
    cs = table(P, R)
    qo, ko = q4.q4_qk_norm_rope(q, k, gq, gk, dev(pos), dev(cs), eps, pairs, yt)
    assert qo.dtype == ko.dtype == TORCH[yt] and qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, gq, cs, pos, eps, pairs, "queries")
    check(ko, k, gk, cs, pos, eps, pairs, "keys")


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_other_layouts(pairs, xt):
    """Head-major inputs, shared heads (stride 0), odd starts, no keys, no gains."""
    rng = np.random.default_rng(7)
    T, H, D, R = 6, 4, 64, 32
    cs, pos = table(50, R), rng.integers(0, 50, T)
    buf = dev(rng.standard_normal(2 * T * H * D + 9).astype(np.float32)).to(TORCH[xt])
    q = buf[1:1 + T * H * D].view(H, T, D).transpose(0, 1)
    k = buf[T * H * D + 3:T * H * D + 3 + T * D].view(T, 1, D).expand(T, H, D)
    qo, ko = q4.q4_qk_norm_rope(q, k, None, None, dev(pos), dev(cs), 1e-5, pairs)
    check(qo, q, None, cs, pos, 1e-5, pairs, "head-major")
    check(ko, k, None, cs, pos, 1e-5, pairs, "shared")
    q2, none = q4.q4_qk_norm_rope(q, None, None, None, dev(pos), dev(cs), 1e-5, pairs)
    assert none is None
    assert_bitwise(host(q2), host(qo), "without keys")


def test_zero_rows_and_non_finite_values():
    T, H, D = 3, 2, 64
    x = torch.zeros((T, H, D), device=DEV)
    x[1, 0, 5] = float("inf")
    x[2, 1, 63] = float("nan")
    cs, pos = dev(table(4, D)), torch.zeros(T, dtype=torch.int64, device=DEV)
    y, _ = q4.q4_qk_norm_rope(x, None, None, None, pos, cs, 1e-6)
    y = host(y)
    assert not y[0].any() and not y[1, 1].any() and not y[2, 0].any()      # zeros stay zeros
    # infinity over its own infinite root mean square, and NaN in its whole row
    assert np.isnan(y[1, 0, 5]) and np.isnan(y[2, 1]).all()
    y0, _ = q4.q4_qk_norm_rope(x, None, None, None, pos, cs, 0.0)          # 0 / 0
    assert np.isnan(host(y0)[0]).all()


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_unknown_positions_give_nan(pairs):
    T, H, D, R, P = 6, 3, 128, 64, 20
    x = torch.randn((T, H, D), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    pos = torch.tensor([0, -1, 19, 20, 2 ** 62, -2 ** 62], device=DEV)
    cs = table(P, R)
    y, _ = q4.q4_qk_norm_rope(x, None, None, None, pos, dev(cs), 1e-6, pairs)
    good = [0, 2]
    check(y[good], x[good], None, cs, pos[good].cpu().numpy(), 1e-6, pairs, "known")
    for t in (1, 3, 4, 5):
        n = np.isnan(host(y[t]))
        assert n[:, :R].all() and not n[:, R:].any()


def test_far_positions_and_large_rows():
    """A table of a million positions; rows whose offsets pass 2^32 bytes."""
    R = D = 128
    P = 1 << 20
    cs = table(P, R)
    T, H = 300000, 64
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 131071, 262143, 262144, T - 1]
    q[torch.tensor(at, device=DEV)] = torch.randn((len(at), H, D), device=DEV,
                                                  generator=torch.Generator(DEV).manual_seed(3)).bfloat16()
    pos = torch.arange(T, device=DEV) * 3 + (P - 3 * T)
    y, _ = q4.q4_qk_norm_rope(q, None, None, None, pos, dev(cs), 1e-6)
    i = torch.tensor(at, device=DEV)
    check(y[i], q[i], None, cs, pos[i].cpu().numpy(), 1e-6, "halves", "ends")
    assert not y[2:131071].any()


def test_empty_and_refused():
    cs = torch.zeros((4, 8), device=DEV)
    q = torch.zeros((0, 3, 16), device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    y, _ = q4.q4_qk_norm_rope(q, None, None, None, none, cs)
    assert y.shape == (0, 3, 16)
    q = torch.zeros((2, 3, 16), device=DEV)
    pos = torch.zeros(2, dtype=torch.int64, device=DEV)
    g = torch.ones(16, device=DEV)
    for bad in (lambda: q4.q4_qk_norm_rope(q.transpose(1, 2), None, None, None, pos, cs),
                lambda: q4.q4_qk_norm_rope(q, q[:1], None, None, pos, cs),
                lambda: q4.q4_qk_norm_rope(q, None, g[:8].contiguous(), None, pos, cs),
                lambda: q4.q4_qk_norm_rope(q, None, None, None, pos[:1], cs)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q4_qk_norm_rope(q, q.bfloat16(), None, None, pos, cs),
                lambda: q4.q4_qk_norm_rope(q, q, g, g.bfloat16(), pos, cs),
                lambda: q4.q4_qk_norm_rope(q, None, None, None, pos.int(), cs),
                lambda: q4.q4_qk_norm_rope(q.half(), None, None, None, pos, cs)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_qk_norm_rope(q, None, None, None, pos, torch.zeros((4, 18), device=DEV))
    assert e.value.status == q4.ESHAPE


def test_graph_replays():
    T, H, D = 5, 8, 128
    cs = dev(table(64, D))
    qk = torch.zeros((T, 2 * H * D), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(T, dtype=torch.int64, device=DEV)

    def call():
        return q4.q4_qk_norm_rope(qk[:, :H * D].view(T, H, D), qk[:, H * D:].view(T, H, D), None, None, pos, cs)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(4):
        gen = torch.Generator(DEV).manual_seed(seed)
        qk.copy_(torch.randn(qk.shape, device=DEV, generator=gen))
        pos.copy_(torch.randint(0, 64, (T,), device=DEV, generator=gen))
        graph.replay()
        got = [host(o) for o in out]
        for a, b in zip(got, call()):
            assert_bitwise(a, host(b), f"replay {seed}")

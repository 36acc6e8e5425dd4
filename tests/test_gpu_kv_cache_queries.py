"""Normalised queries past the range that f32 squares have, against the float64 oracle."""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.serving as S
from tests.gpu_util import DEV, dev
from tests.test_gpu_kv_cache import TORCH, f64, i32, new_pages, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("how", ["halves", "neighbours", "plain", "lds"])
@pytest.mark.parametrize("D", [16, 128, 240])
def test_queries_of_all_sizes(D, how, xt, yt):
    """Normalised queries from 1e-30 to 1e38 with eps 0, rows of both kinds side by side, and one row of zeros with eps:
    a query carries at most D / 2 + 16 half steps of f32 of the magnitudes that it is the sum of."""
    rng = np.random.default_rng(D)
    T, Hq = 24, 3
    R = {"lds": 10}.get(how, D)
    size = np.concatenate([10.0 ** np.array([-30, -25, -22, -20, -19, -18, -10, 0, 10, 18, 19, 20, 25, 30, 37, 37]),
                           np.ones(T - 16)])
    q = dev((np.clip(rng.standard_normal((T, Hq, D)), -9, 9) * size[:, None, None]).astype(np.float32)).to(TORCH[xt])
    k = torch.randn(T, 1, D, device=DEV).to(TORCH[xt])
    g = dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    pages, P = new_pages(rng, [T], 16)
    cs = None if how == "plain" else table(T, R)
    for eps in (0.0, 1e-6):
        if eps:
            q[3] = 0
        cache = q4.q8_kv_cache(P, 1, 16, D)
        out = f64(q4.q8_kv_append(cache, dev(pages), i32([0, T]), i32([T]), k, k, q, None if cs is None else dev(cs), None, g,
                                  eps, "neighbours" if how == "neighbours" else "halves", yt))
        for t in range(T):
            for h in range(Hq):
                x, e = f64(q[t, h]), float(np.float32(eps))
                ref = S.head(x, f64(g), e, None if cs is None else cs[t], how != "neighbours")
                plain = S.head(x, f64(g), e, None, True)
                mag = np.abs(plain) + (0 if cs is None else np.abs(plain).max())
                tol = (D / 2 + 16) * 2.0 ** -24 * mag + 1e-44 + (2.0 ** -8 * np.abs(ref) if yt == "bf16" else 0)
                assert np.all(np.abs(out[t, h] - ref) <= tol), (eps, t, h, size[t], out[t, h][:3], ref[:3])


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_queries_that_are_not_finite(eps, xt):
    """As the formula has it: x / sqrt(mean) with an infinite mean is 0 where x is finite and NaN where it is not."""
    T, Hq, D = 5, 2, 64
    gen = torch.Generator(DEV).manual_seed(1)
    q = torch.randn(T, Hq, D, device=DEV, generator=gen)
    q[1, 0, 7], q[2, 1, 3], q[3, 0, 0], q[3, 0, 9] = float("inf"), float("nan"), float("-inf"), float("inf")
    q = q.to(TORCH[xt])
    k = torch.randn(T, 1, D, device=DEV, generator=gen).to(TORCH[xt])
    pages, P = new_pages(np.random.default_rng(1), [T], 16)
    out = f64(q4.q8_kv_append(q4.q8_kv_cache(P, 1, 16, D), dev(pages), i32([0, T]), i32([T]), k, k, q, eps=eps, dtype="f32"))
    for t in range(T):
        for h in range(Hq):
            with np.errstate(invalid="ignore"):
                ref = S.head(f64(q[t, h]), None, float(np.float32(eps)), None, True)
            tol = (D / 2 + 16) * 2.0 ** -24 * np.abs(ref)
            assert np.all((np.abs(out[t, h] - ref) <= tol) | (np.isnan(out[t, h]) & np.isnan(ref))), (t, h)

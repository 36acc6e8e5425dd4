"""Calls whose launch would have more threads along an axis than a grid can
(2^32): rows of heads past that go out in several launches.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.mx as X
from tests.gpu_util import DEV

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

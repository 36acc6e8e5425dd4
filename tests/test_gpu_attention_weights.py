"""Weights of the attention of single tokens and short chunks (up to 16 rows of a
sequence and key head): bf16 results are those of f32, rounded once, so they carry
no rounding of the weights that the f32 ones do not (which test_gpu_attention.py
bounds by 2^-22)."""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
from tests.gpu_util import DEV, assert_bitwise, dev, host
from tests.test_gpu_attention import on_gpu, random_pool
from tests.test_gpu_kv_cache import i32, new_pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_bf16_results_are_f32_ones_rounded_once(D, xt):
    rng = np.random.default_rng(D)
    lengths, new = [1500, 17, 300, 64], [1, 8, 11, 1]
    pages, P = new_pages(rng, lengths, 32)
    cache = on_gpu(random_pool(rng, P, 2, 32, D))
    q = torch.randn(sum(new), 6, D, device=DEV, generator=torch.Generator(DEV).manual_seed(D))
    q = q.to(torch.bfloat16 if xt == "bf16" else torch.float32)
    starts = i32(np.concatenate([[0], np.cumsum(new)]))
    for kw in ({}, {"max_len": 0}, {"window": 100, "sinks": 3}):
        a, b = (q4.q8_attention(q, cache, dev(pages), starts, i32(lengths), dtype=t, **kw) for t in ("bf16", "f32"))
        assert q4.q4_last_path() == "gemv"
        assert_bitwise(host(a), host(b.bfloat16()), str(kw))

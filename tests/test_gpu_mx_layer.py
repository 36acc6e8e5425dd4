"""The decoder-layer example on the GPU: its projections and rotated heads
against the float64 oracle, and its two paths against each other.

A bf16 result is off by half a bf16 step (2^-8 of itself) and the float32 sum's
1e-5 of its terms' magnitudes; a head's result likewise with (D / 2 + 16) half
steps of float32.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.mx as X
from tests.gpu_util import DEV, host

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_decoder_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("mx_decoder_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def bits(t):
    return F.bf16_bits_to_f32(host(t.contiguous())).astype(np.float64)


def close(got, ref, mag, f32):
    assert np.all(np.abs(got - ref) <= f32 * mag + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134)


@pytest.mark.parametrize("path", ["prompt", "token"])
def test_projection_and_heads_against_the_oracle(path):
    layer = example().Layer(hidden=320, heads=4, kv_heads=2, head=64, ffn=352, positions=128)
    T = 21
    x = torch.randn(T, 320, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).bfloat16()
    at = torch.arange(T, device=DEV) * 5 + 2
    wq, sw = (host(t) for t in layer.qkv)
    if path == "prompt":
        qkv = q4.q4_linear_w4a4_mx_dynamic(x, *layer.qkv)
        ref, mag = X.linear_w4a4(*X.quantize_rows(bits(x)), wq, sw)
    else:
        qkv = q4.q4_linear_w4a16_mx(x, *layer.qkv)
        ref, mag = X.linear_w4a16(bits(x), wq, sw)
    close(bits(qkv), ref, mag, 1e-5)
    q, k, v = layer.heads_of(qkv, at)
    rows = host(layer.cos_sin)[host(at)].astype(np.float64)
    for got, lo, n, gain in ((q, 0, 4, layer.q_gain), (k, 4, 2, layer.k_gain)):
        part = bits(qkv)[:, lo * 64:(lo + n) * 64].reshape(T, n, 64)
        r, m = X.qk_norm_rope(part, bits(gain), rows[:, :32], rows[:, 32:], 1e-6, True)
        close(bits(got), r, m, (32 + 16) * 2.0 ** -24)
    assert np.array_equal(bits(v), bits(qkv)[:, 6 * 64:].reshape(T, 2, 64))


def test_prompts_do_not_see_each_other():
    """A prompt's rows are the same alone and behind another one (to the sums' order)."""
    layer = example().Layer(hidden=320, heads=4, kv_heads=2, head=64, ffn=352, positions=128)
    gen = torch.Generator(DEV).manual_seed(4)
    a, b = (torch.randn(n, 320, device=DEV, generator=gen).bfloat16() for n in (7, 12))
    both, caches = layer.prompt(torch.cat((a, b)), [7, 12])
    ya, (ca,) = layer.prompt(a, [7])
    yb, (cb,) = layer.prompt(b, [12])
    # products of so few weight rows do not depend on the batch, and every other step is by row
    for got, want in ((both[:7], ya), (both[7:], yb), (caches[0][0], ca[0]), (caches[1][1], cb[1])):
        assert torch.equal(got, want)


def test_tokens_extend_the_caches():
    layer = example().Layer(hidden=320, heads=4, kv_heads=2, head=64, ffn=352, positions=128)
    gen = torch.Generator(DEV).manual_seed(5)
    x = torch.randn(9, 320, device=DEV, generator=gen).bfloat16()
    _, caches = layer.prompt(x, [1, 8])
    y = torch.randn(2, 320, device=DEV, generator=gen).bfloat16()
    alone, _ = layer.token(y[1:], caches[1:])
    y, after = layer.token(y, caches)
    assert torch.equal(y[1:], alone) and torch.isfinite(y).all()
    assert [k.shape[0] for k, _ in after] == [2, 9]
    assert torch.equal(after[1][0][:8], caches[1][0])


def test_example_runs():
    example().main()

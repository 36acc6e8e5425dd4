"""The operators between a decoder layer's linears together: norm, int8 product,
cache and attention, call after call, each against the oracle on what the call
before it really gave; then a whole layer for prompts, chunks and single tokens.

Tolerances are those of the operators' own tests; int8 products with f32 scales
are the oracle's bit for bit.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.linear as L
import oracle.serving as S
from tests.gpu_util import DEV, assert_bitwise, host
from tests.test_gpu_attention import check as check_attention
from tests.test_gpu_kv_cache import Both, f64, i32, new_pages
from tests.test_gpu_rmsnorm_rows import check as check_norm

pytestmark = pytest.mark.gpu
EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def small(name="w4a8_decoder_layer"):
    return example(name).Layer(hidden=320, heads=4, kv_heads=2, head=64, ffn=352, positions=256)


def rows(n, seed):
    return torch.randn(n, 320, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))


def test_the_run_against_the_oracle():
    """Prompts, then a chunk beside single tokens: every call of attention's half of the layer."""
    layer, rng = small(), np.random.default_rng(0)
    H, K, D = 4, 2, 64
    final = [50, 9, 35]
    pages, P = new_pages(rng, final, 16)
    both, cs = Both(P, K, 16, D, rng), host(layer.cos_sin)
    have = [0, 0, 0]
    for at, new in enumerate(([30, 7, 20], [20, 1, 1], [0, 1, 14])):
        have = [a + b for a, b in zip(have, new)]
        starts = np.concatenate([[0], np.cumsum(new)])
        x, r = rows(sum(new), 10 + at), rows(sum(new), 20 + at)
        codes, scales, total = check_norm(x, layer.gain_in, r, 1e-6, f"norm {at}")
        qkv = q4.q4_linear_w4a8(codes, scales, *layer.qkv)
        wq, sw = (host(t) for t in layer.qkv)
        assert_bitwise(host(qkv).view(np.uint32), L.linear_w4a8(host(codes), host(scales), wq, sw, 0, F.EXCESS8).view(np.uint32),
                       f"product {at}")
        qkv = qkv.view(-1, H + 2 * K, D)
        q = both.append(pages, starts, have, qkv[:, H:H + K], qkv[:, H + K:], qkv[:, :H], cs, layer.gain_k, layer.gain_q, 1e-6)
        y = q4.q8_attention(q, both.cache, torch.from_numpy(pages).to(DEV), i32(starts), i32(have))
        check_attention(y, q, both.pool, pages, starts, have, np.float32(D ** -0.5), what=f"attention {at}")
    assert have == final


def serve(layer, x, cache, pages, new, have):
    starts = i32(np.concatenate([[0], np.cumsum(new)]))
    step = getattr(layer, "step", None) or layer.served
    return step(x, cache, pages, starts, i32(have))


@pytest.mark.parametrize("name,t", [("w4a8_decoder_layer", torch.float32), ("mx_decoder_layer", torch.bfloat16)])
def test_requests_do_not_see_each_other(name, t):
    """A request's cache holds the same alone and behind another, beside other pages; rows are finite."""
    layer, a, b = small(name), rows(7, 4).to(t), rows(21, 5).to(t)
    pages = torch.tensor([[3, 1], [0, 4]], dtype=torch.int32, device=DEV)
    one, two = (q4.q8_kv_cache(5, 2, 16, 64) for _ in range(2))
    y = serve(layer, torch.cat((a, b)), one, pages, [7, 21], [7, 21])
    alone = serve(layer, b, two, pages[1:], [21], [21])
    for s, u in zip(one, two):
        assert torch.equal(s[[0, 4]], u[[0, 4]])
    assert torch.isfinite(y).all() and torch.isfinite(alone).all()


def test_tokens_of_a_replayed_graph():
    """The captured step with lengths that move on the device against the same steps call by call, bit for bit."""
    layer = small()
    pages = torch.tensor([[3, 1, 6], [0, 4, 2]], dtype=torch.int32, device=DEV)
    prompt, z0 = rows(9 + 30, 6), rows(2, 7)
    ones = i32([0, 1, 2])

    def start():
        cache = q4.q8_kv_cache(7, 2, 16, 64)
        serve(layer, prompt, cache, pages, [9, 30], [9, 30])
        return cache, i32([9, 30]), z0.clone()

    cache, have, z = start()
    want = []
    for _ in range(6):
        have.add_(1)
        z = layer.step(z, cache, pages, ones, have)
        want.append(z.clone())
    g_cache, g_have, g_z = start()

    def token():
        g_have.add_(1)
        g_z.copy_(layer.step(g_z, g_cache, pages, ones, g_have))

    token()                                    # warm, and the first token
    assert torch.equal(g_z, want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    for i in range(1, 6):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g_z, want[i]), i
        other, n, y = start()                  # eager work of the same kind in between
        assert torch.equal(layer.step(y, other, pages, ones, n.add_(1)), want[0])
    for s, u in zip(cache, g_cache):
        assert torch.equal(s, u)
    assert g_have.tolist() == [15, 36]


@pytest.mark.parametrize("name", ["w4a8_decoder_layer", "mx_decoder_layer"])
def test_examples_run(name):
    example(name).main()

"""Appends and reads of so many rows that a workgroup has more than one set of
heads: the same bits as each head by itself, where it has one."""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
from tests.gpu_util import DEV, assert_bitwise, dev, host
from tests.test_gpu_kv_cache import TORCH, i32, new_pages, table

pytestmark = pytest.mark.gpu


def sets_of_a_workgroup(T, N, H, D):
    """Sets of key heads and query heads a workgroup has, for key or query heads H."""
    lanes = 1
    while 16 * lanes < D:
        lanes *= 2
    at_once, tokens = 16 // lanes, 256 // lanes
    sets = -(-H // at_once)
    share = lambda n, most: max(1, min(n // 1024, most))
    return share((T // 16 + 2 * N) * sets, min(sets, 8)), share(-(-T // tokens) * H, min(H, 8))


# lengths with the new tokens, new tokens: most sequences begin inside a block
RAGGED = ([3100, 2807, 16, 3011, 2999, 49], [3005, 2790, 3, 3000, 2990, 33])


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["halves", "neighbours", "plain"])
@pytest.mark.parametrize("H,Hq,D,R", [(7, 14, 256, 256), (5, 10, 128, 128), (7, 7, 256, 100), (5, 10, 128, 42),
                                      (9, 9, 80, 80), (33, 35, 64, 64), (18, 18, 96, 64)])
def test_sets_of_heads(H, Hq, D, R, how, xt):
    lengths, new = RAGGED
    T, N, page = sum(new), len(new), 32
    keys, queries = sets_of_a_workgroup(T, N, H, D)[0], sets_of_a_workgroup(T, N, Hq, D)[1]
    assert keys > 1 and queries > 1 and sets_of_a_workgroup(T, N, 1, D) == (1, 1)
    rng = np.random.default_rng(D + H)
    pages, P = new_pages(rng, lengths, page)
    gen = torch.Generator(DEV).manual_seed(H)
    code = [torch.randint(-127, 128, s, dtype=torch.int8, device=DEV, generator=gen)
            for s in ((P, H, 2, D // 16, 16, 16), (P, H, 2, D, 16))]
    byte = [torch.randint(112, 124, (P, H, 2), dtype=torch.uint8, device=DEV, generator=gen) for _ in range(2)]
    cache = q4.KVCache(*code, *byte)
    alone = [q4.KVCache(*(t[:, h:h + 1].contiguous() for t in cache)) for h in range(H)]
    qkv = (torch.randn(T, (Hq + 2 * H) * D, device=DEV, generator=gen)).to(TORCH[xt])
    q, k, v = (t.view(T, -1, D) for t in qkv.split([Hq * D, H * D, H * D], 1))
    gk, gq = (1 + 0.2 * torch.randn(D, device=DEV, generator=gen) for _ in range(2))
    cs = None if how == "plain" else dev(table(max(lengths), R))
    where = dev(pages), i32(np.concatenate([[0], np.cumsum(new)])), i32(lengths)
    rest = cs, gk, gq, 1e-6, "halves" if how == "plain" else how
    out = q4.q8_kv_append(cache, *where, k, v, q, *rest)
    for h in range(max(H, Hq)):
        hk, hq = h % H, h % Hq
        scratch = alone[hk] if h < H else q4.KVCache(*(t[:, hk:hk + 1].contiguous() for t in cache))
        one = q4.q8_kv_append(scratch, *where, k[:, hk:hk + 1], v[:, hk:hk + 1], q[:, hq:hq + 1], *rest)
        if h < Hq:
            assert_bitwise(host(out[:, h]), host(one[:, 0]), f"query head {h}")
        if h < H:
            for a, b, name in zip(cache, alone[h], ("k", "v", "k_scale", "v_scale")):
                assert_bitwise(host(a[:, h]), host(b[:, 0]), f"{name}, head {h}")
    for dtype in ("bf16", "f32"):
        ko, vo = q4.q8_kv_read(cache, *where, T, dtype)
        for h in range(H):
            for got, want, name in zip((ko, vo), q4.q8_kv_read(alone[h], *where, T, dtype), ("keys", "values")):
                assert_bitwise(host(got[:, h]), host(want[:, 0]), f"read {name}, head {h}, {dtype}")

"""What pins oracle/serving.py on the CPU: closed forms and brute force."""
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle.serving as S


def test_scale_byte_is_the_smallest_power():
    for top in (1.0, 127.0, 127.0000001, 126.9, 254.0, 1e-30, 2.0 ** -120, 2.0 ** -149, 3e38, 0.0):
        b = S.scale_byte(top)
        assert Fraction(top) <= 127 * Fraction(2) ** (b - 127)
        assert b == 0 or Fraction(top) > 127 * Fraction(2) ** (b - 128)
    assert S.scale_byte(127.0) == 127 and S.scale_byte(math.nextafter(127.0, 128.0)) == 128
    assert S.scale_byte(math.inf) == S.scale_byte(math.nan) == 255


def test_rmsnorm_codes_are_the_quotients():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 50)).astype(np.float32)
    g = rng.standard_normal(50).astype(np.float32)
    codes, scales, h = S.rmsnorm_rows(x, None, g, 1e-6)
    for m in range(3):
        u = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(x[m], g)]
        top = max(abs(v) for v in u)
        assert [round(127 * v / top) for v in u] == codes[m].tolist()      # round: ties to even
        y = x[m].astype(np.float64) / np.sqrt(np.mean(x[m].astype(np.float64) ** 2) + 1e-6) * g
        assert np.abs(codes[m] * scales[m] - y).max() <= 0.5000001 * scales[m]
    codes, scales, _ = S.rmsnorm_rows(np.zeros((1, 4)), None, None, 1e-6)
    assert not codes.any() and scales[0] == 0
    assert np.isnan(S.rmsnorm_rows(np.array([[1, np.inf]]), None, None, 0.0)[1][0])


def test_blocks_lie_as_described():
    pool = S.Pool(2, 1, 16, 32)
    x = {n: np.arange(16 * 32).reshape(16, 1, 32) % 100 - 50.0 for n in "kv"}
    pool.append(np.array([[1]]), [0, 16], [16], x)
    assert pool.ks[1, 0, 0] == pool.vs[1, 0, 0] == 127 - 1       # 50 <= 127 / 2
    for t in (0, 3, 15):
        for c in (0, 17, 31):
            v = 2 * ((t * 32 + c) % 100 - 50)
            assert pool.k[1, 0, 0, c // 16, t, c % 16] == v and pool.v[1, 0, 0, c, t] == v
    assert not pool.k[0].any()
    assert np.array_equal(pool.head("k", np.array([[1]]), 0, 0, 16), x["k"][:, 0])


def test_append_by_tokens_grows_the_scale_and_rounds_again():
    pool = S.Pool(1, 1, 16, 16)
    pages = np.array([[0]])
    row = lambda v: {n: np.full((1, 1, 16), v) for n in "kv"}
    pool.append(pages, [0, 1], [1], row(3.0))                # 96 / 32
    assert pool.ks[0, 0, 0] == 127 - 5 and pool.codes("k", 0, 0, 0)[0, 0] == 96
    pool.append(pages, [0, 1], [2], row(0.1))                # the scale stays
    assert pool.ks[0, 0, 0] == 127 - 5 and pool.codes("k", 0, 0, 0)[1, 0] == 3
    pool.append(pages, [0, 1], [3], row(100.0))              # 2^0: 3.0 -> 3, 3 / 32 -> 0
    assert pool.ks[0, 0, 0] == 127 and pool.codes("k", 0, 0, 0)[:3, 0].tolist() == [3, 0, 100]
    pool.append(pages, [0, 1], [4], row(np.nan))
    assert pool.ks[0, 0, 0] == 255 and np.isnan(pool.value("v", pages, 0, 0, 1)).all()
    pool.append(pages, [0, 1], [1], row(1.0))                # its first token again: a new block
    assert pool.ks[0, 0, 0] == 127 - 6


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (1, 50)])
def test_attention_by_brute_force(window, sinks):
    rng = np.random.default_rng(2)
    pool = S.Pool(6, 2, 16, 16)
    pages = np.array([[4, 1], [0, -1], [5, 3]])
    starts, lengths = [0, 2, 3, 5], [20, 7, 32]
    for i, n in enumerate(lengths):
        pool.append(pages[i:i + 1], [0, n], [n], {c: rng.standard_normal((n, 2, 16)) for c in "kv"})
    q = rng.standard_normal((6, 4, 16))
    y, size, terms, flat, peak = S.attention(q, pool, pages, starts, lengths, 0.3, window, sinks)
    assert np.isnan(y[5]).all()                              # behind the last sequence
    for row, i, pos in ((0, 0, 18), (1, 0, 19), (2, 1, 6), (3, 2, 30), (4, 2, 31)):
        for g in range(4):
            num, den = np.zeros(16), 0.0
            for j in range(pos + 1):
                if window and j <= pos - window and j >= sinks:
                    continue
                w = math.exp(0.3 * float(q[row, g] @ pool.value("k", pages, i, g // 2, j)))
                num, den = num + w * pool.value("v", pages, i, g // 2, j), den + w
            assert np.abs(y[row, g] - num / den).max() < 1e-12
            assert (np.abs(y[row, g]) <= size[row, g] + 1e-12).all() and 0 < terms[row, g] <= flat[row, g] + 1e-12
            assert 0 < peak[row, g] < 127 * 2.0 ** (int(pool.vs.max()) - 127)


def test_rows_without_keys_are_zero():
    pool = S.Pool(1, 1, 16, 16)
    y, size, _, _, _ = S.attention(np.ones((3, 1, 16)), pool, np.array([[0]]), [0, 3], [1], 1.0)
    assert not y[:2].any() and not size[:2].any()            # positions -2, -1

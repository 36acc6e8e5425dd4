"""Attention over the paged 8-bit cache where scores are so large that f32 holds
no fractions of them: one key has all of a row's weight, so the result is its
value, off by the weight's rounding (2^-11 of itself with bf16 in and out, 2^-22
otherwise), a few roundings of f32 and the result's own.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.serving as S
from tests.gpu_util import DEV, dev
from tests.test_gpu_attention import PATHS, TYPES, on_gpu
from tests.test_gpu_kv_cache import TORCH, f64, i32

pytestmark = pytest.mark.gpu
L, D, H, HQ = 131, 32, 1, 2


@pytest.fixture(autouse=True)
def _auto_path():
    yield
    q4.q4_set_path("auto")


def pool_of(rng, bytes_of_values):
    """Keys that differ in column 0 alone, no two of them alike; values of every size that the bytes give."""
    pool = S.Pool(9, H, 16, D)
    pages = rng.permutation(9).astype(np.int32)[None]
    pool.ks[...] = 127
    column = rng.permutation(np.arange(-90, 91))[:144]
    for b in range(9):
        pool.k[pages[0, b], 0, 0, 0, :, 0] = column[16 * b:16 * b + 16]
    pool.v[...] = rng.integers(-127, 128, pool.v.shape)
    pool.vs[...] = rng.choice(bytes_of_values, pool.vs.shape)
    return pool, pages


def compare(y, q, pool, pages, n, scale, window, what):
    ref = S.attention(f64(q), pool, pages, [0, n], [L], scale, window)[0]
    coarse = q.dtype == torch.bfloat16 and y.dtype == torch.bfloat16
    tol = ((2.0 ** -11 if coarse else 2.0 ** -22) + 16 * 2.0 ** -24 + (2.0 ** -8 if y.dtype == torch.bfloat16 else 0)) * np.abs(ref)
    got = f64(y)
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), [(got[tuple(b)], ref[tuple(b)]) for b in bad[:3]])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("window", [0, 1, 40])
def test_one_key_has_all_of_the_weight(window, xt, yt, path):
    """Scores times log2(e) from 2^18 to 2^40, of both signs; with a window of 1 each row sees one key."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(window)
    n = 50
    for of_values in ([127], [126], [120, 121, 122, 123], [90, 127, 150]):
        pool, pages = pool_of(rng, of_values)
        for power in list(range(18, 34)) + [40]:
            q = np.zeros((n, HQ, D), np.float32)
            q[:, :, 0] = 2.0 ** (power - 7) * rng.uniform(1, 2, (n, HQ)) * rng.choice([-1, 1], (n, HQ))
            q = dev(q).to(TORCH[xt])
            y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, n]), i32([L]), 0.731, window, dtype=yt)
            compare(y, q, pool, pages, n, np.float32(0.731), window, (of_values, power))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt,yt", TYPES)
def test_rows_of_all_sizes_side_by_side(xt, yt, path):
    """A row's size does not touch its neighbours, which share its instructions: some with scores of 2^35, some with
    scores of a few units."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(1)
    n = 60
    pool, pages = pool_of(rng, [125, 126, 127])
    q = np.zeros((n, HQ, D), np.float32)
    small = rng.random((n, HQ)) < 0.4
    q[:, :, 0] = np.where(small, rng.uniform(-0.05, 0.05, (n, HQ)), 2.0 ** rng.uniform(12, 28, (n, HQ)) * rng.choice([-1, 1], (n, HQ)))
    q = dev(q).to(TORCH[xt])
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, n]), i32([L]), 1.0, dtype=yt)
    ref, size, terms, flat, peak = S.attention(f64(q), pool, pages, [0, n], [L], 1.0)
    coarse = xt == yt == "bf16"
    h = 2.0 ** -24
    # scores of large rows decide nothing but which key is the largest
    score = np.where(terms < 2.0 ** 10, (D + 12) * h * terms + 2.0 ** -22 * flat, 0)
    weight = score + (2.0 ** -11 if coarse else 2.0 ** -22) + 4 * h
    tol = (2 * weight + (L / 8 + 64) * h)[..., None] * size + (L * (2.0 ** -33 if coarse else 2.0 ** -34) * peak)[..., None]
    tol = tol + (2.0 ** -8 if yt == "bf16" else 0) * np.abs(ref)
    got = f64(y)
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), [(got[tuple(b)], ref[tuple(b)], q[b[0], b[1], 0].item()) for b in bad[:3]])


@pytest.mark.parametrize("xt,yt", TYPES)
def test_joined_splits(xt, yt):
    """The shares of a sequence's keys have largest scores that differ by far, and are joined."""
    q4.q4_set_path("gemv")
    rng = np.random.default_rng(2)
    pool, pages = pool_of(rng, [100, 127, 128])
    for power in (18, 24, 28, 31, 36):
        q = np.zeros((3, HQ, D), np.float32)
        q[:, :, 0] = 2.0 ** (power - 7) * rng.uniform(1, 2, (3, HQ)) * rng.choice([-1, 1], (3, HQ))
        q = dev(q).to(TORCH[xt])
        for max_len in (1024, 5000, 10 ** 6):
            y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, 3]), i32([L]), 0.731, max_len=max_len, dtype=yt)
            compare(y, q, pool, pages, 3, np.float32(0.731), 0, (power, max_len))

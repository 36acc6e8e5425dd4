"""Attention over the paged 8-bit cache on the GPU against the float64 oracle.

What a result may be off by, in units of `size`, the weighted mean of |v|: a
weight is off by twice (itself and the sum) what its score is off by, its
rounding and the exponential's; then the sums' roundings.  A score is a sum of D
products (D + 8 half steps, 2^-24, of sum |q k| scale) and the factors of the scale
(4 half steps more), of queries rounded to 2^-22 of the row's
largest (f32: two halves) or exact to 2^-25 of it (bf16).  Weights have half a
step of 2^-11 (bf16 in and out) or 2^-22, the exponential two steps of f32; n
keys are summed in chains of n / 16 and some joints.  Halves end at steps of
2^-24, so a weight times its values' scale is off by half of that where the
largest such product is 2^8 or more (2^9 with two halves): n times 2^-33 (2^-34)
of `peak`, the largest, in all.  bf16 results are rounded once more, 2^-8 of
themselves.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.serving as S
from tests.gpu_util import DEV, assert_bitwise, dev, host
from tests.test_gpu_kv_cache import TORCH, f64, i32, new_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _auto_path():
    q4.q4_set_path("auto")
    yield
    q4.q4_set_path("auto")


def random_pool(rng, P, H, page, D, low=118, high=123):
    pool = S.Pool(P, H, page, D)
    pool.k[...] = np.clip(np.rint(40 * rng.standard_normal(pool.k.shape)), -127, 127)
    pool.v[...] = np.clip(np.rint(40 * rng.standard_normal(pool.v.shape)), -127, 127)
    pool.ks[...] = rng.integers(low, high, pool.ks.shape)
    pool.vs[...] = rng.integers(low, high, pool.vs.shape)
    return pool


def on_gpu(pool):
    return q4.KVCache(*(dev(a) for a in (pool.k, pool.v, pool.ks, pool.vs)))


def check(y, q, pool, pages, starts, lengths, scale, window=0, sinks=0, what=""):
    q64 = f64(q)
    ref, size, terms, flat, peak = S.attention(q64, pool, pages, starts, lengths, scale, window, sinks)
    coarse = q.dtype == torch.bfloat16 and y.dtype == torch.bfloat16
    D, n = q.shape[2], max(list(lengths) + [1])
    h = 2.0 ** -24
    score = (D + 12) * h * terms + (2.0 ** -22 if q.dtype == torch.float32 else 2.0 ** -25) * flat
    weight = score + (2.0 ** -11 if coarse else 2.0 ** -22) + 4 * h
    tol = (2 * weight + (n / 8 + 64) * h)[..., None] * size + (n * (2.0 ** -33 if coarse else 2.0 ** -34) * peak)[..., None]
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    got = f64(y)
    rows = [r for r, _, _ in S.rows_of(starts, lengths, len(q64))]
    g, r, t = got[rows], ref[rows], tol[rows]
    bad = np.argwhere(~((np.abs(g - r) <= t + 1e-40) | (np.isnan(g) & np.isnan(r))))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), [(g[tuple(b)], r[tuple(b)], t[tuple(b)]) for b in bad[:3]])


def run(rng, lengths, new, H, Hq, D, page, window=0, sinks=0, xt="bf16", yt=None, what="", **kw):
    pages, P = new_pages(rng, lengths, page)
    pool = random_pool(rng, P, H, page, D)
    T = sum(new)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = dev((3 * rng.standard_normal((T, Hq, D))).astype(np.float32)).to(TORCH[xt])
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths), window=window, sinks=sinks, dtype=yt, **kw)
    assert y.shape == q.shape and y.dtype == TORCH[yt or xt] and y.is_contiguous()
    check(y, q, pool, pages, starts, lengths, np.float32(D ** -0.5), window, sinks, what)
    return y


PATHS = ["gemv", "tiled"]
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 160, 176, 192, 208, 224, 240, 256])
def test_head_sizes(D, xt, yt, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(D)
    run(rng, [70, 1, 45], [1, 1, 20], 2, 6, D, 16, xt=xt, yt=yt, what="mixed")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt,yt", TYPES[:2])
@pytest.mark.parametrize("lengths,new", [([1], [1]), ([15], [15]), ([16], [1]), ([17], [17]), ([31, 32, 33], [1, 32, 2]),
                                         ([64, 65], [64, 65]), ([200, 0, 3], [1, 0, 0]), ([130], [129]),
                                         ([257, 40], [257, 3]), ([700], [300])])
def test_lengths(lengths, new, xt, yt, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(sum(lengths) + sum(new))
    run(rng, lengths, new, 2, 4, 64, 32, xt=xt, yt=yt)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("H,Hq", [(1, 1), (3, 3), (1, 5), (2, 14), (1, 16), (1, 33), (1, 71), (4, 32)])
def test_shared_heads(H, Hq, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(Hq)
    run(rng, [90, 33], [9, 1], H, Hq, 64, 16)
    run(rng, [90, 133], [1, 1], H, Hq, 64, 16, xt="f32")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("page", [16, 32, 64, 1024])
def test_page_sizes(page, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(page)
    run(rng, [150, 77], [3, 60], 2, 4, 128, page)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (16, 4), (17, 16), (33, 17), (64, 40), (100, 0),
                                          (10 ** 12, 3), (20, 10 ** 12)])
def test_windows_and_sinks(window, sinks, xt, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(window % 1000 + sinks % 1000)
    run(rng, [300, 20, 150], [1, 20, 140], 2, 4, 64, 16, window, sinks, xt=xt)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("max_len", [0, 100, 5000, None, 2 ** 31 - 1])
def test_splits_of_the_keys(max_len, xt):
    """One workgroup or several to a sequence's keys: with a bound below, at and above the lengths."""
    rng = np.random.default_rng(5)
    kw = {} if max_len is None else {"max_len": max_len}
    run(rng, [5000, 1, 300, 2049], [1, 1, 1, 1], 2, 8, 64, 64, xt=xt, **kw)
    run(rng, [4000], [1], 1, 3, 128, 16, 1500, 20, xt=xt, **kw)
    run(rng, [3000], [5], 1, 4, 96, 32, xt=xt, **kw)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_scores_of_all_sizes(xt, path):
    """Peaked and flat weights, large and tiny queries, negative scale, blocks whose scales differ by far."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(6)
    lengths, new = [260, 90], [3, 90]
    starts = [0, 3, 93]
    pages, P = new_pages(rng, lengths, 16)
    for low, high, size in ((118, 123, 1.0), (127, 128, 4.0), (100, 130, 1.0), (60, 61, 2.0 ** 60), (118, 123, 0.0),
                            (200, 201, 2.0 ** -80)):
        pool = random_pool(rng, P, 2, 16, 64, low, high)
        q = dev((size * rng.standard_normal((93, 4, 64))).astype(np.float32)).to(TORCH[xt])
        for scale in (0.125, -0.125, 0.0):
            y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths), scale)
            check(y, q, pool, pages, starts, lengths, scale, what=(low, high, size, scale))


@pytest.mark.parametrize("path", PATHS)
def test_values_of_extreme_scales(path):
    """Value blocks under the smallest scales beside each other and beside large ones."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(16)
    pages, P = new_pages(rng, [1100], 16)
    for low, high in ((0, 3), (20, 40), (225, 230)):
        pool = random_pool(rng, P, 1, 16, 32)
        pool.vs[...] = rng.integers(low, high, pool.vs.shape)
        q = dev(rng.standard_normal((40, 1, 32)).astype(np.float32))
        y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, 40]), i32([1100]))
        ref = S.attention(f64(q), pool, pages, [0, 40], [1100], np.float32(32 ** -0.5))
        tol = (2 * (2.0 ** -24 * 44 * ref[2] + 2.0 ** -22 * ref[3] + 2.0 ** -21) + 202 * 2.0 ** -24)[..., None] * ref[1]
        tol = tol + (1100 * 2.0 ** -34 * ref[4])[..., None]
        assert np.all(np.abs(f64(y) - ref[0]) <= tol + 2.0 ** -148), (low, high)
    # blocks of zeros under scale 0 in front of and between others
    pool = random_pool(rng, P, 1, 16, 32)
    zero = rng.random(pool.vs.shape) < 0.7
    pool.vs[zero] = 0
    pool.v[zero] = 0
    q = dev(rng.standard_normal((40, 1, 32)).astype(np.float32)).bfloat16()
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, 40]), i32([1100]))
    check(y, q, pool, pages, [0, 40], [1100], np.float32(32 ** -0.5), what="zero blocks")


@pytest.mark.parametrize("path", PATHS)
def test_values_of_unlike_scales_and_weights(path):
    """A key with nearly all of the weight and values 2^-40 of another's: the smaller products count for what they are."""
    q4.q4_set_path(path)
    pool = S.Pool(4, 1, 16, 16)
    pages = np.array([[3, 1, 0, 2]], np.int32)
    x = np.zeros((64, 1, 16))
    x[5, 0, 0], x[40, 0, 0] = 1.0, -4.0
    v = np.full((64, 1, 16), 2.0 ** -60)
    v[5], v[40] = 1.0, 2.0 ** 40
    pool.append(pages, [0, 64], [64], {"k": x, "v": v})
    for size in (5.0, 8.0, 20.0):
        q = torch.zeros(64, 1, 16, device=DEV)
        q[:, 0, 0] = size
        for t in (q, q.bfloat16()):
            y = q4.q8_attention(t, on_gpu(pool), dev(pages), i32([0, 64]), i32([64]), 1.0)
            check(y, t, pool, pages, [0, 64], [64], 1.0, what=size)
            # the row at 20 does not see the large values; the one at 45 does
            assert abs(f64(y)[20, 0, 0] - 1.0 / (1 + 20 * np.exp(-size))) < 2.0 ** -6


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_what_a_row_does_not_see_does_not_touch_it(xt, path):
    """NaN blocks, bad pages and extreme codes behind the sequence, ahead of the row and outside its window."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(7)
    lengths, new, D = [100, 75], [6, 75], 64
    starts = [0, 6, 81]
    pages = np.array([[3, 0, 7, 5, 1, 9, 11, -1], [2, 4, 6, 8, 10, 2 ** 30, -5, 99]], np.int32)
    q = dev(rng.standard_normal((81, 4, D)).astype(np.float32)).to(TORCH[xt])
    pool = random_pool(rng, 12, 2, 16, D)
    for a, n in ((pool.ks, 4), (pool.vs, 4)):
        a[11, :, 0] = 255                       # tokens 96 .. 111 of the first: only rows at 96 .. 99 see them
        a[10, 1, 0] = 255                       # tokens 64 .. 79 of the second, one head
        a[0, :, 0] = 255                        # tokens 16 .. 31 of the first: outside a window of 40
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths), 0.125, 40, 5)
    check(y, q, pool, pages, starts, lengths, 0.125, 40, 5)
    got = f64(y)
    assert np.isfinite(got[:2]).all() and np.isnan(got[2:6]).all()          # positions 94, 95 | 96 ..
    assert np.isfinite(got[6:70]).all() and np.isnan(got[70:, 2:]).all() and np.isfinite(got[70:, :2]).all()
    # a page that is not there: NaN for who sees it
    lengths2 = [100, 85]
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths2), 0.125, 5, 0)
    check(y, q, pool, pages, starts, lengths2, 0.125, 5, 0)
    got = f64(y)
    assert np.isfinite(got[6:60]).all() and np.isnan(got[76:81]).all()      # positions 80 .. 84
    # and past the table
    short = pages[:, :4].copy()
    y = q4.q8_attention(q, on_gpu(pool), dev(short), i32(starts), i32(lengths), 0.125, 8, 0)
    check(y, q, pool, short, starts, lengths, 0.125, 8, 0)


@pytest.mark.parametrize("path", PATHS)
def test_non_finite_queries(path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(8)
    pages, P = new_pages(rng, [50], 16)
    pool = random_pool(rng, P, 1, 16, 32)
    q = dev(rng.standard_normal((20, 3, 32)).astype(np.float32))
    q[3, 1, 5], q[7, 0, 31], q[7, 2, 0] = float("nan"), float("inf"), float("-inf")
    for t in (q, q.bfloat16()):
        got = f64(q4.q8_attention(t, on_gpu(pool), dev(pages), i32([0, 20]), i32([50])))
        nan = np.isnan(got).all(axis=2)
        assert np.array_equal(nan, np.isnan(got).any(axis=2))
        assert np.array_equal(np.argwhere(nan), [[3, 1], [7, 0], [7, 2]])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_rows_without_keys_and_rows_of_nobody(xt, path):
    q4.q4_set_path(path)
    rng = np.random.default_rng(9)
    pool = random_pool(rng, 5, 1, 16, 32)
    pages = np.array([[4], [2], [0]], np.int32)
    starts, lengths = [1, 6, 6, 9], [2, 0, 0]       # 5 rows for 2 tokens; none; 3 rows without tokens
    q = dev(rng.standard_normal((11, 2, 32)).astype(np.float32)).to(TORCH[xt])
    for max_len in (16, 10 ** 6):                   # one split, many
        y = torch.full((11, 2, 32), 77.0, device=DEV).to(q.dtype)
        q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths), max_len=max_len, y=y)
        check(y, q, pool, pages, starts, lengths, np.float32(32 ** -0.5))
        got = f64(y)
        assert (got[[0, 9, 10]] == 77).all() and not got[1:4].any() and not got[6:9].any() and got[4:6].all()


@pytest.mark.parametrize("path", PATHS)
def test_layouts_streams_and_workspaces(path):
    """A slice of a fused projection and head-major rows at odd addresses; given outputs and workspaces; a side stream."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(10)
    H, Hq, D, T = 2, 4, 48, 30
    lengths, starts = [600, 400], [0, 29, 30]
    pages, P = new_pages(rng, lengths, 16)
    pool = random_pool(rng, P, H, 16, D)
    cache, p, st, ln = on_gpu(pool), dev(pages), i32(starts), i32(lengths)
    fused = dev(rng.standard_normal((T, (Hq + 2 * H) * D)).astype(np.float32)).bfloat16()
    a = fused[:, :Hq * D].view(T, Hq, D)
    b = fused.view(-1)[1:1 + T * Hq * D].view(Hq, T, D).transpose(0, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for q in (a, b):
            y = torch.empty(T, Hq, D, dtype=torch.float32, device=DEV)
            need = q4.q8_attention_workspace(T, 2, Hq, H, D, 600)
            ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
            out = q4.q8_attention(q, cache, p, st, ln, max_len=600, dtype="f32", ws=ws, y=y)
            assert out.data_ptr() == y.data_ptr()
            check(y, q, pool, pages, starts, lengths, np.float32(D ** -0.5))
            assert_bitwise(host(q4.q8_attention(q.contiguous(), cache, p, st, ln, max_len=600, dtype="f32")), host(y), "again")
    side.synchronize()


def test_a_large_pool_and_a_long_context():
    """Blocks past 2^32 bytes, 200000 tokens on pages from all over the pool."""
    H, D, page, P = 8, 128, 64, 70000
    gen = torch.Generator(DEV).manual_seed(1)
    k = torch.randint(-127, 128, (P, H, 4, 8, 16, 16), dtype=torch.int8, device=DEV, generator=gen)
    v = torch.randint(-127, 128, (P, H, 4, D, 16), dtype=torch.int8, device=DEV, generator=gen)
    ks, vs = (torch.randint(117, 121, (P, H, 4), dtype=torch.uint8, device=DEV, generator=gen) for _ in range(2))
    L = 200000
    pages = torch.randperm(P, device=DEV, generator=gen)[:L // page + 1].int()[None]
    pages[0, -1] = P - 1
    q = torch.randn(1, 8, D, device=DEV, generator=gen)
    y = q4.q8_attention(q, q4.KVCache(k, v, ks, vs), pages.contiguous(), i32([0, 1]), i32([L]))
    pg = pages[0].long()
    for h in range(H):
        K = k[pg, h].double() * torch.exp2(ks[pg, h].double() - 127)[..., None, None, None]
        K = K.permute(0, 1, 3, 2, 4).reshape(-1, D)[:L]
        V = (v[pg, h].double() * torch.exp2(vs[pg, h].double() - 127)[..., None, None]).transpose(2, 3).reshape(-1, D)[:L]
        x = K @ q[0, h].double() * D ** -0.5
        w = torch.softmax(x, 0)
        terms = float((K.abs() @ q[0, h].double().abs()).max()) * D ** -0.5
        flat = float(q[0, h].abs().max() * K.abs().sum(1).max()) * D ** -0.5
        tol = 2 * ((D + 12) * 2.0 ** -24 * terms + 2.0 ** -22 * flat + 2.0 ** -21) + (L / 8 + 64) * 2.0 ** -24
        err = (y[0, h].double() - w @ V).abs()
        assert bool((err <= tol * (w @ V.abs())).all()), h


def test_many_sequences():
    rng = np.random.default_rng(11)
    new = rng.integers(0, 4, 200)
    lengths = (new + rng.integers(0, 30, 200)).tolist()
    run(rng, lengths, new.tolist(), 1, 2, 32, 16)
    run(rng, [5] * 5000, [1] * 5000, 1, 1, 16, 16)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_the_same_call_gives_the_same_bits(xt):
    rng = np.random.default_rng(12)
    pages, P = new_pages(rng, [3000, 100], 16)
    cache = on_gpu(random_pool(rng, P, 2, 16, 64))
    q = dev(rng.standard_normal((80, 4, 64)).astype(np.float32)).to(TORCH[xt])
    for starts in ([0, 1, 2], [0, 40, 80]):
        a = [host(q4.q8_attention(q, cache, dev(pages), i32(starts), i32([3000, 100]))[:starts[-1]]) for _ in range(3)]
        assert_bitwise(a[1], a[0], "twice")
        assert_bitwise(a[2], a[0], "thrice")


def test_graph_replays():
    """Two captured graphs of one cache, a decode step and a chunk, replayed in turn with eager calls between."""
    rng = np.random.default_rng(13)
    N, H, Hq, D = 3, 2, 4, 64
    pages, P = new_pages(rng, [4000] * N, 64)
    pool = random_pool(rng, P, H, 64, D)
    cache, p = on_gpu(pool), dev(pages)
    lengths = i32([1] * N)
    one, many = i32(range(N + 1)), i32([0, 20, 20, 45])
    q1 = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device=DEV)
    q2 = torch.zeros(45, Hq, D, device=DEV)

    def step():
        return q4.q8_attention(q1, cache, p, one, lengths)

    def chunk():
        return q4.q8_attention(q2, cache, p, many, lengths, window=500, sinks=4)

    step(), chunk()
    graphs, outs = [], []
    for f in (step, chunk):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    for seed in range(4):
        gen = torch.Generator(DEV).manual_seed(seed)
        q1.copy_(torch.randn(q1.shape, device=DEV, generator=gen))
        q2.copy_(torch.randn(q2.shape, device=DEV, generator=gen))
        lengths.copy_(torch.randint(25, 4000, (N,), device=DEV, generator=gen))
        for g in graphs:
            g.replay()
        got = [host(o) for o in outs]
        assert_bitwise(got[0], host(step()), f"step {seed}")
        assert_bitwise(got[1], host(chunk()), f"chunk {seed}")
        check(step(), q1, pool, pages, range(N + 1), host(lengths).tolist(), np.float32(D ** -0.5))


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own."""
    rng = np.random.default_rng(14)
    pages, P = new_pages(rng, [3000] * 2, 64)
    cache, p = on_gpu(random_pool(rng, P, 2, 64, 128)), dev(pages)
    qs = [dev(rng.standard_normal((2, 8, 128)).astype(np.float32)).bfloat16() for _ in range(2)]
    want = [host(q4.q8_attention(q, cache, p, i32([0, 1, 2]), i32([3000, 2000]))) for q in qs]
    st, ln = i32([0, 1, 2]), i32([3000, 2000])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(q4.q8_attention(q, cache, p, st, ln))
    for i, y in enumerate(got):
        assert_bitwise(host(y), want[i % 2], f"call {i}")


def test_refused():
    c = q4.q8_kv_cache(3, 2, 16, 32)
    pages, starts, lengths = i32([[0, 1]]), i32([0, 2]), i32([2])
    q = torch.zeros(2, 4, 32, device=DEV)
    for bad in (lambda: q4.q8_attention(q[..., :16], c, pages, starts, lengths),
                lambda: q4.q8_attention(q.transpose(1, 2), c, pages, starts, lengths),
                lambda: q4.q8_attention(q[0], c, pages, starts, lengths),
                lambda: q4.q8_attention(q, c, pages[0], starts, lengths),
                lambda: q4.q8_attention(q, c, pages, starts, lengths, y=q[:1].clone())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q8_attention(q.half(), c, pages, starts, lengths),
                lambda: q4.q8_attention(q, c, pages.long(), starts, lengths),
                lambda: q4.q8_attention(q, c, pages, starts, lengths, dtype="bf16", y=q.clone()),
                lambda: q4.q8_attention(q, c, pages, starts, lengths, ws=np.zeros(9))):
        with pytest.raises(TypeError):
            bad()
    for bad, status in ((lambda: q4.q8_attention(q[:, :3], c, pages, starts, lengths), q4.ESHAPE),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, scale=float("inf")), q4.EINVAL),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, window=-1), q4.EINVAL),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, sinks=-1), q4.EINVAL),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, max_len=-1), q4.EINVAL),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, y=q), q4.EINVAL),
                        (lambda: q4.q8_attention(q, c, pages, starts, lengths, max_len=10 ** 6,
                                                 ws=torch.empty(256, dtype=torch.uint8, device=DEV)), q4.EINVAL)):
        with pytest.raises(q4.Q4Error) as e:
            bad()
        assert e.value.status == status
    assert q4.q8_attention(q[:0], c, pages, i32([0, 0]), lengths).shape == (0, 4, 32)
    assert q4.q8_attention(q[:, :0], c, pages, starts, lengths).shape == (2, 0, 32)


def test_both_paths_of_the_binding_agree(monkeypatch):
    rng = np.random.default_rng(15)
    pages, P = new_pages(rng, [900], 32)
    cache = on_gpu(random_pool(rng, P, 2, 32, 64))
    q = dev(rng.standard_normal((3, 4, 64)).astype(np.float32))
    args = (q, cache, dev(pages), i32([0, 3]), i32([900]), 0.1, 300, 5, 900, "bf16")
    a = q4.q8_attention(*args)
    monkeypatch.setattr(q4, "_DIRECT", q4._NoDirect())
    assert_bitwise(host(q4.q8_attention(*args)), host(a), "paths")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (8, 0), (8, 3), (30, 100), (8, 10 ** 9), (2 ** 31 - 1, 0), (2 ** 40, 2 ** 40)])
def test_lengths_past_the_table(window, sinks, xt, path):
    """Tokens that the table has no entry for are NaN to whoever sees them, without
    work that goes by the length; the next sequence does not notice."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(3)
    H, Hq, D, page, new = 2, 6, 64, 16, 150
    pages, P = new_pages(rng, [64, 60], page)
    pool = random_pool(rng, P, H, page, D)
    starts = [0, new, new + 2]
    q = dev((3 * rng.standard_normal((new + 2, Hq, D))).astype(np.float32)).to(TORCH[xt])
    for first in (75, 160, 64 + new, 2 ** 20, 2 ** 31 - 1):
        y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32([first, 60]), window=window, sinks=sinks)
        if first < 1000:
            check(y, q, pool, pages, starts, [first, 60], np.float32(D ** -0.5), window, sinks, first)
        else:
            assert torch.isnan(y[:new]).all()
            rest = q[new:].contiguous()
            own = q4.q8_attention(rest, on_gpu(pool), dev(pages[1:]), i32([0, 2]), i32([60]), window=window, sinks=sinks)
            check(own, rest, pool, pages[1:], [0, 2], [60], np.float32(D ** -0.5), window, sinks, "alone")
            check(y[new:], rest, pool, pages[1:], [0, 2], [60], np.float32(D ** -0.5), window, sinks, first)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 128, 144, 208, 256])
def test_joined_splits(D, xt, yt):
    """Four to 64 splits of every head size, rows that fill no workgroup of the join, in front of them
    and behind them rows of nobody; a workspace with the given bytes and no more."""
    rng = np.random.default_rng(D + 1)
    H, Hq, T, lengths, starts = 1, 3, 9, [1100, 0, 40], [2, 5, 5, 7]
    pages, P = new_pages(rng, lengths, 32)
    pool = random_pool(rng, P, H, 32, D)
    q = dev((3 * rng.standard_normal((T, Hq, D))).astype(np.float32)).to(TORCH[xt])
    for max_len in (1024, 1100, 5000, 10 ** 6):
        need = q4.q8_attention_workspace(T, 3, Hq, H, D, max_len)
        assert need > 0
        room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        room = room[-room.data_ptr() % 256:]
        y = torch.full((T, Hq, D), 77.0, dtype=TORCH[yt], device=DEV)
        q4.q8_attention(q, on_gpu(pool), dev(pages), i32(starts), i32(lengths), max_len=max_len, dtype=yt, ws=room[:need], y=y)
        check(y, q, pool, pages, starts, lengths, np.float32(D ** -0.5), what=max_len)
        assert (f64(y)[[0, 1, 7, 8]] == 77).all() and bool((room[need:] == 0xA5).all())


@pytest.mark.parametrize("xt,D,n,path,want", [
    ("bf16", 128, 1, "auto", "gemv"), ("bf16", 128, 2048, "auto", "tiled"), ("bf16", 144, 2048, "auto", "gemv"),
    ("f32", 64, 4096, "auto", "tiled"), ("f32", 96, 4096, "auto", "gemv"), ("bf16", 128, 2048, "gemv", "gemv"),
    ("bf16", 128, 3, "tiled", "tiled"), ("f32", 80, 3, "tiled", "gemv"), ("bf16", 128, 3, "generic", "gemv")])
def test_route(xt, D, n, path, want):
    """What is reported, and the first and last row against the oracle."""
    q4.q4_set_path(path)
    rng = np.random.default_rng(16)
    H, Hq = 8, 32
    pages, P = new_pages(rng, [n + 40], 64)
    pool = random_pool(rng, P, H, 64, D)
    q = dev((3 * rng.standard_normal((n, Hq, D))).astype(np.float32)).to(TORCH[xt])
    y = q4.q8_attention(q, on_gpu(pool), dev(pages), i32([0, n]), i32([n + 40]))
    assert q4.q4_last_path() == want
    for row in (0, n - 1):
        check(y[row:row + 1], q[row:row + 1], pool, pages, [0, 1], [40 + row + 1], np.float32(D ** -0.5), what=row)

"""The paged 8-bit cache on the GPU against the float64 oracle.

Codes and scale bytes are the oracle's, bit for bit: keys are computed in f64 on
both sides, and one next to a border by less than their roundings (2^-50 of
itself) does not occur in these inputs.  A query row carries at most D / 2 + 16
roundings of half a step (2^-24) of the magnitudes that it is the sum of, a bf16
one half a bf16 step (2^-8) of itself more.  Reading back is exact.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.serving as S
from tests.gpu_util import DEV, assert_bitwise, dev, host

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def table(P, R, base=10000.0):
    a = np.arange(P)[:, None] * base ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def new_pages(rng, lengths, page, spare=2):
    """Pages of sequences, in any order, with entries that mean nothing behind them -> (table, pages in all)."""
    used = [-(-n // page) for n in lengths]
    P = sum(used) + spare
    order = rng.permutation(P)
    width = max(used + [1])
    t = np.full((len(lengths), width), -7, np.int32)
    at = 0
    for i, n in enumerate(used):
        t[i, :n] = order[at:at + n]
        at += n
    return t, P


class Both:
    """A cache on the GPU and the oracle's."""

    def __init__(self, P, H, page, D, rng=None):
        self.pool = S.Pool(P, H, page, D)
        if rng is not None:                # what earlier sequences left
            self.pool.k[...] = rng.integers(-127, 128, self.pool.k.shape)
            self.pool.v[...] = rng.integers(-127, 128, self.pool.v.shape)
            self.pool.ks[...] = rng.integers(0, 256, self.pool.ks.shape)
            self.pool.vs[...] = rng.integers(0, 256, self.pool.vs.shape)
        self.cache = q4.KVCache(*(dev(a) for a in (self.pool.k, self.pool.v, self.pool.ks, self.pool.vs)))

    def append(self, pages, starts, lengths, k, v, q=None, cs=None, gk=None, gq=None, eps=None, pairs="halves", dtype=None):
        """On both; returns the queries and checks them."""
        T = k.shape[0]
        out = q4.q8_kv_append(self.cache, dev(pages), i32(starts), i32(lengths), k, v, q,
                              None if cs is None else dev(cs), gk, gq, eps, pairs, dtype)
        k64, q64 = f64(k), f64(q)
        keys = np.zeros(k64.shape)
        D = k64.shape[2]
        for row, _, pos in S.rows_of(starts, lengths, T):
            angles = None
            if cs is not None:
                angles = cs[pos] if 0 <= pos < len(cs) else np.full(cs.shape[1], np.nan)
            for h in range(k64.shape[1]):
                keys[row, h] = S.head(k64[row, h], f64(gk), eps, angles, pairs == "halves")
            for h in range(0 if q is None else q64.shape[1]):
                ref = S.head(q64[row, h], f64(gq), eps, angles, pairs == "halves")
                plain = S.head(q64[row, h], f64(gq), eps, None, True)
                mag = np.abs(plain) + (0 if cs is None else np.abs(plain).max())
                tol = (D / 2 + 16) * 2.0 ** -24 * mag + 1e-44
                if out.dtype == torch.bfloat16:
                    tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
                got = f64(out[row, h])
                assert np.all((np.abs(got - ref) <= tol) | (np.isnan(got) & np.isnan(ref))), ("queries", row, h)
        self.pool.append(pages, starts, lengths, {"k": keys, "v": f64(v)})
        return out

    def check(self, what, pages=None, starts=None, lengths=None):
        """The whole pool but the codes behind a block's last token, which mean nothing: compared with what was there
        is what the oracle keeps, so they are left out where `pages` names the sequences."""
        got = [host(t) for t in self.cache]
        want = [self.pool.k, self.pool.v, self.pool.ks, self.pool.vs]
        if pages is not None:
            for i, n in enumerate(lengths):
                if n % 16:
                    at = self.pool.place(pages, i, n - 1)
                    if at is not None:
                        for a in (got[0], want[0]):
                            a[at[0], :, at[1], :, n % 16:] = 0
                        for a in (got[1], want[1]):
                            a[at[0], :, at[1], :, n % 16:] = 0
        for g, w, name in zip(got, want, ("k", "v", "k_scale", "v_scale")):
            assert_bitwise(g, w, f"{what}: {name}")


CASES = [
    # lengths with the new tokens, new tokens, H, Hq, D, R, page
    ([1], [1], 1, 1, 16, 16, 16),
    ([37], [37], 2, 4, 64, 64, 16),
    ([1000], [1], 4, 16, 128, 128, 64),
    ([16, 17, 33, 15], [1, 1, 1, 1], 3, 3, 80, 40, 16),
    ([48, 5, 70], [16, 0, 39], 2, 6, 96, 96, 32),
    ([129, 64], [100, 64], 1, 5, 256, 64, 128),
    ([31, 31, 31], [15, 16, 17], 2, 2, 32, 6, 16),
    ([50], [20], 8, 8, 112, 112, 32),
    ([300] * 70, [1] * 70, 1, 1, 48, 48, 16),
]


@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("how", ["halves", "neighbours", "plain", "norm only"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, how, xt, yt):
    """Slices of a fused projection, as they lie, into a pool that others have used."""
    lengths, new, H, Hq, D, R, page = CASES[case]
    rng = np.random.default_rng(100 * case + len(how))
    pages, P = new_pages(rng, lengths, page)
    both = Both(P, H, page, D, rng)
    both.pool.ks[...] = rng.integers(117, 124, both.pool.ks.shape)
    both.pool.vs[...] = rng.integers(117, 124, both.pool.vs.shape)
    both.cache.k_scale.copy_(dev(both.pool.ks))
    both.cache.v_scale.copy_(dev(both.pool.vs))
    T = sum(new)
    starts = np.concatenate([[0], np.cumsum(new)])
    qkv = dev(rng.standard_normal((T, (Hq + 2 * H) * D)).astype(np.float32)).to(TORCH[xt])
    q, k, v = (t.view(T, -1, D) for t in qkv.split([Hq * D, H * D, H * D], 1))
    gk, gq = (dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(TORCH[yt]) for _ in range(2))
    cs = table(max(lengths), R) if how != "norm only" and how != "plain" else None
    norm = how in ("halves", "norm only")
    both.append(pages, starts, lengths, k, v, q, cs, gk if norm else None, gq if norm else None, 1e-6 if norm else None,
                how if how == "neighbours" else "halves", yt)
    both.check(how, pages, starts, lengths)
    # reading back: whole contexts would hold what others left, so the new tokens
    for dtype in ("f32", "bf16"):
        ko, vo = q4.q8_kv_read(both.cache, dev(pages), i32(starts), i32(lengths), T, dtype)
        want = np.zeros((2, T, H, D))
        for row, i, pos in S.rows_of(starts, lengths, T):
            for h in range(H):
                want[0, row, h], want[1, row, h] = (both.pool.value(n, pages, i, h, pos) for n in "kv")
        for got, w, name in ((ko, want[0], "k"), (vo, want[1], "v")):
            w = w.astype(np.float32)
            assert_bitwise(host(got), w if dtype == "f32" else F.f32_to_bf16_bits(w), f"read {name} {dtype}")


def test_tokens_one_by_one():
    """A sequence grown by single tokens and chunks, values of growing size: scales grow, codes are rounded again."""
    rng = np.random.default_rng(7)
    H, D, page = 2, 64, 32
    pages, P = new_pages(rng, [100], page)
    both = Both(P, H, page, D)
    n = 0
    for step in [1] * 40 + [7, 1, 16, 3, 1, 1, 30]:
        n += step
        k, v = (dev((rng.standard_normal((step, H, D)) * 1.15 ** (n % 40)).astype(np.float32)) for _ in range(2))
        both.append(pages, [0, step], [n], k, v)
        both.check(f"{n} tokens", pages, [0, step], [n])
    # the same tokens again change nothing
    before = [host(t) for t in both.cache]
    q4.q8_kv_append(both.cache, dev(pages), i32([0, step]), i32([n]), k, v)
    for a, b in zip(before, both.cache):
        assert_bitwise(host(b), a, "again")


def test_error_of_repeated_rounding():
    """Doublings at every token: what a block's first token loses stays below one step of the last scale."""
    rng = np.random.default_rng(8)
    D = 64
    both = Both(1, 1, 16, D)
    pages = np.zeros((1, 1), np.int32)
    first = rng.standard_normal((1, 1, D)).astype(np.float32)
    for t in range(12):
        x = first if t == 0 else np.full((1, 1, D), 2.0 ** t, np.float32)
        both.append(pages, [0, 1], [t + 1], dev(x), dev(x))
        step = 2.0 ** (int(both.pool.ks[0, 0, 0]) - 127)
        got = host(q4.q8_kv_read(both.cache, dev(pages), i32([0, t + 1]), i32([t + 1]), t + 1, "f32")[0])
        assert np.abs(got[0, 0] - first[0, 0]).max() < step
    both.check("doublings", pages, [0, 1], [12])


def test_rows_of_no_sequence_are_left():
    rng = np.random.default_rng(9)
    H, D, T = 2, 32, 9
    pages, P = new_pages(rng, [4, 20], 16)
    both = Both(P, H, 16, D)
    x = dev(rng.standard_normal((T, 3 * H, D)).astype(np.float32))
    starts = [2, 5, 7]                    # rows 0, 1, 7, 8 belong to nobody
    out = torch.full((T, H, D), 77.0, device=DEV)
    q4.q8_kv_append(both.cache, dev(pages), i32(starts), i32([4, 20]), x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q_out=out)
    both.pool.append(pages, starts, [4, 20], {"k": f64(x[:, :H]), "v": f64(x[:, H:2 * H])})
    both.check("cache", pages, starts, [4, 20])
    got = host(out)
    assert (got[[0, 1, 7, 8]] == 77).all()
    assert_bitwise(got[2:7], host(x[2:7, 2 * H:]), "queries as they were")


def test_more_rows_than_tokens_and_bad_pages():
    """Positions below 0 are dropped; tokens on pages out of the table or the pool are dropped and read as NaN."""
    rng = np.random.default_rng(10)
    H, D, page = 1, 16, 16
    both = Both(4, H, page, D, rng)
    pages = np.array([[2, -1, 9], [0, 3, 1]], np.int32)
    starts, lengths = [0, 60, 64], [60, 2]          # 60 tokens: pages 2, none, none, past the table
    x = dev(rng.standard_normal((64, H, D)).astype(np.float32))
    both.append(pages, starts, lengths, x, x)
    both.check("cache", pages, starts, lengths)
    k, v = q4.q8_kv_read(both.cache, dev(pages), i32(starts), i32(lengths), 64, "f32")
    k = host(k)
    assert np.isfinite(k[:16]).all() and np.isnan(k[16:60]).all()
    assert np.array_equal(k[62:, 0], np.stack([both.pool.value("k", pages, 1, 0, p) for p in (0, 1)]).astype(np.float32))


def test_non_finite_values_mark_their_block():
    rng = np.random.default_rng(11)
    H, D = 2, 32
    pages, P = new_pages(rng, [40], 16)
    both = Both(P, H, 16, D)
    x = rng.standard_normal((40, H, D)).astype(np.float32)
    x[3, 0, 5], x[20, 1, 0], x[39, 0, 31] = np.nan, np.inf, -np.inf
    both.append(pages, [0, 40], [40], dev(x), dev(x))
    both.check("cache", pages, [0, 40], [40])
    k = host(q4.q8_kv_read(both.cache, dev(pages), i32([0, 40]), i32([40]), 40, "f32")[0])
    nan = np.isnan(k).all(axis=2)
    assert np.array_equal(nan, np.isnan(k).any(axis=2))
    want = np.zeros((40, H), bool)
    want[:16, 0] = want[16:32, 1] = want[32:, 0] = True
    assert np.array_equal(nan, want)
    # an angle that is not in the table is NaN
    cs = table(20, D)
    both.append(pages, [0, 40], [40], dev(np.ones((40, H, D), np.float32)), dev(x), None, cs)
    both.check("angles", pages, [0, 40], [40])


def test_extreme_sizes_of_values():
    D = 16
    both = Both(1, 1, 64, D)
    pages = np.zeros((1, 1), np.int32)
    x = np.zeros((64, 1, D), np.float32)
    x[:16] = 3.4e38
    x[16:32, 0, 0] = 5 * 2.0 ** -127       # subnormal
    x[32:48, 0, 1] = 127 * 2.0 ** -120
    both.append(pages, [0, 64], [64], dev(x), dev(-x))
    both.check("cache", pages, [0, 64], [64])
    # 3.4e38 is above 127 2^121 = 3.376e38
    assert both.pool.ks[0, 0].tolist() == [249, 0, 7, 0]
    k, v = q4.q8_kv_read(both.cache, dev(pages), i32([0, 64]), i32([64]), 64, "f32")
    assert_bitwise(host(k)[16:], x[16:], "exact")
    assert np.array_equal(host(v)[16:], -x[16:])           # code 0 has no sign


def test_a_large_pool():
    """Blocks past 2^32 bytes."""
    H, D, page, P = 8, 128, 64, 70000
    cache = q4.q8_kv_cache(P, H, page, D)
    rng = np.random.default_rng(12)
    pages = np.array([[P - 1, 0], [65535, 40000]], np.int32)
    x = dev(rng.standard_normal((200, H, D)).astype(np.float32))
    q4.q8_kv_append(cache, dev(pages), i32([0, 100, 200]), i32([100, 100]), x, x)
    small = Both(4, H, page, D)
    near = np.array([[3, 0], [2, 1]], np.int32)
    small.append(near, [0, 100, 200], [100, 100], x, x)
    k, v = q4.q8_kv_read(cache, dev(pages), i32([0, 100, 200]), i32([100, 100]), 200)
    k2, v2 = q4.q8_kv_read(small.cache, dev(near), i32([0, 100, 200]), i32([100, 100]), 200)
    assert_bitwise(host(k), host(k2), "keys")
    assert_bitwise(host(v), host(v2), "values")
    for far, page_ in ((P - 1, 3), (65535, 2), (40000, 1)):
        for a, b, name in zip(cache, small.cache, ("k", "v", "k_scale", "v_scale")):
            assert_bitwise(host(a[far]), host(b[page_]), name)


def test_many_sequences():
    """More than 64, and more than 4096: the search for a row's sequence takes several turns."""
    rng = np.random.default_rng(13)
    for N in (65, 4500):
        new = rng.integers(0, 3, N)
        lengths = new + rng.integers(0, 15, N)
        pages, P = new_pages(rng, lengths, 16)
        both = Both(P, 1, 16, 16)
        starts = np.concatenate([[0], np.cumsum(new)])
        x = dev(rng.standard_normal((starts[-1], 1, 16)).astype(np.float32))
        out = q4.q8_kv_append(both.cache, dev(pages), i32(starts), i32(lengths), x, x, x, dev(table(20, 16)), None, None,
                              None, "neighbours")
        keys = np.zeros(x.shape)
        for row, _, pos in S.rows_of(starts, lengths, len(x)):
            keys[row, 0] = S.head(f64(x[row, 0]), None, None, table(20, 16)[pos], False)
        assert np.abs(f64(out) - keys).max() < 24 * 2.0 ** -24 * 8
        both.pool.append(pages, starts, lengths, {"k": keys, "v": f64(x)})
        # old content of blocks that were never written is zero under scale 0 on both sides
        both.check(f"{N} sequences", pages, starts, lengths)


def test_other_layouts_and_streams():
    """Head-major inputs at odd addresses, on a side stream."""
    rng = np.random.default_rng(14)
    T, H, D = 21, 2, 48
    pages, P = new_pages(rng, [21], 16)
    both = Both(P, H, 16, D)
    buf = dev(rng.standard_normal(3 * T * H * D + 9).astype(np.float32)).bfloat16()
    k = buf[1:1 + T * H * D].view(H, T, D).transpose(0, 1)
    v = buf[T * H * D + 2:2 * T * H * D + 2].view(H, T, D).transpose(0, 1)
    q = buf[2 * T * H * D + 5:3 * T * H * D + 5].view(H, T, D).transpose(0, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both.append(pages, [0, T], [T], k, v, q, table(T, D), None, None, 1e-6)
    side.synchronize()
    both.check("head-major", pages, [0, T], [T])


def test_graph_replays():
    """A captured step: lengths, starts and rows change between the replays."""
    H, Hq, D, N = 2, 4, 64, 5
    cs = dev(table(64, D))
    caches = [q4.q8_kv_cache(N * 4, H, 16, D) for _ in range(2)]
    pages = torch.randperm(N * 4, generator=torch.Generator().manual_seed(1)).int().view(N, 4).to(DEV)
    starts, lengths = torch.arange(N + 1, device=DEV).int(), torch.ones(N, dtype=torch.int32, device=DEV)
    x = torch.zeros(N, Hq + 2 * H, D, dtype=torch.bfloat16, device=DEV)

    def call(c):
        return q4.q8_kv_append(c, pages, starts, lengths, x[:, Hq:Hq + H], x[:, Hq + H:], x[:, :Hq], cs, None, None, 1e-6)

    call(caches[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(caches[0])
    for step in range(1, 21):
        x.copy_(torch.randn(x.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(step)) * step)
        lengths.fill_(step)
        graph.replay()
        got = host(out)
        assert_bitwise(got, host(call(caches[1])), f"queries {step}")
        for a, b in zip(*caches):
            assert_bitwise(host(a), host(b), f"cache {step}")


def test_refused():
    H, D = 2, 32
    c = q4.q8_kv_cache(3, H, 16, D)
    pages, starts, lengths = i32([[0, 1]]), i32([0, 2]), i32([2])
    x = torch.zeros(2, H, D, device=DEV)
    for bad in (lambda: q4.q8_kv_append(c, pages, starts[:1], lengths, x, x),
                lambda: q4.q8_kv_append(c, pages, starts, i32([1, 2]), x, x),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x[:, :1], x),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x[:1]),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x.transpose(1, 2)),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, k_gain=torch.ones(D, device=DEV)),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, k_gain=torch.ones(D + 1, device=DEV), eps=1e-6),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, q_out=x),
                lambda: q4.q8_kv_append((c.k, c.v[:2], c.k_scale, c.v_scale), pages, starts, lengths, x, x),
                lambda: q4.q8_kv_append((c.k, c.v, c.k_scale[:, :1].contiguous(), c.v_scale), pages, starts, lengths, x, x),
                lambda: q4.q8_kv_read(c, pages, starts, i32([1, 2]), 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q8_kv_append(c, pages.long(), starts, lengths, x, x),
                lambda: q4.q8_kv_append(c, pages, starts.long(), lengths, x, x),
                lambda: q4.q8_kv_append(c, pages, starts, lengths.long(), x, x),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x.bfloat16()),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x.half(), x.half()),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, x.bfloat16()),
                lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, x, dtype="bf16", q_out=x.clone())):
        with pytest.raises(TypeError):
            bad()
    for bad, status in ((lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, x, torch.zeros(4, 34, device=DEV)), q4.ESHAPE),
                        (lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, eps=-1.0), q4.EINVAL),
                        (lambda: q4.q8_kv_append(c, pages, starts, lengths, x, x, x, q_out=x), q4.EINVAL),
                        (lambda: q4.q8_kv_append(c, c.k.view(-1)[:8].view(torch.int32).view(1, 2), starts, lengths, x, x), q4.EINVAL)):
        with pytest.raises(q4.Q4Error) as e:
            bad()
        assert e.value.status == status
    none = torch.zeros(0, H, D, device=DEV)
    assert q4.q8_kv_append(c, pages, i32([0, 0]), lengths, none, none) is None
    assert q4.q8_kv_append(c, pages[:0], i32([0]), lengths[:0], x, x, x).shape == x.shape
    assert q4.q8_kv_read(c, pages, i32([0, 0]), lengths, 0)[0].shape == (0, H, D)
    assert not any(t.any() for t in c)


def test_both_paths_of_the_binding_agree(monkeypatch):
    rng = np.random.default_rng(15)
    H, D, T = 2, 32, 30
    pages, P = new_pages(rng, [T], 16)
    x = dev(rng.standard_normal((T, 3 * H, D)).astype(np.float32))
    g = dev(rng.standard_normal(D).astype(np.float32))
    results = []
    for direct in (True, False):
        if not direct:
            monkeypatch.setattr(q4, "_DIRECT", q4._NoDirect())
        c = q4.q8_kv_cache(P, H, 16, D)
        out = q4.q8_kv_append(c, dev(pages), i32([0, T]), i32([T]), x[:, :H], x[:, H:2 * H], x[:, 2 * H:], dev(table(T, 8)),
                              g, g, 1e-6, "neighbours", "bf16")
        results.append([host(t) for t in (*c, out, *q4.q8_kv_read(c, dev(pages), i32([0, T]), i32([T]), T, "f32"))])
    for a, b in zip(*results):
        assert_bitwise(a, b, "paths")

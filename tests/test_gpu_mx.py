"""MX FP4 on the GPU against the float64 oracle.

Quantisation and its inverse are compared bit for bit.  A product of n terms
in f32 is off by at most n + 8 roundings (half a step, 2^-24, each) of the sum
of the terms' magnitudes, and never by more than the 1e-5 of that sum which
the library's float products keep; a bf16 result by half a bf16 step (2^-8)
of itself more.
"""
import numpy as np
import pytest
import torch

import int4_dequantize_matmul_amd as q4
import oracle.formats as F
import oracle.mx as X
from tests.gpu_util import DEV, assert_bitwise, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _auto_path():
    q4.q4_set_path("auto")
    yield
    q4.q4_set_path("auto")


def bf16(x):
    """float array -> (bf16 bits uint16, their values float64)."""
    x = np.asarray(x, np.float32)
    b = F.f32_to_bf16_bits(np.where(np.isfinite(x), x, 0))
    b = np.where(np.isfinite(x), b, np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16)
    return b, F.bf16_bits_to_f32(b).astype(np.float64)


def rows(seed, M, K, xt):
    """Rows with columns of different sizes, a zero row and a zero block -> (device array, float64 values)."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((M, K)) * np.exp2(rng.integers(-6, 7, K))).astype(np.float32)
    if M > 2:
        x[1] = 0
        x[2, :32] = 0
    if xt == "bf16":
        b, v = bf16(x)
        return dev(b), v
    return dev(x), x.astype(np.float64)


def weights(seed, N, K):
    rng = np.random.default_rng(seed)
    c, s = X.quantize_rows((0.02 * rng.standard_normal((N, K))).astype(np.float32))
    return c, s


def check(y, ref, mag, K, what):
    got = host(y)
    if y.dtype == torch.bfloat16:
        got = F.bf16_bits_to_f32(got)
    got = got.astype(np.float64)
    tol = min(1e-5, (K + 8) * 2.0 ** -24) * mag + 1e-44
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


# ---- quantisation ----------------------------------------------------------

@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (1, 32), (3, 33), (5, 7), (2, 2048), (7, 1023), (65, 96),
                                 (4, 4099), (300, 64), (1, 70000)])
def test_quantize_bitwise(M, K, xt):
    xd, v = rows(M * 7919 + K, M, K, xt)
    c, s = q4.q4_mx_quantize_rows(xd)
    cr, sr = X.quantize_rows(v)
    assert_bitwise(host(s), sr, "scales")
    assert_bitwise(host(c), cr, "codes")
    y = q4.q4_mx_dequantize_rows(c, s, K, "f32")
    assert_bitwise(host(y), X.dequantize_rows(cr, sr, K).astype(np.float32), "f32 values")
    yb = q4.q4_mx_dequantize_rows(c, s, K, "bf16")
    assert_bitwise(host(yb), F.f32_to_bf16_bits(X.dequantize_rows(cr, sr, K).astype(np.float32)), "bf16 values")


def test_quantize_every_bf16_and_borders():
    # every finite bf16, 31 of them under each of some block maxima
    allb = np.arange(65536, dtype=np.uint16)
    v = F.bf16_bits_to_f32(allb)
    allb = allb[np.isfinite(v)]
    allb = allb[: len(allb) // 31 * 31].reshape(-1, 31)
    for top in (0x0000, 0x0001, 0x0080, 0x00FF, 0x3F80, 0x40DF, 0x7F7F):
        x = np.concatenate([allb, np.full((len(allb), 1), top, np.uint16)], 1)
        c, s = q4.q4_mx_quantize_rows(dev(x))
        cr, sr = X.quantize_rows(F.bf16_bits_to_f32(x))
        assert_bitwise(host(s), sr, f"scales under {top:#x}")
        assert_bitwise(host(c), cr, f"codes under {top:#x}")
    # the borders between codes and both float32 neighbours of each, at several scales
    mid = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5], np.float32)
    b = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9))])
    for e in (-147, -127, -126, -125, -30, 0, 60, 125):
        with np.errstate(under="ignore"):
            r = np.ldexp(np.concatenate([b, [4.0], -b, [-0.0]]).astype(np.float32), e)[None, :]
        c, s = q4.q4_mx_quantize_rows(dev(np.ascontiguousarray(r, np.float32)))
        cr, sr = X.quantize_rows(r)
        assert_bitwise(host(s), sr, f"scale at {e}")
        assert_bitwise(host(c), cr, f"codes at {e}")


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_quantize_non_finite_blocks(xt):
    x = np.ones((4, 70), np.float32)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 69] = -np.inf
    xd = dev(x) if xt == "f32" else dev(bf16(x)[0])
    c, s = (host(t) for t in q4.q4_mx_quantize_rows(xd))
    assert (s == 255).tolist() == [[True, False, False], [False, True, False], [False, False, True], [False] * 3]
    cr, sr = X.quantize_rows(x)
    assert_bitwise(c, cr)
    y = host(q4.q4_mx_dequantize_rows(dev(c), dev(s), 70))
    assert np.array_equal(np.isnan(y), np.isnan(X.dequantize_rows(cr, sr, 70)))


def test_dequantize_every_code_and_scale():
    s = np.arange(256, dtype=np.uint8).reshape(-1, 1)
    c = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))
    c = np.concatenate([np.roll(c, i, axis=0) for i in range(16)])
    s = np.repeat(np.arange(256, dtype=np.uint8), 16).reshape(-1, 1)
    with np.errstate(over="ignore"):
        want = X.dequantize_rows(c, s).astype(np.float32)
    got = host(q4.q4_mx_dequantize_rows(dev(c), dev(s)))
    assert np.array_equal(got, want, equal_nan=True)
    gb = F.bf16_bits_to_f32(host(q4.q4_mx_dequantize_rows(dev(c), dev(s), dtype="bf16")))
    assert np.array_equal(gb, want, equal_nan=True)


# ---- products ----------------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 16, 32), (2, 3, 31), (1, 100, 33), (3, 17, 65), (15, 33, 511), (16, 16, 512),
          (17, 40, 513), (16, 129, 544), (31, 64, 2080), (32, 257, 96), (33, 70, 1023), (1, 512, 2048),
          (64, 80, 640), (65, 300, 128), (100, 256, 256), (128, 128, 320), (129, 255, 1056), (200, 513, 2048),
          (300, 384, 33), (257, 130, 4096)]


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("path", ["auto", "gemv", "tiled"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_w4a4(M, N, K, path, yt):
    q4.q4_set_path(path)
    xt = "bf16" if (M + N) % 2 else "f32"
    xd, v = rows(M + N + K, M, K, xt)
    wq, sw = weights(K + N, N, K)
    xq, sx = X.quantize_rows(v)
    ref, mag = X.linear_w4a4(xq, sx, wq, sw)
    check(q4.q4_linear_w4a4_mx(dev(xq), dev(sx), dev(wq), dev(sw), yt), ref, mag, K, "quantized rows")
    check(q4.q4_linear_w4a4_mx_dynamic(xd, dev(wq), dev(sw), yt), ref, mag, K, "rows quantized in the call")


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("path", ["auto", "gemv", "tiled"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_w4a16(M, N, K, path, yt):
    q4.q4_set_path(path)
    xd, v = rows(M + N + 3 * K, M, K, "bf16")
    wq, sw = weights(K + N, N, K)
    ref, mag = X.linear_w4a16(v, wq, sw)
    check(q4.q4_linear_w4a16_mx(xd, dev(wq), dev(sw), yt), ref, mag, K, "w4a16")


# More tiles than compute units: whole large tiles and the cut ones at the end,
# with edges in both directions; rows of scales that start on 16 bytes, on 4,
# and on any; rows of activations that start on 16 bytes and on 2.
LARGE = [(1000, 8210, 512), (1290, 6401, 640), (1100, 8300, 96), (1030, 8193, 130), (700, 5000, 1024),
         (513, 4100, 192), (260, 8197, 512), (900, 4600, 37), (130, 13317, 512)]


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_products_of_many_tiles(M, N, K, yt):
    xd, v = rows(M + N, M, K, "bf16")
    wq, sw = weights(K + N, N, K)
    ref, mag = X.linear_w4a16(v, wq, sw)
    check(q4.q4_linear_w4a16_mx(xd, dev(wq), dev(sw), yt), ref, mag, K, "w4a16")
    xq, sx = X.quantize_rows(v)
    ref, mag = X.linear_w4a4(xq, sx, wq, sw)
    check(q4.q4_linear_w4a4_mx(dev(xq), dev(sx), dev(wq), dev(sw), yt), ref, mag, K, "w4a4")


@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_scales_and_rows_of_any_alignment(off):
    """Scale arrays and bf16 rows that start at odd addresses (codes start on 16 bytes)."""
    for M, N, K in ((40, 300, 512), (20, 100, 256), (300, 8200, 512)):
        _, v = rows(off, M, K, "bf16")
        wq, sw = weights(off + 1, N, K)
        xq, sx = X.quantize_rows(v)

        def at(a, o):
            buf = torch.zeros(a.size + o, dtype=torch.uint8, device=DEV)
            buf[o:] = torch.from_numpy(np.ascontiguousarray(a).reshape(-1)).to(DEV)
            return buf[o:].view(a.shape)

        xb = bf16(v)[0]
        xs = torch.zeros(xb.size + off, dtype=torch.bfloat16, device=DEV)
        xs[off:] = dev(xb).reshape(-1)
        ref, mag = X.linear_w4a16(v, wq, sw)
        check(q4.q4_linear_w4a16_mx(xs[off:].view(M, K), dev(wq), at(sw, off), "f32"), ref, mag, K, "w4a16")
        ref, mag = X.linear_w4a4(xq, sx, wq, sw)
        check(q4.q4_linear_w4a4_mx(dev(xq), at(sx, off), dev(wq), at(sw, 16 - off), "f32"), ref, mag, K, "w4a4")


@pytest.mark.parametrize("path", ["auto", "gemv", "tiled"])
@pytest.mark.parametrize("M", [1, 5, 16, 40, 130])
def test_products_index_probe(M, path):
    """One-hot rows read single weights: exact, every column and every block's own scale."""
    q4.q4_set_path(path)
    N, K = 70, 1100
    rng = np.random.default_rng(M)
    B = X.blocks(K)
    wq = rng.integers(0, 256, (N, 16 * B), dtype=np.uint8)
    wq[:, 16 * (B - 1) + (K % 32 + 1) // 2:] = 0                 # codes past K
    sw = rng.integers(100, 140, (N, B), dtype=np.uint8)
    w = X.dequantize_rows(wq, sw, K)
    for k0 in range(0, K, 13 * M):
        ks = [(k0 + 13 * m) % K for m in range(M)]
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), ks] = 1
        want = w[:, ks].T.astype(np.float32)
        y = host(q4.q4_linear_w4a4_mx_dynamic(dev(x), dev(wq), dev(sw), "f32"))
        assert np.array_equal(y, want), ("w4a4", k0)
        y = host(q4.q4_linear_w4a16_mx(dev(bf16(x)[0]), dev(wq), dev(sw), "f32"))
        assert np.array_equal(y, want), ("w4a16", k0)


@pytest.mark.parametrize("path", ["auto", "gemv", "tiled"])
@pytest.mark.parametrize("M", [3, 70])
def test_products_nan_and_extreme_scales(M, path):
    q4.q4_set_path(path)
    N, K = 40, 100
    xd, v = rows(5, M, K, "bf16")
    wq, sw = weights(6, N, K)
    sw[4, 1] = 255                                            # column 4 of y: NaN
    x = v.copy()
    x[0, 99] = np.nan                                         # rows 0 and 2: NaN
    x[2, 5] = np.inf
    xb = dev(bf16(x)[0])
    for y in (q4.q4_linear_w4a4_mx_dynamic(xb, dev(wq), dev(sw), "f32"),
              q4.q4_linear_w4a4_mx_dynamic(xb, dev(wq), dev(sw), "bf16").float()):
        n = np.isnan(host(y))
        assert n[0].all() and n[2].all() and n[:, 4].all()
        n[[0, 2]] = False
        n[:, 4] = False
        assert not n.any()
    for dt in ("f32", "bf16"):
        y = host(q4.q4_linear_w4a16_mx(xb, dev(wq), dev(sw), dt).float())
        want = x.astype(np.float64)[2, 5] * X.dequantize_rows(wq, sw, K)[:, 5]
        assert np.isnan(y[0]).all() and np.isnan(y[:, 4]).all() and not np.isnan(y[1, :4]).any()
        inf = np.isfinite(X.dequantize_rows(wq, sw, K)).all(1) & (want != 0) & ~np.isnan(want)
        assert np.array_equal(y[2][inf], want[inf])
    # scales at both ends of the range that cancel
    sw[:] = 0
    sx = np.full((M, 4), 254, np.uint8)
    xq = np.zeros((M, 64), np.uint8)
    xq[:, :50] = 0x22                                         # ones, 2^127 each
    ref, mag = X.linear_w4a4(xq, sx, wq, sw)
    check(q4.q4_linear_w4a4_mx(dev(xq), dev(sx), dev(wq), dev(sw), "f32"), ref, mag, K, "2^127 times 2^-127")


@pytest.mark.parametrize("op", ["w4a4", "w4a16"])
def test_batch_rows_do_not_depend_on_the_batch(op):
    N, K = 100, 1600
    xd, _ = rows(9, 16, K, "bf16")
    wq, sw = (dev(a) for a in weights(10, N, K))
    f = q4.q4_linear_w4a4_mx_dynamic if op == "w4a4" else q4.q4_linear_w4a16_mx
    y = host(f(xd, wq, sw, "f32"))
    for M in (1, 2, 7, 15):
        assert_bitwise(host(f(xd[:M].contiguous(), wq, sw, "f32")), y[:M], f"M = {M}")


def test_empty_sizes():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    x = torch.zeros((3, 0), device=DEV)
    c, s = q4.q4_mx_quantize_rows(x)
    assert c.shape == (3, 0) and s.shape == (3, 0)
    assert q4.q4_mx_dequantize_rows(c, s, 0).shape == (3, 0)
    y = torch.full((3, 5), float("nan"), device=DEV)
    assert not host(q4.q4_linear_w4a4_mx(c, s, z(5, 0), z(5, 0), "f32", y=y)).any()
    y.fill_(float("nan"))
    assert not host(q4.q4_linear_w4a4_mx_dynamic(x, z(5, 0), z(5, 0), "f32", y=y)).any()
    yb = torch.full((3, 5), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert not host(q4.q4_linear_w4a16_mx(x.bfloat16(), z(5, 0), z(5, 0), "bf16", y=yb)).any()
    assert q4.q4_linear_w4a16_mx(x[:0].bfloat16(), z(5, 0), z(5, 0)).shape == (0, 5)
    assert q4.q4_linear_w4a4_mx_dynamic(x, z(0, 0), z(0, 0)).shape == (3, 0)


def test_python_refusals():
    z = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d, device=DEV)
    x = z(2, 64, d=torch.bfloat16)
    for bad in (lambda: q4.q4_linear_w4a16_mx(x, z(3, 16), z(3, 1)),              # one block for 64 columns
                lambda: q4.q4_linear_w4a16_mx(x, z(3, 32), z(3, 3)),
                lambda: q4.q4_linear_w4a16_mx(x, z(3, 32), z(4, 2)),
                lambda: q4.q4_linear_w4a16_mx(x.t(), z(3, 16), z(3, 1)),
                lambda: q4.q4_linear_w4a4_mx(z(2, 16), z(2, 1), z(3, 32), z(3, 2)),
                lambda: q4.q4_linear_w4a16_mx(x, z(3, 32), z(3, 2), y=z(2, 4, d=torch.bfloat16)),
                lambda: q4.q4_mx_dequantize_rows(z(2, 32), z(2, 2), 32)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q4.q4_linear_w4a16_mx(x.half(), z(3, 32), z(3, 2)),
                lambda: q4.q4_mx_quantize_rows(x.half()),
                lambda: q4.q4_linear_w4a16_mx(x, z(3, 32, d=torch.int8), z(3, 2))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(q4.Q4Error) as e:
        q4.q4_linear_w4a4_mx_dynamic(x, z(3, 32), z(3, 2), ws=z(8))
    assert e.value.status == q4.EINVAL


@pytest.mark.parametrize("op", ["w4a4", "w4a16"])
def test_results_past_32_bit_offsets(op):
    """An output of more than 2^32 bytes: its first, middle and last rows."""
    M, N, K = 40003, 60001, 40
    rng = np.random.default_rng(0)
    x = torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    wq, sw = weights(3, N, K)
    y = (q4.q4_linear_w4a4_mx_dynamic if op == "w4a4" else q4.q4_linear_w4a16_mx)(x, dev(wq), dev(sw), "bf16")
    at = np.unique(np.concatenate([[0, 1, M // 2, 35791, 35792, M - 2, M - 1], rng.integers(0, M, 9)]))
    v = F.bf16_bits_to_f32(host(x[torch.from_numpy(at).to(DEV)])).astype(np.float64)
    if op == "w4a4":
        ref, mag = X.linear_w4a4(*X.quantize_rows(v), wq, sw)
    else:
        ref, mag = X.linear_w4a16(v, wq, sw)
    check(y[torch.from_numpy(at).to(DEV)], ref, mag, K, op)


def test_rows_past_32_bit_offsets():
    """Activations of more than 2^32 elements: quantised, and through a product, at both ends."""
    M, K, N = 1048000, 4128, 17
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 520000, 520001, M - 1]
    vals = torch.randn(len(at), K, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).bfloat16()
    x[torch.tensor(at, device=DEV)] = vals
    v = F.bf16_bits_to_f32(host(vals)).astype(np.float64)
    cr, sr = X.quantize_rows(v)
    c, s = q4.q4_mx_quantize_rows(x)
    assert_bitwise(host(c[torch.tensor(at, device=DEV)]), cr)
    assert_bitwise(host(s[torch.tensor(at, device=DEV)]), sr)
    wq, sw = weights(4, N, K)
    y = q4.q4_linear_w4a4_mx(c, s, dev(wq), dev(sw), "f32")
    check(y[torch.tensor(at, device=DEV)], *X.linear_w4a4(cr, sr, wq, sw), K, "w4a4")
    assert not y[2:520000].any()
    y = q4.q4_linear_w4a16_mx(x, dev(wq), dev(sw), "f32")
    check(y[torch.tensor(at, device=DEV)], *X.linear_w4a16(v, wq, sw), K, "w4a16")
    assert not y[2:520000].any()


def test_streams_and_graph_replays():
    """Calls on a side stream, and captured: every replay against the eager result on the same inputs."""
    M, N, K = 70, 200, 640
    wq, sw = (dev(a) for a in weights(20, N, K))
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(q4.q4_w4a4_mx_dynamic_workspace(M, K), dtype=torch.uint8, device=DEV)
    ys = [torch.empty((M, N), device=DEV) for _ in range(2)]

    def calls():
        q4.q4_linear_w4a4_mx_dynamic(x, wq, sw, "f32", ws=ws, y=ys[0])
        q4.q4_linear_w4a16_mx(x, wq, sw, "f32", y=ys[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in range(4):
        x.copy_(torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)))
        graph.replay()
        got = [host(y) for y in ys]
        calls()
        for g, y in zip(got, ys):
            assert_bitwise(g, host(y), f"replay {seed}")


class _NoDirect:
    """In the place of the C++ path: takes nothing."""

    def __getattr__(self, name):
        return lambda *args: None


@pytest.mark.parametrize("M,K", [(1, 2048), (3, 33), (20, 96), (70, 640)])
def test_both_paths_of_the_binding_agree(M, K, monkeypatch):
    """The calls through C++ and through ctypes give the same bits, types and shapes."""
    N, T, D = 50, M, 64
    gen = torch.Generator(DEV).manual_seed(M)
    x = torch.randn(M, K, device=DEV, generator=gen)
    wq, sw = (dev(a) for a in weights(M + K, N, K))
    heads = torch.randn(T, 6, D, device=DEV, generator=gen)
    gain, pos = torch.ones(D, device=DEV), torch.arange(T, device=DEV) % 5
    cs = torch.randn(5, 32, device=DEV, generator=gen)

    def calls():
        xq, sx = q4.q4_mx_quantize_rows(x)
        out = [xq, sx]
        for dt in ("f32", "bf16"):
            out += [q4.q4_mx_dequantize_rows(xq, sx, K, dt), q4.q4_linear_w4a4_mx(xq, sx, wq, sw, dt),
                    q4.q4_linear_w4a4_mx_dynamic(x, wq, sw, dt), q4.q4_linear_w4a16_mx(x.bfloat16(), wq, sw, dt)]
            for pairs in ("halves", "neighbours"):
                out += q4.q4_qk_norm_rope(heads[:, :4], heads[:, 4:], gain, gain, pos, cs, 1e-5, pairs, dt)
        return out

    direct = calls()
    monkeypatch.setattr(q4, "_direct", lambda: _NoDirect())
    for a, b in zip(direct, calls()):
        assert a.dtype == b.dtype and a.is_contiguous()
        assert_bitwise(host(a), host(b))


def test_the_direct_path_leaves_what_it_does_not_take():
    d = q4._direct()
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    c, s = q4.q4_mx_quantize_rows(x)
    for args in ((x.cpu(), c, s, 1), (x.half(), c, s, 1), (x.t(), c, s, 1), (x[:0], c, s, 1), (x, c, s[:, :1], 1),
                 (x, c[:, ::2], s, 1), (x, c.int(), s, 1), (x, None, s, 1), (x, c, s), (1, 2, 3, 4)):
        assert d.w4a16(*args) is None and d.w4a4_dynamic(*args) is None
    assert d.dequantize_rows(c, s, 65, 0) is None and d.dequantize_rows(c, s, 32, 0) is None
    assert d.dequantize_rows(c, s, 0, 0) is None and d.dequantize_rows(c, s, -5, 0) is None
    assert d.w4a4(c, s, c[:, :16].contiguous(), s[:, :1].contiguous(), 0) is None
    assert d.quantize_rows(x.double()) is None and d.quantize_rows([1.0]) is None
    h, g, p, t = x.view(2, 1, 64), x[0], torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(4, 64, device=DEV)
    for args in ((h, h, g, g, p.int(), t, 1e-6, 0, -1), (h, None, g, g, p, t, 1e-6, 0, -1),
                 (h, h.float(), g, g, p, t, 1e-6, 0, -1), (h, h, g[:32], g, p, t, 1e-6, 0, -1),
                 (h, h, g, g, p[:1], t, 1e-6, 0, -1), (h.transpose(1, 2), h, g, g, p, t, 1e-6, 0, -1),
                 (h, h, g, g, p, t[:, :7].contiguous(), 1e-6, 0, -1)):
        assert d.qk_norm_rope(*args) is None

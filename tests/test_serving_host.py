"""Argument checks of the row norm, cache and attention calls on the CPU: a
refused call returns its status before any device call and writes nothing."""
import ctypes

import pytest
import torch

import int4_dequantize_matmul_amd as q4

BUF = (ctypes.c_uint8 * (1 << 18))()
BASE = (ctypes.addressof(BUF) + 255) & ~255
X, R, G, S, C, SX, K, V, KS, VS, PG, ST, LEN, Q, QO, CS, WS, Y = (BASE + 8192 * i for i in range(18))
F32, BF16 = 0, 1
E, SH = q4.EINVAL, q4.ESHAPE


@pytest.fixture(autouse=True)
def _canary():
    ctypes.memset(BUF, 0xA5, len(BUF))
    yield
    assert bytes(BUF) == b"\xA5" * len(BUF)


def call(name, args):
    args = {k: (ctypes.byref(v) if isinstance(v, q4.KVCacheC) else v) for k, v in args.items()}
    return getattr(q4.raw(), name)(*args.values())


def expect(name, good, changes):
    """`good` with one argument changed at a time gives the status."""
    for status, change in changes:
        assert call(name, dict(good, **change)) == status, (name, change)


def cache(**change):
    """Two pages of 32 tokens of two heads of 16: 2048 bytes of codes each, 8 scales; 3 sequences, 4 entries."""
    f = dict(k=K, v=V, k_scale=KS, v_scale=VS, pages=PG, n_pages=2, page=32, heads=2, D=16, sequences=3, table=4)
    f.update(change)
    return q4.KVCacheC(*f.values())


BAD_CACHES = [(E, cache(**{p: None})) for p in ("k", "v", "k_scale", "v_scale", "pages")] + [
    (E, cache(**{p: -1})) for p in ("n_pages", "page", "heads", "D", "sequences", "table")] + [
    (E, cache(k=K + 8)), (E, cache(v=V + 4)), (SH, cache(D=24)), (SH, cache(D=0)), (SH, cache(D=272)),
    (SH, cache(page=0)), (SH, cache(page=8)), (SH, cache(page=48)), (SH, cache(page=131072)), (SH, cache(heads=0)),
    (SH, cache(n_pages=0)), (SH, cache(table=0)), (SH, cache(n_pages=2 ** 31)), (SH, cache(n_pages=2 ** 30, page=16)),
    (SH, cache(n_pages=2 ** 20, heads=2 ** 10, page=64)), (SH, cache(sequences=2 ** 31)), (SH, cache(table=2 ** 31))]


def test_rmsnorm_rows():
    good = dict(x=X, residual=R, xt=BF16, gain=G, gt=F32, eps=1e-6, M=2, K=40, sum=S, xq=C, sx=SX, stream=None)
    expect("q8_rmsnorm_rows", good, [
        (E, {p: None}) for p in ("x", "xq", "sx")] + [
        (E, {"M": -1}), (E, {"K": -1}), (E, {"xt": 2}), (E, {"gt": -1}), (E, {"eps": -1e-9}), (E, {"eps": float("nan")}),
        (E, {"residual": None}), (E, {"xq": X + 159}), (E, {"xq": R}), (E, {"xq": G + 159}), (E, {"xq": S + 1}),
        (E, {"sx": X}), (E, {"sx": C + 79}), (E, {"sum": X + 2}), (E, {"sum": R + 158}), (E, {"sum": G}),
        (SH, {"M": 2 ** 30 + 1}), (SH, {"K": 2 ** 30 + 1}), (q4.OK, {"M": 0}),
        (q4.OK, {"M": 0, "sum": R}), (q4.OK, {"M": 0, "sum": X}), (q4.OK, {"M": 0, "residual": None, "sum": None})])


APPEND = dict(cache=cache(), starts=ST, lengths=LEN, T=5, k=X, k_token=32, k_head=16, v=R, v_token=32, v_head=16, q=Q,
              q_token=64, q_head=16, Hq=4, xt=BF16, cos_sin=CS, P=9, R=8, pairs=0, norm=1, k_gain=G, q_gain=G, gt=BF16,
              eps=1e-6, q_out=QO, yt=BF16, stream=None)


def test_kv_append():
    expect("q8_kv_append", APPEND, [(s, {"cache": c}) for s, c in BAD_CACHES] + [
        (E, {p: None}) for p in ("cache", "starts", "lengths", "k", "v", "q", "q_out")] + [
        (E, {p: -1}) for p in ("T", "k_token", "k_head", "v_token", "v_head", "q_token", "q_head", "Hq", "P", "R")] + [
        (E, {"xt": 2}), (E, {"gt": 2}), (E, {"yt": 2}), (E, {"pairs": 2}), (E, {"eps": -1.0}), (E, {"eps": float("nan")}),
        (E, {"k": K + 2047}), (E, {"v": VS + 7}), (E, {"q": V}), (E, {"cos_sin": K}), (E, {"k_gain": KS}),
        (E, {"q_out": X}), (E, {"q_out": K + 16}), (E, {"starts": KS + 4}), (E, {"lengths": V}), (E, {"q_out": Q + 64}),
        (E, {"cache": cache(v=K + 16)}), (E, {"cache": cache(k_scale=VS + 7)}), (E, {"cache": cache(pages=K)}),
        (SH, {"R": 7}), (SH, {"R": 18}), (SH, {"R": 0}), (SH, {"P": 0}), (SH, {"P": 2 ** 30 + 1}), (SH, {"T": 2 ** 31}),
        (SH, {"Hq": 2 ** 30}), (SH, {"k_token": 2 ** 60}), (q4.OK, {"T": 0}), (q4.OK, {"cache": cache(sequences=0)}),
        (q4.OK, {"T": 0, "Hq": 0, "q": None, "q_out": None}), (q4.OK, {"T": 0, "cos_sin": None, "R": 7, "P": 0}),
        (q4.OK, {"T": 0, "norm": 0, "eps": -1.0, "k_gain": None, "q_gain": None})])


def test_kv_read():
    good = dict(cache=cache(), starts=ST, lengths=LEN, T=5, k_out=X, v_out=Y, yt=F32, stream=None)
    expect("q8_kv_read", good, [(s, {"cache": c}) for s, c in BAD_CACHES] + [
        (E, {p: None}) for p in ("cache", "starts", "lengths", "k_out", "v_out")] + [
        (E, {"T": -1}), (E, {"yt": 2}), (E, {"k_out": K}), (E, {"v_out": VS}), (E, {"v_out": X + 639}), (E, {"k_out": PG}),
        (E, {"k_out": ST}), (E, {"v_out": LEN}), (SH, {"T": 2 ** 31}), (q4.OK, {"T": 0}),
        (q4.OK, {"cache": cache(sequences=0)})])


ATTENTION = dict(q=Q, q_token=64, q_head=16, xt=BF16, cache=cache(), starts=ST, lengths=LEN, T=5, Hq=4, max_len=128,
                 scale=0.25, window=0, sinks=0, y=Y, yt=BF16, ws=WS, ws_bytes=0, stream=None)


def test_attention():
    expect("q8_attention", ATTENTION, [(s, {"cache": c}) for s, c in BAD_CACHES] + [
        (E, {p: None}) for p in ("q", "cache", "starts", "lengths", "y")] + [
        (E, {p: -1}) for p in ("q_token", "q_head", "T", "Hq", "max_len", "window", "sinks")] + [
        (E, {"xt": 2}), (E, {"yt": -1}), (E, {"scale": float("inf")}), (E, {"scale": float("nan")}), (E, {"ws": WS + 16}),
        (E, {"y": Q + 639}), (E, {"y": K}), (E, {"y": V + 2032}), (E, {"y": KS}), (E, {"y": PG}), (E, {"y": ST}),
        (E, {"y": LEN}), (SH, {"Hq": 3}), (SH, {"Hq": 2 ** 30}), (SH, {"T": 2 ** 31}), (SH, {"max_len": 2 ** 31}),
        (SH, {"q_token": 2 ** 60}), (q4.OK, {"T": 0}), (q4.OK, {"Hq": 0}), (q4.OK, {"cache": cache(sequences=0)})])


def test_attention_workspace():
    f = q4.q8_attention_workspace
    assert f(1, 1, 32, 8, 128, 0) == 0
    need = f(1, 1, 32, 8, 128, 131072)
    assert need > 0
    # the split of the keys, and so the workspace, goes by the keys that a row can see
    assert f(1, 1, 32, 8, 128, 131072, 128, 4) <= need
    for bad in ((0, 1, 32, 8, 128, 9), (1, 0, 32, 8, 128, 9), (1, 1, 30, 8, 128, 9), (1, 1, 32, 8, 24, 9),
                (1, 1, 32, 8, 128, -1), (2 ** 31, 1, 32, 8, 128, 9), (1, 1, 32, 8, 128, 2 ** 31)):
        assert f(*bad) == 0
    good = dict(ATTENTION, T=1, Hq=32, cache=cache(heads=8, D=128, n_pages=1, page=16, table=8192, sequences=1,
                                                   k=BASE, v=BASE + 16384, k_scale=BASE + 32768, v_scale=BASE + 32776,
                                                   pages=BASE + 36864),
                max_len=131072, q=BASE + 73728, y=BASE + 90112, starts=BASE + 106496, lengths=BASE + 106504,
                ws=BASE + 110592)
    expect("q8_attention", good, [(E, {"ws_bytes": need - 1}), (E, {"ws": None, "ws_bytes": need}),
                                  (E, {"ws": BASE, "ws_bytes": need}), (E, {"ws": BASE + 90112, "ws_bytes": need})])


def test_the_binding_takes_no_host_tensors():
    x = torch.zeros(2, 16)
    c = q4.q8_kv_cache(2, 1, 16, 16, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    h = torch.zeros(2, 1, 16)
    for bad in (lambda: q4.q8_rmsnorm_rows(x), lambda: q4.q8_kv_append(c, i[None], torch.zeros(2).int(), i, h, h),
                lambda: q4.q8_kv_read(c, i[None], torch.zeros(2).int(), i, 2),
                lambda: q4.q8_attention(h, c, i[None], torch.zeros(2).int(), i)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        q4.q8_kv_cache(2, 1, 24, 16, device="cpu")


def test_limits_of_the_cache():
    """Tokens of a table, heads, and workgroups of a launch."""
    many = cache(heads=64)
    for status, c, T in ((SH, cache(table=2 ** 26), 5), (SH, cache(table=2 ** 26 - 63), 5), (SH, cache(heads=65537), 5),
                         (SH, many, 2 ** 31 - 1)):
        assert call("q8_kv_append", dict(APPEND, cache=c, T=T, Hq=0, q=None, q_out=None)) == status
        assert call("q8_kv_read", dict(cache=c, starts=ST, lengths=LEN, T=T, k_out=X, v_out=Y, yt=F32, stream=None)) == status
    for c in (cache(table=2 ** 26), cache(table=2 ** 26 - 63), cache(heads=65537)):
        assert call("q8_attention", dict(ATTENTION, cache=c)) == SH

"""Argument checks of the MX FP4 and query/key calls on the CPU: a refused
call returns its status before any device call and writes nothing."""
import ctypes

import numpy as np
import pytest

import int4_dequantize_matmul_amd as q4

BUF = (ctypes.c_uint8 * (1 << 16))()
BASE = (ctypes.addressof(BUF) + 255) & ~255
X, C, S, W, SW, Y, WS = (BASE + 4096 * i for i in range(7))
F32, BF16 = 0, 1


@pytest.fixture(autouse=True)
def _canary():
    ctypes.memset(BUF, 0xA5, len(BUF))
    yield
    assert bytes(BUF) == b"\xA5" * len(BUF)


def expect(name, good, changes):
    """`good` with one argument changed at a time gives the status."""
    f = getattr(q4.raw(), name)
    for status, change in changes:
        args = dict(good, **change)
        assert f(*args.values()) == status, (name, change)


E, SH = q4.EINVAL, q4.ESHAPE


def test_quantize_rows():
    good = dict(x=X, xt=BF16, M=2, K=40, codes=C, scales=S, stream=None)
    expect("q4_mx_quantize_rows", good, [
        (E, {"x": None}), (E, {"codes": None}), (E, {"scales": None}), (E, {"M": -1}), (E, {"K": -1}),
        (E, {"xt": 2}), (E, {"xt": -1}), (E, {"codes": C + 8}), (E, {"codes": X}), (E, {"scales": X + 159}),
        (E, {"scales": C + 63}), (SH, {"M": 2 ** 31}), (SH, {"K": 2 ** 31}),
        (q4.OK, {"M": 0}), (q4.OK, {"K": 0})])


def test_dequantize_rows():
    good = dict(codes=C, scales=S, M=2, K=40, y=Y, yt=F32, stream=None)
    expect("q4_mx_dequantize_rows", good, [
        (E, {"codes": None}), (E, {"scales": None}), (E, {"y": None}), (E, {"M": -1}), (E, {"K": -3}),
        (E, {"yt": 7}), (E, {"codes": C + 4}), (E, {"y": C + 48}), (E, {"y": S}), (SH, {"M": 2 ** 31}),
        (SH, {"K": 2 ** 31}), (q4.OK, {"M": 0}), (q4.OK, {"K": 0})])


def test_linear_w4a4():
    good = dict(xq=X, sx=S, wq=W, sw=SW, y=Y, yt=BF16, M=2, N=3, K=64, stream=None)
    expect("q4_linear_w4a4_mx", good, [
        (E, {p: None}) for p in ("xq", "sx", "wq", "sw", "y")] + [
        (E, {"M": -1}), (E, {"N": -1}), (E, {"K": -1}), (E, {"yt": 2}), (E, {"xq": X + 1}), (E, {"wq": W + 8}),
        (E, {"y": X + 60}), (E, {"y": S + 3}), (E, {"y": W + 95}), (E, {"y": SW + 5}),
        (SH, {"M": 16 * 65535 + 1}), (SH, {"N": 2 ** 31}), (SH, {"K": 2 ** 31}), (q4.OK, {"M": 0}),
        (q4.OK, {"N": 0})])


def test_linear_w4a4_dynamic():
    need = q4.q4_w4a4_mx_dynamic_workspace(2, 64)
    assert need == 512 and q4.q4_w4a4_mx_dynamic_workspace(17, 33) == 17 * 32 + 224 + 256
    assert q4.q4_w4a4_mx_dynamic_workspace(-1, 5) == 0 and q4.q4_w4a4_mx_dynamic_workspace(3, 0) == 0
    good = dict(x=X, xt=F32, wq=W, sw=SW, y=Y, yt=F32, M=2, N=3, K=64, ws=WS, n=need, stream=None)
    expect("q4_linear_w4a4_mx_dynamic", good, [
        (E, {p: None}) for p in ("x", "wq", "sw", "y", "ws")] + [
        (E, {"M": -1}), (E, {"N": -1}), (E, {"K": -1}), (E, {"xt": 2}), (E, {"yt": 2}), (E, {"wq": W + 8}),
        (E, {"ws": WS + 128}), (E, {"n": need - 1}), (E, {"ws": X + 256}), (E, {"y": WS + 500}),
        (E, {"y": X + 511}), (E, {"sw": WS}), (SH, {"M": 16 * 65535 + 1}), (SH, {"N": 2 ** 31}),
        (SH, {"K": 2 ** 31}), (q4.OK, {"M": 0}), (q4.OK, {"N": 0})])


def test_linear_w4a16():
    good = dict(x=X, wq=W, sw=SW, y=Y, yt=BF16, M=2, N=3, K=33, stream=None)
    expect("q4_linear_w4a16_mx", good, [
        (E, {p: None}) for p in ("x", "wq", "sw", "y")] + [
        (E, {"M": -1}), (E, {"N": -1}), (E, {"K": -1}), (E, {"yt": 9}), (E, {"wq": W + 2}), (E, {"y": X + 131}),
        (E, {"y": W}), (E, {"y": SW + 5}), (SH, {"M": 16 * 65535 + 1}), (SH, {"N": 2 ** 31}),
        (SH, {"K": 2 ** 31}), (q4.OK, {"M": 0}), (q4.OK, {"N": 0})])


def test_qk_norm_rope():
    gq, gk, pos, cs = BASE + 28672, BASE + 29696, BASE + 30720, BASE + 31744
    good = dict(q=X, qt=32, qh=16, k=X + 2048, kt=16, kh=16, xt=F32, gq=gq, gk=gk, gt=F32, pos=pos, cs=cs, qo=Y,
                ko=WS, yt=F32, T=2, Hq=2, Hk=1, D=16, R=8, P=5, eps=1e-6, pairs=0, stream=None)
    nan = float("nan")
    expect("q4_qk_norm_rope", good, [
        (E, {p: None}) for p in ("q", "k", "pos", "cs", "qo", "ko")] + [
        (E, {p: -1}) for p in ("T", "Hq", "Hk", "D", "R", "P", "qt", "qh", "kt", "kh", "xt", "gt", "yt", "pairs")] + [
        (E, {"xt": 2}), (E, {"gt": 2}), (E, {"yt": 2}), (E, {"pairs": 2}), (E, {"eps": -1.0}), (E, {"eps": nan}),
        (E, {"qo": X + 252}), (E, {"ko": X + 2048}), (E, {"qo": gq}), (E, {"ko": gk + 60}), (E, {"qo": pos + 8}),
        (E, {"ko": cs + 156}), (E, {"ko": Y + 255}),
        (SH, {"D": 15}), (SH, {"D": 0}), (SH, {"D": 65538}), (SH, {"R": 7}), (SH, {"R": 0}), (SH, {"R": 18}),
        (SH, {"P": 0}), (SH, {"T": 2 ** 31}), (SH, {"Hq": 2 ** 31}), (SH, {"T": 2 ** 30}),
        (SH, {"qt": 2 ** 59}), (SH, {"kt": 2 ** 59}),
        (q4.OK, {"T": 0}), (q4.OK, {"Hq": 0, "Hk": 0})])


def test_python_checks_need_device_tensors():
    import torch
    x = torch.zeros(2, 32)
    u = torch.zeros(2, 16, dtype=torch.uint8)
    for call in (lambda: q4.q4_mx_quantize_rows(x), lambda: q4.q4_mx_dequantize_rows(u, u),
                 lambda: q4.q4_linear_w4a4_mx(u, u, u, u), lambda: q4.q4_linear_w4a4_mx_dynamic(x, u, u),
                 lambda: q4.q4_linear_w4a16_mx(x, u, u),
                 lambda: q4.q4_qk_norm_rope(x[:, None], None, None, None, x, x)):
        with pytest.raises(TypeError):
            call()
    assert np.all(u.numpy() == 0)


class _Recorder:
    """In the place of the library: every call is noted and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


def test_a_workspace_has_to_be_contiguous_device_memory(monkeypatch):
    """A host tensor's address, or a strided view's, never reaches the kernels."""
    import torch
    lib = _Recorder()
    monkeypatch.setattr(q4, "_dev", lambda t, *rest: t)       # host tensors stand in for the other arguments
    monkeypatch.setattr(q4, "_direct", lambda: None)
    monkeypatch.setattr(q4, "_lib", lambda: lib)
    monkeypatch.setattr(q4, "_stream", lambda t: 0)
    x, w, s = torch.zeros(20, 32), torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.uint8)
    for ws in (torch.zeros(4096, dtype=torch.uint8), np.zeros(4096, np.uint8), 4096):
        with pytest.raises(TypeError):
            q4.q4_linear_w4a4_mx_dynamic(x, w, s, ws=ws)
    assert not lib.calls

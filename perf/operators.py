"""What is measured of the microscaled (MX) FP4 operators and of the head
normalisation with rotation: the cases, their inputs, and each operator in
plain torch form.

MX FP4: a row of K numbers is cut into blocks of 32 columns (the last one may
be short).  A block is 16 bytes of E2M1 codes (low nibble = even column;
columns past K hold code 0) and one E8M0 byte b that stands for 2^(b - 127).
The shared exponent is floor(log2(max|x|)) - 2, the codes are rounded to the
nearest (ties to even) and saturate at +-6.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = "cuda:0"
else:
    DEV = "cpu"

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's activations before a 2048-wide linear: latency
        {"name": "quantize_token", "op": "quantize", "M": 1, "K": 2048, "type": "bf16"},
        # a weight matrix quantized at load time, its K no multiple of a block
        {"name": "quantize_weight_odd", "op": "quantize", "M": 2048, "K": 1023, "type": "f32"},
        # a prompt's activations in front of the down projection
        {"name": "quantize_prompt", "op": "quantize", "M": 2048, "K": 5632, "type": "bf16"},
        # one token through the wide decode linear, activations quantized in the call
        {"name": "w4a4_token", "op": "w4a4", "M": 1, "N": 13312, "K": 2048, "type": "bf16", "given": False},
        # a ragged batch of requests through a square projection, float32 result
        {"name": "w4a4_batch_ragged", "op": "w4a4", "M": 77, "N": 2049, "K": 2080, "type": "f32", "given": False},
        # a prompt through the wide linear, activations quantized before (one set for several linears)
        {"name": "w4a4_prompt", "op": "w4a4", "M": 2048, "N": 13312, "K": 2048, "type": "bf16", "given": True},
        # a long prompt through the down projection
        {"name": "w4a4_prompt_long", "op": "w4a4", "M": 8192, "N": 2048, "K": 5632, "type": "bf16", "given": False},
        # one token, weight-only
        {"name": "w4a16_token", "op": "w4a16", "M": 1, "N": 13312, "K": 2048, "type": "bf16"},
        # a small ragged batch, float32 result
        {"name": "w4a16_batch_ragged", "op": "w4a16", "M": 13, "N": 5631, "K": 2048, "type": "f32"},
        # a prompt, weight-only
        {"name": "w4a16_prompt", "op": "w4a16", "M": 2048, "N": 13312, "K": 2048, "type": "bf16"},
        # one token's queries and keys (2048 = 16 heads of 128): latency
        {"name": "qk_token", "op": "qk", "T": 1, "Hq": 16, "Hk": 16, "D": 128, "R": 128, "type": "bf16",
         "pairs": "halves", "positions": 32768},
        # a long prompt with shared key heads
        {"name": "qk_prompt", "op": "qk", "T": 8190, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "type": "bf16",
         "pairs": "halves", "positions": 16384},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "w4a4", "w4a16", "qk"))
    t = rng.choice(("bf16", "f32"))
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 2048), "K": _log(rng, 1, 5632), "type": t}
    if op == "qk":
        D = 2 * rng.randint(8, 128)
        if rng.random() < 0.6:
            D = rng.choice((64, 96, 128, 256))
        R = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
        Hk = rng.randint(1, 8)
        return {"op": op, "T": _log(rng, 1, 4096), "Hq": Hk * rng.randint(1, 4), "Hk": Hk, "D": D, "R": R,
                "type": t, "pairs": rng.choice(("halves", "neighbours")), "positions": _log(rng, 64, 32768)}
    # products: the columns of K are whole blocks in most models, but not in all
    K = 32 * _log(rng, 2, 128) if rng.random() < 0.75 else _log(rng, 33, 4096)
    c = {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 16, 8192), "K": K, "type": t}
    if op == "w4a4":
        c["given"] = rng.random() < 0.4
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pad(x):
    """float32 rows with zeros up to whole blocks, as [M, blocks, 32]."""
    M, K = x.shape
    B = (K + 31) // 32
    x = x.float()
    if 32 * B != K:
        x = torch.cat([x, x.new_zeros(M, 32 * B - K)], 1)
    return x.reshape(M, B, 32)


def _quantize(x):
    """Rows -> (E2M1 codes 0..15 as [M, blocks, 32], scale bytes [M, blocks])."""
    v = _pad(x)
    top = v.abs().amax(2)
    _, e = torch.frexp(top)                      # top = f 2^e, f in [0.5, 1): floor(log2 top) = e - 1
    byte = torch.where(top > 0, (e - 3 + 127).clamp(0, 254), torch.zeros_like(e))
    # times 2^(127 - byte), in two exact steps, since the factor can pass float32's range
    n = 127 - byte
    half = torch.div(n, 2, rounding_mode="floor")
    u = torch.ldexp(torch.ldexp(v, half[..., None]), (n - half)[..., None])
    a = u.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * torch.signbit(u).int()
    return code.to(torch.uint8), byte.to(torch.uint8)


def _bytes(code):
    """Codes [M, blocks, 32] -> packed bytes [M, 16 blocks]."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(code.shape[0], -1).contiguous()


def _values(packed, byte):
    """Packed rows and scale bytes -> float32 values [M, 32 blocks]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    code = torch.stack((packed & 15, packed >> 4), 2).reshape(packed.shape[0], -1, 32)
    v = torch.ldexp(table[code.int()], byte.int()[..., None] - 127)
    return v.reshape(packed.shape[0], -1)


def _activations(gen, M, K, dtype):
    """Normal rows whose columns differ in size by a few times, one in 64 of them by far."""
    col = torch.exp(0.5 * torch.randn(K, generator=gen, device=DEV))
    col = torch.where(torch.rand(K, generator=gen, device=DEV) < 1 / 64, 8 * col, col)
    return (torch.randn(M, K, generator=gen, device=DEV) * col).to(dtype)


def _table(P, R):
    """cos and sin of position times 10000^(-2 i / R), float32 [P, R], the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    a = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "quantize":
        x = _activations(gen, case["M"], case["K"], torch.float32)
        dead = torch.rand(x.shape[0], (x.shape[1] + 31) // 32, generator=gen, device=DEV) < 0.01
        s["x"] = x.masked_fill(dead.repeat_interleave(32, 1)[:, :x.shape[1]], 0).to(t)
    elif case["op"] in ("w4a4", "w4a16"):
        W = 0.02 * torch.randn(case["N"], case["K"], generator=gen, device=DEV)
        code, s["sw"] = _quantize(W)
        s["wq"] = _bytes(code)
        # float32 results come with float32 activations where the call quantizes them itself
        x = _activations(gen, case["M"], case["K"], t if case["op"] == "w4a4" else torch.bfloat16)
        if case.get("given"):
            code, s["sx"] = _quantize(x)
            s["xq"] = _bytes(code)
        else:
            s["x"] = x
    else:
        T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
        # the product of the fused projection: queries, keys and values side by side
        s["qkv"] = torch.randn(T, (Hq + 2 * Hk) * D, generator=gen, device=DEV).to(t)
        s["q"] = s["qkv"][:, :Hq * D].view(T, Hq, D)
        s["k"] = s["qkv"][:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["wq"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(t)
        s["wk"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(t)
        # several requests in one batch, each from a position of its own
        P = case["positions"]
        begin = torch.randint(0, P, (1 + T // 512,), generator=gen, device=DEV)
        i = torch.arange(T, device=DEV)
        s["pos"] = (begin[i // 512] + i % 512) % P
        s["table"] = _table(P, R)
        s["eps"] = 1e-6
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _head(x, w, eps, c, s, R, pairs, dtype):
    """Norm of each head's row, times w, then the rotation of its first R columns."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + eps) * w.float()
    r, rest = y[..., :R], y[..., R:]
    if pairs == "halves":
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), 2)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), 3).reshape(r.shape)
    return torch.cat((r, rest), 2).to(dtype)


def run(state):
    case = state["case"]
    t = TYPES[case["type"]]
    if own:
        import int4_dequantize_matmul_amd as q4
        if case["op"] == "quantize":
            packed, scales = q4.q4_mx_quantize_rows(state["x"])
            return q4.q4_mx_dequantize_rows(packed, scales, case["K"], case["type"])
        if case["op"] == "w4a4":
            if case["given"]:
                return q4.q4_linear_w4a4_mx(state["xq"], state["sx"], state["wq"], state["sw"], case["type"])
            return q4.q4_linear_w4a4_mx_dynamic(state["x"], state["wq"], state["sw"], case["type"])
        if case["op"] == "w4a16":
            return q4.q4_linear_w4a16_mx(state["x"], state["wq"], state["sw"], case["type"])
        return q4.q4_qk_norm_rope(state["q"], state["k"], state["wq"], state["wk"], state["pos"], state["table"],
                                  state["eps"], case["pairs"])
    if case["op"] == "quantize":
        code, byte = _quantize(state["x"])
        return _values(_bytes(code), byte)[:, :case["K"]].to(t)
    if case["op"] == "w4a4":
        if case["given"]:
            x = _values(state["xq"], state["sx"])
        else:
            code, byte = _quantize(state["x"])
            x = _values(_bytes(code), byte)
        return torch.matmul(x, _values(state["wq"], state["sw"]).t()).to(t)
    if case["op"] == "w4a16":
        return torch.matmul(state["x"].float(), _values(state["wq"], state["sw"])[:, :case["K"]].t()).to(t)
    R = case["R"]
    cs = state["table"][state["pos"]][:, None, :]
    c, s = cs[..., :R // 2], cs[..., R // 2:]
    return (_head(state["q"], state["wq"], state["eps"], c, s, R, case["pairs"], t),
            _head(state["k"], state["wk"], state["eps"], c, s, R, case["pairs"], t))


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        # in, the packed form, and out again
        return {"bytes": 2 * M * K * size + M * ((K + 31) // 32) * 17, "flops": 4 * M * K}
    if case["op"] in ("w4a4", "w4a16"):
        M, N, K = case["M"], case["N"], case["K"]
        row = 17 * ((K + 31) // 32)
        x = M * row if case.get("given") else M * K * (2 if case["op"] == "w4a16" else size)
        return {"bytes": x + N * row + M * N * size, "flops": 2 * M * N * K}
    T, H, D, R = case["T"], case["Hq"] + case["Hk"], case["D"], case["R"]
    return {"bytes": 2 * T * H * D * size + T * (R * 4 + 8) + 2 * D * size, "flops": T * H * (4 * D + 3 * R)}


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_rounded(x):
    """Rows rounded to MX FP4, float64 [M, K]: the step of E2M1 at a value is
    half up to 2, one up to 4, two above; torch.round takes ties to even."""
    x = x.double()
    M, K = x.shape
    out = torch.empty_like(x)
    whole = K // 32 * 32
    for lo, hi, n in ((0, whole, 32), (whole, K, K - whole)):
        if hi == lo or M == 0:
            continue
        v = x[:, lo:hi].reshape(M, -1, n)
        top = v.abs().max(2, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        e = torch.where(torch.exp2(e) > top, e - 1, e)          # a log2 rounded up to the next power
        e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)     # or down below it
        unit = torch.exp2(torch.clamp(e - 2, min=-127.0))
        u = v / unit
        step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0)).double()
        u = torch.clamp(torch.round(u / step) * step, -6.0, 6.0)
        out[:, lo:hi] = (u * unit).reshape(M, hi - lo)
    return out


def _exact_decoded(packed, byte, K):
    """Packed rows from the bit fields: sign, two exponent bits, one mantissa bit."""
    code = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.int64, device=packed.device)
    code[:, 0::2] = packed % 16
    code[:, 1::2] = packed // 16
    sign = 1 - 2 * (code // 8)
    ex, m = code // 2 % 4, code % 2
    mag = torch.where(ex == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2(ex.double() - 1))
    scale = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)
    return (sign * mag * scale)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_rounded(s["x"])
    if case["op"] in ("w4a4", "w4a16"):
        K = case["K"]
        w = _exact_decoded(s["wq"], s["sw"], K)
        if case["op"] == "w4a16":
            x = s["x"].double()
        elif case["given"]:
            x = _exact_decoded(s["xq"], s["sx"], K)
        else:
            x = _exact_rounded(s["x"])
        return x @ w.t().contiguous()
    R, table = case["R"], s["table"].double()
    rows = table.index_select(0, s["pos"])
    angle = torch.complex(rows[:, :R // 2], rows[:, R // 2:])[:, None, :]
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        y = y / torch.sqrt((y * y).sum(2, keepdim=True) / case["D"] + s["eps"]) * w.double()
        if case["pairs"] == "halves":
            z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * angle
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * angle
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        outs.append(y)
    return tuple(outs)

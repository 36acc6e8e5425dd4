"""What is measured of the operators around a decoder layer's 8-bit state: the
normalisation of rows to int8 codes, the paged 8-bit cache of keys and values,
and the attention that reads it.  The cases, their inputs, and each operator in
plain torch form.

Rows: h = x + r, u = h g, codes = round(127 u / max|u|) (ties to even), scale =
max|u| / (127 sqrt(mean(h^2) + eps)).

Cache: a page of a key head is cut into blocks of 16 tokens.  A block of keys
is int8 [D/16, 16 tokens, 16 columns], a block of values int8 [D, 16 tokens],
each under one scale byte b that stands for 2^(b - 127): the smallest power of
two with max|x| <= 127 scale.  Where tokens join a block that has some, its
scale only grows, and the codes it has are rounded to the new one.

Attention: the last n of a sequence's L tokens are queries; the query at
position p sees the keys j <= p with j > p - window or j < sinks.
"""
import math
import random

import torch

own = False

if torch.cuda.is_available():
    DEV = "cuda:0"
else:
    DEV = "cpu"

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's row in front of a 2048-wide layer's linears: latency
        {"name": "norm_token", "op": "norm", "M": 1, "K": 2048, "type": "bf16", "residual": True},
        # a ragged batch of float32 rows of odd width, without a residual
        {"name": "norm_batch_odd", "op": "norm", "M": 77, "K": 5631, "type": "f32", "residual": False},
        # a long prompt's rows, the residual stream updated on the way
        {"name": "norm_prompt", "op": "norm", "M": 8192, "K": 2048, "type": "bf16", "residual": True},
        # one token of one request joins a block that has some, heads normalised: latency
        {"name": "append_token", "op": "append", "N": 1, "new": 1, "context": 1000, "ragged": False, "Hq": 16, "Hk": 16,
         "D": 128, "R": 128, "page": 64, "type": "bf16", "norm": True, "pairs": "halves"},
        # a batch of requests, one float32 token each, half of the head rotated as neighbours
        {"name": "append_batch", "op": "append", "N": 61, "new": 1, "context": 2000, "ragged": True, "Hq": 24, "Hk": 6,
         "D": 80, "R": 40, "page": 16, "type": "f32", "norm": False, "pairs": "neighbours"},
        # four prompts, the longer part of them new, shared key heads
        {"name": "append_prompt", "op": "append", "N": 4, "new": 4095, "context": 5000, "ragged": True, "Hq": 32, "Hk": 8,
         "D": 128, "R": 128, "page": 64, "type": "bf16", "norm": True, "pairs": "halves"},
        # one token of one request over a short context: latency
        {"name": "attend_token", "op": "attend", "N": 1, "new": 1, "context": 1023, "ragged": False, "Hq": 16, "Hk": 16,
         "D": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16"},
        # one token over a very long context: the cache's bytes
        {"name": "attend_long", "op": "attend", "N": 1, "new": 1, "context": 131071, "ragged": False, "Hq": 32, "Hk": 8,
         "D": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16"},
        # a batch of requests of all lengths, one token each
        {"name": "attend_batch", "op": "attend", "N": 64, "new": 1, "context": 8192, "ragged": True, "Hq": 32, "Hk": 8,
         "D": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16"},
        # long contexts with a window and first tokens that stay visible, float32
        {"name": "attend_window", "op": "attend", "N": 16, "new": 1, "context": 32768, "ragged": True, "Hq": 16, "Hk": 4,
         "D": 64, "page": 32, "window": 1024, "sinks": 4, "type": "f32"},
        # chunks of several prompts behind what they have in the cache, float32, three query heads a key head
        {"name": "attend_chunks", "op": "attend", "N": 5, "new": 333, "context": 2100, "ragged": True, "Hq": 12, "Hk": 4,
         "D": 96, "page": 128, "window": 700, "sinks": 3, "type": "f32"},
        # a long prompt
        {"name": "attend_prompt", "op": "attend", "N": 1, "new": 8190, "context": 8190, "ragged": False, "Hq": 32, "Hk": 8,
         "D": 128, "page": 64, "window": 0, "sinks": 0, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "attend", "attend"))
    t = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 1, 5632), "type": t, "residual": rng.random() < 0.7}
    Hk = rng.randint(1, 8)
    c = {"op": op, "Hq": Hk * rng.randint(1, 8), "Hk": Hk, "D": rng.choice((64, 64, 128, 128, 128, 16 * rng.randint(1, 16))),
         "page": 16 << rng.randint(0, 4), "type": t, "ragged": rng.random() < 0.7}
    if op == "append":
        c["new"] = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        c["N"] = _log(rng, 1, 128 if c["new"] == 1 else 4)
        c["context"] = c["new"] + _log(rng, 1, 2048)
        c["R"] = c["D"] if rng.random() < 0.6 else 2 * rng.randint(1, c["D"] // 2)
        c["norm"] = rng.random() < 0.5
        c["pairs"] = rng.choice(("halves", "neighbours"))
        return c
    if rng.random() < 0.6:
        c["N"], c["new"] = _log(rng, 1, 64), 1
        c["context"] = min(_log(rng, 1, 65536), 262144 // c["N"])
    else:
        c["N"], c["new"] = _log(rng, 1, 6), _log(rng, 2, 2048)
        c["context"] = c["new"] + _log(rng, 1, 2048) - 1
        c["N"] = max(1, min(c["N"], (1 << 30) // (c["new"] * c["context"] * c["Hq"])))
    windowed = rng.random() < 0.4
    c["window"] = _log(rng, 1, 4096) if windowed else 0
    c["sinks"] = rng.choice((0, 1, 4, 17)) if windowed else 0
    return c


def _sequences(case):
    """(tokens, new ones among them) of each sequence: part of the case, not of the seed."""
    N, new, context = case["N"], case["new"], case["context"]
    if not case["ragged"]:
        return [(context, new)] * N
    rng = random.Random(N * 1000003 + new * 1009 + context)
    got = [(context, new)]                    # the longest one
    while len(got) < N:
        n = rng.randint(1, new)
        got.append((n + rng.randint(0, context - new), n))
    rng.shuffle(got)
    return got


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _starts(counts):
    return torch.tensor([0] + counts, device=DEV).cumsum(0).int()


def _table(P, R):
    """cos and sin of position times 10000^(-2 i / R), float32 [P, R], the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    a = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _pool(gen, case, s):
    """The cache as a run of such requests leaves it: pages in any order, every
    block's largest code between 64 and 127, blocks and heads of several sizes."""
    Hk, D, page = case["Hk"], case["D"], case["page"]
    seqs = _sequences(case)
    width = max(-(-L // page) for L, _ in seqs)
    used = [-(-L // page) for L, _ in seqs]
    P = sum(used) + 2
    order = torch.randperm(P, generator=gen, device=DEV)
    i = torch.arange(width, device=DEV)[None, :]
    first = _starts(used)[:-1].long()[:, None]
    table = order[(first + i).clamp(max=P - 1)]
    # entries past a sequence's last page mean nothing
    s["pages"] = torch.where(i < torch.tensor(used, device=DEV)[:, None], table, -1).int().contiguous()
    s["lengths"] = torch.tensor([L for L, _ in seqs], device=DEV, dtype=torch.int32)
    s["starts"] = _starts([n for _, n in seqs])
    s["T"] = sum(n for _, n in seqs)
    blocks = page // BLOCK
    for name, shape in (("k", (P, Hk, blocks, D // 16, 16, 16)), ("v", (P, Hk, blocks, D, 16))):
        n = P * Hk * blocks
        code = torch.empty(n, 16 * D, dtype=torch.int8, device=DEV)
        for a in range(0, n, 1 << 16):        # by parts, so that the float32 form stays small
            x = torch.randn(min(n - a, 1 << 16), 16 * D, generator=gen, device=DEV)
            top = 64 + 63 * torch.rand(x.shape[0], 1, generator=gen, device=DEV)
            code[a:a + (1 << 16)] = torch.round(x * (top / x.abs().amax(1, keepdim=True))).to(torch.int8)
        s[name] = code.view(shape)
        s[name + "_scale"] = (121 + torch.randint(-1, 2, (P, Hk, blocks), generator=gen, device=DEV)).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        # columns of several sizes, one in 64 of them by far, as a residual stream has them
        col = torch.exp(0.5 * torch.randn(K, generator=gen, device=DEV))
        col = torch.where(torch.rand(K, generator=gen, device=DEV) < 1 / 64, 8 * col, col)
        s["x"] = (torch.randn(M, K, generator=gen, device=DEV) * col).to(t)
        s["residual"] = (torch.randn(M, K, generator=gen, device=DEV) * col).to(t) if case["residual"] else None
        s["gain"] = (1 + 0.1 * torch.randn(K, generator=gen, device=DEV)).to(t)
        s["eps"] = 1e-6
        return s
    _pool(gen, case, s)
    T, Hq, Hk, D = s["T"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "append":
        # the product of the fused projection: queries, keys and values side by side
        qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=gen, device=DEV).to(t)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["new_k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["new_v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        s["gain_q"], s["gain_k"], s["eps"] = None, None, None
        if case["norm"]:
            s["gain_q"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(t)
            s["gain_k"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEV)).to(t)
            s["eps"] = 1e-6
        s["table"] = _table(case["context"], case["R"])
        # what is read back: the new tokens and those that share their first block
        rows = [n + (L - n) % BLOCK for L, n in _sequences(case)]
        s["read_starts"], s["read_T"] = _starts(rows), sum(rows)
    else:
        # scores of a few units: some keys matter, most do little
        s["q"] = (4 * torch.randn(T, Hq, D, generator=gen, device=DEV)).to(t)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _places(starts, lengths, T):
    """Sequence and position of each of T rows."""
    row = torch.arange(T, device=DEV)
    seq = torch.searchsorted(starts, row.int(), right=True) - 1
    return seq, lengths[seq].long() - starts[seq + 1].long() + row


def _rotate(x, c, s, R, pairs):
    r, rest = x[..., :R], x[..., R:]
    if pairs == "halves":
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat((a * c - b * s, b * c + a * s), 2)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * c - b * s, b * c + a * s), 3).reshape(r.shape)
    return torch.cat((r, rest), 2)


def _heads(x, gain, eps, c, s, R, pairs):
    """Norm of each head's row, if there is one, and its rotation, in 64 bits:
    8-bit codes follow, and a code next to a border must not depend on a sum's order."""
    x = x.double()
    if eps is not None:
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + eps) * gain.double()
    return _rotate(x, c, s, R, pairs)


def _power(top):
    """The scale byte: the smallest 2^e with top <= 127 2^e."""
    m, e = torch.frexp(top)                   # top = m 2^e, m in [0.5, 1); 127 = 0.9921875 2^7
    return torch.where(top > 0, (torch.where(m <= 0.9921875, e - 7, e - 6) + 127).clamp(0, 254), 0)


def _append(s, name, x, seq, pos):
    """Rows x [T, Hk, D] (float64) at their sequences' positions into the cache."""
    case = s["case"]
    page, Hk, D = case["page"], case["Hk"], case["D"]
    codes, scales = s[name], s[name + "_scale"]
    blocks = page // BLOCK
    pg, blk, tok = s["pages"][seq, pos // page].long(), pos % page // BLOCK, pos % BLOCK
    where = pg * blocks + blk                 # a block's number in the pool
    top = torch.zeros(codes.shape[0] * blocks, Hk, dtype=torch.float64, device=DEV)
    top.scatter_reduce_(0, where[:, None].expand(-1, Hk), x.abs().amax(2), "amax")
    need = _power(top)[where]                 # the same for all rows of a block
    # blocks that had tokens before: those of the first new position, unless it begins one
    first = (s["lengths"] - (s["starts"][1:] - s["starts"][:-1])).long()[seq]
    joins = (first % BLOCK > 0) & (first // BLOCK == pos // BLOCK)
    old = scales[pg, :, blk].int()
    new = torch.where(joins[:, None], torch.maximum(old, need), need)
    shape = (-1, Hk) + (1,) * (codes.dim() - 3)
    grown = torch.round(torch.ldexp(codes[pg, :, blk].float(), (old - new).view(shape))).to(torch.int8)
    codes[pg, :, blk] = torch.where(joins.view((-1,) + (1,) * (codes.dim() - 2)), grown, codes[pg, :, blk])
    scales[pg, :, blk] = new.to(torch.uint8)
    code = torch.round(torch.ldexp(x, (127 - new)[..., None])).to(torch.int8)
    if name == "k":
        codes[pg, :, blk, :, tok] = code.view(-1, Hk, D // 16, 16)
    else:
        codes[pg, :, blk, :, tok] = code


def _read(s, name, seq, pos):
    """What the cache holds of positions pos of sequences seq: bf16 [T, Hk, D], exactly."""
    page, Hk, D = s["case"]["page"], s["case"]["Hk"], s["case"]["D"]
    pg, blk, tok = s["pages"][seq, pos // page].long(), pos % page // BLOCK, pos % BLOCK
    code = s[name][pg, :, blk, :, tok].reshape(-1, Hk, D)
    return torch.ldexp(code.float(), s[name + "_scale"][pg, :, blk].int()[..., None] - 127).bfloat16()


def _whole(s, name):
    """All positions of all sequences, float32 [N, Hk, positions, D]."""
    case = s["case"]
    N, width = s["pages"].shape
    pg = s["pages"].clamp(min=0).long()
    code, scale = s[name][pg], s[name + "_scale"][pg]        # [N, width, Hk, blocks, ...]
    code = code.transpose(4, 5)               # tokens first, then the columns (of a chunk, in keys)
    code = code.reshape(N, width, case["Hk"], -1, BLOCK, case["D"]).float()
    x = torch.ldexp(code, scale.int()[..., None, None] - 127)
    return x.permute(0, 2, 1, 3, 4, 5).reshape(N, case["Hk"], -1, case["D"])


def _attend(s):
    """Every sequence padded to the longest one, all heads at a time."""
    case = s["case"]
    N, Hq, Hk, D, n = case["N"], case["Hq"], case["Hk"], case["D"], case["new"]
    G = Hq // Hk
    seq, pos = _places(s["starts"], s["lengths"], s["T"])
    row = torch.arange(s["T"], device=DEV) - s["starts"][seq].long()
    q = torch.zeros(N, n, Hq, D, device=DEV)
    q[seq, row] = s["q"].float()
    q = q.view(N, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * n, D)
    k, v = _whole(s, "k"), _whole(s, "v")
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).view(N, Hk, G, n, -1)
    score *= D ** -0.5
    first = (s["lengths"] - (s["starts"][1:] - s["starts"][:-1])).long()
    p = (first[:, None] + torch.arange(n, device=DEV))[:, :, None]          # rows past a sequence's own are not read below
    j = torch.arange(score.shape[4], device=DEV)
    hidden = j > p
    if case["window"]:
        hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
    score.masked_fill_(hidden[:, None, None], float("-inf"))
    score -= score.amax(4, keepdim=True)
    score.exp_()
    total = score.sum(4, keepdim=True)
    y = torch.matmul(score.view(N, Hk, G * n, -1), v).view(N, Hk, G, n, D) / total
    return y.permute(0, 3, 1, 2, 4).reshape(N, n, Hq, D)[seq, row].to(TYPES[case["type"]])


def run(state):
    s = state
    case = s["case"]
    t = TYPES[case["type"]]
    if own:
        import int4_dequantize_matmul_amd as q4
        if case["op"] == "norm":
            codes, scale, total = q4.q8_rmsnorm_rows(s["x"], s["gain"], s["residual"], s["eps"])
            return (torch.mul(codes, scale[:, None]), scale) + ((total,) if case["residual"] else ())
        cache = q4.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            q = q4.q8_kv_append(cache, s["pages"], s["starts"], s["lengths"], s["new_k"], s["new_v"], s["q"],
                                s["table"], s["gain_k"], s["gain_q"], s["eps"], case["pairs"])
            return (q,) + tuple(q4.q8_kv_read(cache, s["pages"], s["read_starts"], s["lengths"], s["read_T"]))
        return q4.q8_attention(s["q"], cache, s["pages"], s["starts"], s["lengths"], window=case["window"],
                               sinks=case["sinks"], max_len=case["context"])
    if case["op"] == "norm":
        # in 64 bits: codes next to a border
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        u = h * s["gain"].double()
        top = u.abs().amax(1, keepdim=True)
        codes = torch.round(127 * u / torch.where(top > 0, top, 1))
        scale = (top * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) / 127).float()
        return (codes.float() * scale, scale[:, 0]) + ((h.float().to(t),) if case["residual"] else ())
    if case["op"] == "append":
        seq, pos = _places(s["starts"], s["lengths"], s["T"])
        R = case["R"]
        cs = s["table"][pos][:, None, :].double()
        c, sn = cs[..., :R // 2], cs[..., R // 2:]
        q = _heads(s["q"], s["gain_q"], s["eps"], c, sn, R, case["pairs"]).float().to(t)
        _append(s, "k", _heads(s["new_k"], s["gain_k"], s["eps"], c, sn, R, case["pairs"]), seq, pos)
        _append(s, "v", s["new_v"].double(), seq, pos)
        seq, pos = _places(s["read_starts"], s["lengths"], s["read_T"])
        return q, _read(s, "k", seq, pos), _read(s, "v", seq, pos)
    return _attend(s)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        # in (and the residual in and the sum out), codes out; the codes read and the values they stand for written
        return {"bytes": M * K * (size * (3 if case["residual"] else 1) + 1 + 1 + 4) + K * size + 8 * M, "flops": 8 * M * K}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    seqs = _sequences(case)
    T = sum(n for _, n in seqs)
    if case["op"] == "append":
        rows = sum(n + (L - n) % BLOCK for L, n in seqs)
        b = T * (Hq * 2 * size + Hk * 2 * (size + 1)) * D + T * case["R"] * 4      # q in and out, k and v in, codes out
        b += rows * Hk * D * 2 * (1 + 2)                                           # codes in, bf16 out
        return {"bytes": b, "flops": T * (Hq + 2 * Hk) * D * 4}
    keys = pairs = 0
    for L, n in seqs:
        w, k = case["window"], case["sinks"]
        first = max(0, L - n - w + 1) if w else 0
        keys += L - first + min(first, k)
        if not w:
            pairs += n * (L - n) + n * (n + 1) // 2
        else:
            pairs += sum(min(p + 1, w) + min(k, max(0, p + 1 - w)) for p in range(L - n, L))
    return {"bytes": keys * Hk * (2 * D + 1 / 8) + 2 * T * Hq * D * size, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_norm(s):
    case = s["case"]
    h = s["x"].double()
    if case["residual"]:
        h = h + s["residual"].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + s["eps"]) * s["gain"].double()
    step = torch.linalg.vector_norm(y, float("inf"), 1, keepdim=True) / 127
    # the codes from u = h g, whose quotients are those of y without y's roundings
    u = h * s["gain"].double()
    codes = torch.round(u * 127 / torch.linalg.vector_norm(u, float("inf"), 1, keepdim=True).clamp(min=1e-300))
    return (codes * step, step[:, 0]) + ((h,) if case["residual"] else ())


def _exact_head(x, gain, eps, rows, R, pairs):
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt((y * y).sum(2, keepdim=True) / y.shape[2] + eps) * gain.double()
    y = y.clone()
    angle = torch.complex(rows[:, :R // 2], rows[:, R // 2:])[:, None, :]
    if pairs == "halves":
        z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * angle
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * angle
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    return y


def _exact_step(top):
    """top [blocks, Hk, 1, 1] -> the power of two, by its definition."""
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 127))
    e = torch.where(127 * torch.exp2(e - 1) >= top, e - 1, e)
    e = torch.where(127 * torch.exp2(e) < top, e + 1, e)
    return torch.where(top > 0, torch.exp2(e.clamp(min=-127)), 2.0 ** -127)


def _exact_append(s):
    case = s["case"]
    Hk, D, R, page = case["Hk"], case["D"], case["R"], case["page"]
    at = s["starts"].tolist()
    pages = s["pages"].tolist()
    qs, ks, vs = [], [], []
    for i, (L, n) in enumerate(_sequences(case)):
        lo, hi, first = at[i], at[i + 1], L - n
        rows = s["table"][first:L].double()
        qs.append(_exact_head(s["q"][lo:hi], s["gain_q"], s["eps"], rows, R, case["pairs"]))
        new = {"k": _exact_head(s["new_k"][lo:hi], s["gain_k"], s["eps"], rows, R, case["pairs"]),
               "v": s["new_v"][lo:hi].double()}
        had = first % BLOCK
        for name, outs in (("k", ks), ("v", vs)):
            x = torch.zeros(-(-(had + n) // BLOCK) * BLOCK, Hk, D, dtype=torch.float64, device=DEV)
            x[had:had + n] = new[name]
            blocks = x.view(-1, BLOCK, Hk, D).transpose(1, 2)               # [blocks, Hk, 16, D]
            step = _exact_step(blocks.abs().amax((2, 3), keepdim=True))
            if had:
                pg, b = pages[i][first // page], first % page // BLOCK
                step[0] = torch.maximum(step[0], torch.exp2(s[name + "_scale"][pg, :, b].double() - 127)[:, None, None])
                code = s[name][pg, :, b].double()
                code = code.permute(0, 2, 1, 3).reshape(Hk, BLOCK, D) if name == "k" else code.transpose(1, 2)
                old = code * torch.exp2(s[name + "_scale"][pg, :, b].double() - 127)[:, None, None]
                blocks[0, :, :had] = old[:, :had]
            y = torch.round(blocks / step) * step
            outs.append(y.transpose(1, 2).reshape(-1, Hk, D)[:had + n])
    return torch.cat(qs), torch.cat(ks), torch.cat(vs)


def _exact_attend(s):
    case = s["case"]
    Hq, Hk, D, page = case["Hq"], case["Hk"], case["D"], case["page"]
    G = Hq // Hk
    at = s["starts"].tolist()
    y = torch.empty(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    for i, (L, n) in enumerate(_sequences(case)):
        pg = s["pages"][i, :-(-L // page)].long()
        p = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None, :]
        seen = j <= p
        if case["window"]:
            seen &= (p - j < case["window"]) | (j < case["sinks"])
        for h in range(Hk):
            k = s["k"][pg, h].double() * torch.exp2(s["k_scale"][pg, h].double() - 127)[..., None, None, None]
            k = k.permute(0, 1, 3, 2, 4).reshape(-1, D)[:L]
            v = s["v"][pg, h].double() * torch.exp2(s["v_scale"][pg, h].double() - 127)[..., None, None]
            v = v.transpose(2, 3).reshape(-1, D)[:L]
            for g in range(h * G, h * G + G):
                w = (s["q"][at[i]:at[i + 1], g].double() @ k.t()) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(~seen, float("-inf")), 1)
                y[at[i]:at[i + 1], g] = w @ v
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)

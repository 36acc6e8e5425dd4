"""Rows in front of int8 linears, the paged 8-bit cache and its attention, in
float64 from their definitions.  Layouts as in include/q4.h."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def rmsnorm_rows(x, residual, gain, eps):
    """x, residual [M, K] or None, gain [K] or None -> (codes int8, scales float64, h float64)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    u = h if gain is None else h * np.asarray(gain, np.float64)
    M, K = h.shape
    codes = np.zeros((M, K), np.int8)
    scales = np.zeros(M)
    for m in range(M):
        if not np.isfinite(u[m]).all() or not np.isfinite(h[m]).all():
            scales[m] = np.nan
            continue
        top = np.abs(u[m]).max(initial=0.0)
        if top == 0:
            continue
        codes[m] = np.rint(127 * u[m] / top).astype(np.int8)
        scales[m] = top / math.sqrt((h[m] * h[m]).sum() / K + eps) / 127
    return codes, scales, h


def scale_byte(top: float) -> int:
    """The smallest byte b with top <= 127 2^(b - 127); 255 for what is not finite."""
    if not math.isfinite(top):
        return 255
    b = 0
    if top > 0:
        m, e = math.frexp(top)           # top = m 2^e
        b = max(e - 7 + 127, 0)
        while top > math.ldexp(127.0, b - 127):
            b += 1
    return b


def rows_of(starts, lengths, T):
    """(row, sequence, position) of every row of a sequence."""
    clamp = [min(max(int(s), 0), T) for s in starts]
    for i in range(len(lengths)):
        n = max(clamp[i + 1] - clamp[i], 0)
        for t in range(n):
            yield clamp[i] + t, i, max(int(lengths[i]), 0) - n + t


def head(x, gain, eps, table_row, halves: bool):
    """One head's row: norm if eps is not None, rotation by R/2 cosines and sines if there is a row."""
    y = np.asarray(x, np.float64).copy()
    if eps is not None:
        y = y / math.sqrt((y * y).sum() / y.size + eps)
        if gain is not None:
            y = y * np.asarray(gain, np.float64)
    if table_row is not None:
        half = len(table_row) // 2
        c, s = np.asarray(table_row[:half], np.float64), np.asarray(table_row[half:], np.float64)
        p, q = (np.arange(half), np.arange(half) + half) if halves else (2 * np.arange(half), 2 * np.arange(half) + 1)
        a, b = y[p].copy(), y[q].copy()
        y[p], y[q] = a * c - b * s, b * c + a * s
    return y


class Pool:
    """A cache in host memory: codes k [P, H, B, D/16, 16, 16], v [P, H, B, D, 16], scale bytes ks, vs [P, H, B]."""

    def __init__(self, P, H, page, D):
        self.P, self.H, self.page, self.D = P, H, page, D
        B = page // BLOCK
        self.k = np.zeros((P, H, B, D // 16, 16, 16), np.int8)
        self.v = np.zeros((P, H, B, D, 16), np.int8)
        self.ks = np.zeros((P, H, B), np.uint8)
        self.vs = np.zeros((P, H, B), np.uint8)

    def place(self, pages, i, pos):
        """(page, block) of a position, or None where there is no such page."""
        p = pos // self.page
        if p >= pages.shape[1] or not 0 <= pages[i, p] < self.P:
            return None
        return int(pages[i, p]), pos % self.page // BLOCK

    def codes(self, name, page, h, b):
        """A block's codes as [16 tokens, D], a view."""
        if name == "v":
            return self.v[page, h, b].T
        return self.k[page, h, b].transpose(1, 0, 2).reshape(BLOCK, self.D)

    def put(self, name, page, h, b, t, codes):
        if name == "v":
            self.v[page, h, b][:, t] = codes
        else:
            self.k[page, h, b][:, t, :] = codes.reshape(-1, 16)

    def append(self, pages, starts, lengths, rows):
        """rows: {"k", "v"}: float64 [T, H, D], keys normalised and rotated."""
        T = rows["k"].shape[0]
        blocks = {}
        for row, i, pos in rows_of(starts, lengths, T):
            if pos >= 0:
                at = self.place(pages, i, pos)
                if at is not None:
                    blocks.setdefault((at, i, pos // BLOCK), []).append((pos, row))
        for (at, _, _), new in blocks.items():
            had = min(pos for pos, _ in new) % BLOCK
            for name, scales in (("k", self.ks), ("v", self.vs)):
                for h in range(self.H):
                    x = {pos % BLOCK: rows[name][row, h] for pos, row in new}
                    byte = scale_byte(max(float(np.abs(r).max()) if np.isfinite(r).all() else math.inf
                                          for r in x.values()))
                    old = int(scales[at[0], h, at[1]])
                    if had:
                        byte = max(byte, old)
                        if byte != 255 and byte > old:
                            c = self.codes(name, at[0], h, at[1]).astype(np.float64)
                            for t in range(had):
                                self.put(name, at[0], h, at[1], t, np.rint(np.ldexp(c[t], old - byte)).astype(np.int8))
                    for t, r in x.items():
                        code = np.zeros(self.D, np.int8) if byte == 255 else np.rint(np.ldexp(r, 127 - byte)).astype(np.int8)
                        self.put(name, at[0], h, at[1], t, code)
                    scales[at[0], h, at[1]] = byte

    def value(self, name, pages, i, h, pos):
        """Float64 [D] of a position; NaN where there is no such page."""
        at = self.place(pages, i, pos)
        byte = 255 if at is None else int((self.ks if name == "k" else self.vs)[at[0], h, at[1]])
        if byte == 255:
            return np.full(self.D, np.nan)
        return np.ldexp(self.codes(name, at[0], h, at[1])[pos % BLOCK].astype(np.float64), byte - 127)

    def byte(self, pages, i, h, b) -> int:
        """The scale byte of the values of block b."""
        at = self.place(pages, i, b * BLOCK)
        return 255 if at is None else int(self.vs[at[0], h, at[1]])

    def head(self, name, pages, i, h, n):
        """Positions 0 .. n - 1 of sequence i and a head, float64 [n, D]."""
        out = np.empty((-(-n // BLOCK) * BLOCK, self.D))
        for b in range(len(out) // BLOCK):
            at = self.place(pages, i, b * BLOCK)
            byte = 255 if at is None else int((self.ks if name == "k" else self.vs)[at[0], h, at[1]])
            out[b * BLOCK:(b + 1) * BLOCK] = np.nan if byte == 255 else np.ldexp(
                self.codes(name, at[0], h, at[1]).astype(np.float64), byte - 127)
        return out[:n]


def seen(pos, n, window, sinks):
    """Which of the keys 0 .. n - 1 the row at a position sees."""
    j = np.arange(n)
    s = j <= pos
    if window > 0:
        s &= (j > pos - window) | (j < sinks)
    return s


def attention(q, pool: Pool, pages, starts, lengths, scale, window=0, sinks=0):
    """q float64 [T, Hq, D] -> (y float64 [T, Hq, D], size [T, Hq, D], terms, flat,
    peak [T, Hq]): size is the weighted mean of |v|; terms and flat are the largest
    over a row's keys of what a score's terms add up to, sum |q k| |scale|, and of
    max|q| sum |k| |scale|; peak is the largest of a key's weight times 127 of its
    values' scale.  Rows of no sequence are NaN in all."""
    T, Hq, D = q.shape
    G = Hq // pool.H
    y, size = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    terms, flat, peak = (np.full((T, Hq), np.nan) for _ in range(3))
    rows = {}
    for row, i, pos in rows_of(starts, lengths, T):
        rows.setdefault(i, []).append((row, pos))
    for i, rs in rows.items():
        for h in range(pool.H):
            n = max(int(lengths[i]), 0)
            K, V = pool.head("k", pages, i, h, n), pool.head("v", pages, i, h, n)
            step = np.ldexp(127.0, np.array([pool.byte(pages, i, h, b) for b in range(-(-n // BLOCK))], int) - 127)
            step = np.repeat(step, BLOCK)[:n]
            for row, pos in rs:
                s = seen(pos, n, window, sinks)
                k, v = K[s], V[s]
                for g in range(h * G, h * G + G):
                    if not len(k):
                        y[row, g], size[row, g], terms[row, g], flat[row, g], peak[row, g] = 0, 0, 0, 0, 0
                        continue
                    x = (k @ q[row, g]) * scale
                    with np.errstate(invalid="ignore"):
                        p = np.exp(x - x.max())
                    p /= p.sum()
                    y[row, g], size[row, g], peak[row, g] = p @ v, p @ np.abs(v), (p * step[s]).max()
                    terms[row, g] = (np.abs(k) @ np.abs(q[row, g])).max() * abs(scale)
                    flat[row, g] = np.abs(q[row, g]).max() * np.abs(k).sum(1).max() * abs(scale)
    return y, size, terms, flat, peak

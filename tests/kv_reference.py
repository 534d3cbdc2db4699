"""Plain 64-bit statements of the paged cache's operators, for its tests."""
from __future__ import annotations

import numpy as np


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """Round to nearest even, as bits; NaN stays NaN."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def q4_encode(x: np.ndarray):
    """(codes -8..7, fp16 scales) of rows [..., d] of fp32 values, block by block."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        top = np.abs(b).max(-1, keepdims=True)
        s = np.minimum(top / np.float32(7), np.float32(65504)).astype(np.float16)
        s = np.where(np.isfinite(b).all(-1, keepdims=True), s, np.float16(np.nan))
        c = np.rint(b.astype(np.float64) / s.astype(np.float64))
        c = np.where(s > 0, np.clip(c, -8, 7), 0)
    return c.astype(np.int64).reshape(x.shape), s[..., 0]


def q4_value(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return codes * np.repeat(scales.astype(np.float64), 32, -1)


class Pages:
    """One layer's pool as bytes, by its documented layout."""

    def __init__(self, fmt, n_kv_heads, head_dim, page_rows):
        self.fmt, self.h, self.d, self.R = fmt, n_kv_heads, head_dim, page_rows
        self.head_bytes = page_rows * (2 * head_dim if fmt == "bf16" else head_dim // 2 + head_dim // 16)
        self.page_bytes = 2 * n_kv_heads * self.head_bytes
        e = np.arange(head_dim)
        self.nibble = ((e % 32 // 4) * (head_dim // 32) + e // 32) * 4 + e % 4

    def put(self, page: np.ndarray, which, head, row, x):
        """Writes one row of fp32 values into the bytes of a page."""
        base = (which * self.h + head) * self.head_bytes
        if self.fmt == "bf16":
            at = base + row * 2 * self.d
            page[at:at + 2 * self.d] = bf16_bits(x).view(np.uint8)
            return
        c, s = q4_encode(x)
        n = np.zeros(self.d, np.uint8)
        n[self.nibble] = c + 8
        at = base + row * self.d // 2
        page[at:at + self.d // 2] = n[0::2] | (n[1::2] << 4)
        at = base + self.R * self.d // 2 + row * self.d // 16
        page[at:at + self.d // 16] = s.view(np.uint8)

    def values(self, page: np.ndarray) -> np.ndarray:
        """fp64 [2][head][row][dim] of a page."""
        p = page.reshape(2, self.h, self.head_bytes)
        if self.fmt == "bf16":
            return bf16_value(p.view(np.uint16)).astype(np.float64).reshape(2, self.h, self.R, self.d)
        codes = p[..., :self.R * self.d // 2].reshape(2, self.h, self.R, self.d // 2)
        scales = np.ascontiguousarray(p[..., self.R * self.d // 2:]).view(np.float16)
        n = np.stack((codes & 15, codes >> 4), -1).reshape(2, self.h, self.R, self.d)[..., self.nibble]
        return q4_value(n.astype(np.int64) - 8, scales.reshape(2, self.h, self.R, self.d // 32))


def visible(n: int, window: int, sinks: int) -> np.ndarray:
    j = np.arange(n)
    return j[(j >= n - window) | (j < sinks)] if window else j


def attention(q, k, v, scale):
    """q [heads][d], k and v [kv heads][rows][d] (fp64): (o, error scale), where the second is what a
    relative error of one in the weights moves an output by at most, sum_j w_j |v_j|, and the largest
    sum |q||k| scale behind a score."""
    heads, kvh = q.shape[0], k.shape[0]
    o, size, dots = np.zeros(q.shape), np.zeros(q.shape), np.zeros(heads)
    if k.shape[1] == 0:
        return o, size, dots
    for h in range(heads):
        g = h * kvh // heads
        s = k[g] @ q[h] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        o[h], size[h] = w @ v[g], w @ np.abs(v[g])
        dots[h] = (np.abs(k[g]) @ np.abs(q[h])).max() * scale
    return o, size, dots


class Model:
    """The tables of a cache, call by call as the header words it."""

    def __init__(self, n_pages, n_seqs, max_pages, R):
        self.table = np.full((n_seqs, max_pages), -1, np.int32)
        self.lens, self.refs = np.zeros(n_seqs, np.int32), np.zeros(n_pages, np.int32)
        self.R, self.cap, self.bits = R, max_pages * R, 0
        self.copies = []  # (source, destination) pages of the last call

    def _take(self, k):
        free = np.flatnonzero(self.refs <= 0)
        return None if len(free) < k else list(free[:k])

    def extend(self, seqs, n_new=None):
        add = [1] * len(seqs) if n_new is None else list(n_new)
        live = [(s, a) for s, a in zip(seqs, add) if s >= 0]
        bits = 0
        if any(s >= len(self.lens) or a < 0 for s, a in live):
            bits |= 1
        ok = [(s, a) for s, a in live if s < len(self.lens) and a >= 0]
        if len({s for s, _ in ok}) < len(ok):
            bits |= 4
        if any(self.lens[s] + a > self.cap for s, a in ok):
            bits |= 2
        up = lambda x: -(-x // self.R)  # noqa: E731
        need = [] if bits else [(s, i) for s, a in ok for i in range(up(self.lens[s]), up(self.lens[s] + a))]
        pages = self._take(len(need))
        if not bits and pages is None:
            bits = 2
        self.bits |= bits
        if bits:
            return
        for (s, i), p in zip(need, pages):
            self.table[s, i], self.refs[p] = p, 1
        for s, a in ok:
            self.lens[s] += a

    def fork(self, parents, children):
        self.copies = []
        pairs = [(a, b) for a, b in zip(parents, children) if a >= 0 and b >= 0]
        n, bits = len(self.lens), 0
        if any(a >= n or b >= n for a, b in pairs):
            bits |= 1
        ok = [(a, b) for a, b in pairs if a < n and b < n]
        kids = [b for _, b in ok]
        if len(set(kids)) < len(kids) or any(self.lens[b] for b in kids) or set(kids) & {a for a, _ in ok}:
            bits |= 4
        tails = [(a, b) for a, b in ok if self.lens[a] % self.R]
        pages = None if bits else self._take(len(tails))
        if not bits and pages is None:
            bits = 2
        self.bits |= bits
        if bits:
            return
        new = dict(zip([b for _, b in tails], pages))
        for a, b in ok:
            self.table[b] = self.table[a]
            if b in new:
                i = self.lens[a] // self.R
                self.copies.append((int(self.table[a, i]), int(new[b])))
                self.table[b, i] = new[b]
            for p in self.table[b][self.table[b] >= 0]:
                self.refs[p] += 1
            self.lens[b] = self.lens[a]

    def release(self, seqs, window=0, sinks=0):
        for s in seqs:
            if s < 0:
                continue
            if s >= len(self.lens):
                self.bits |= 1
                continue
            for i, p in enumerate(self.table[s]):
                gone = not window or (i * self.R >= sinks and (i + 1) * self.R <= self.lens[s] - window)
                if p >= 0 and gone:
                    self.refs[p] -= 1
                    self.table[s, i] = -1
            if not window:
                self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        self.copies = list(zip(movers, holes))
        for a, b in self.copies:
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0

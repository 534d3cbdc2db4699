"""Plain 64-bit statements of 8-bit pages and of rotary positions, for their tests."""
from __future__ import annotations

import math

import numpy as np


def scale_exponent(top: float) -> int:
    """The least e of -126 .. 121 with top <= 127 * 2^e (121 if there is none)."""
    if top == 0:
        return -126
    m, e = math.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    return min(max(e - 7 if m <= 127 / 128 else e - 6, -126), 121)


class Pages8:
    """One layer's pool as bytes, by its documented layout."""

    def __init__(self, n_kv_heads, head_dim, page_rows):
        self.fmt, self.h, self.d, self.R = "q8", n_kv_heads, head_dim, page_rows
        self.code_bytes = n_kv_heads * page_rows * head_dim
        self.half_bytes = -(-(self.code_bytes + n_kv_heads * page_rows // 16 * 4) // 64) * 64
        self.page_bytes = 2 * self.half_bytes

    def parts(self, page: np.ndarray):
        """codes uint8 [2][head][row][dim] and scales fp32 [2][head][block]: views of a page's bytes."""
        halves = page.reshape(2, self.half_bytes)
        codes = [h[:self.code_bytes].reshape(self.h, self.R, self.d) for h in halves]
        scales = [h[self.code_bytes:self.code_bytes + self.h * self.R // 4].view(np.float32).reshape(self.h, self.R // 16)
                  for h in halves]
        return codes, scales

    def values(self, page: np.ndarray) -> np.ndarray:
        """fp64 [2][head][row][dim] of a page."""
        codes, scales = self.parts(page)
        with np.errstate(invalid="ignore"):
            return np.stack([(c.astype(np.float64) - 128) * np.repeat(s.astype(np.float64), 16, 1)[..., None]
                             for c, s in zip(codes, scales)])

    def write(self, page: np.ndarray, block: int, rows: dict):
        """What a call that writes rows {row of the block: x [2][head][dim], fp32} of one block makes of it."""
        codes, scales = self.parts(page)
        first = min(rows)
        for i in range(2):
            for h in range(self.h):
                new = np.stack([x[i, h] for x in rows.values()]).astype(np.float64)
                old = float(scales[i][h, block])
                finite = bool(np.isfinite(new).all()) and not (first and math.isnan(old))
                at = slice(16 * block, 16 * block + first)
                if not finite:
                    scales[i][h, block] = np.nan
                    continue
                e = scale_exponent(float(np.abs(new).max()))
                s = max(2.0 ** e, old) if first else 2.0 ** e
                if first and s > old:
                    c = codes[i][h, at].astype(np.float64) - 128
                    codes[i][h, at] = np.rint(c * (old / s)) + 128
                scales[i][h, block] = s
                for r, x in rows.items():
                    codes[i][h, 16 * block + r] = np.clip(np.rint(x[i, h].astype(np.float64) / s), -127, 127) + 128


def frequencies(rot, theta=1e4, scaling=None, factor=1.0, context=0.0, slow=1.0, fast=32.0):
    """Radians per position of each pair, and the magnitude."""
    out = []
    for i in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
        w = base ** (-2 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            turns = context * w / (2 * math.pi)
            keep = min(max((turns - slow) / (fast - slow), 0.0), 1.0)
            w = w * keep + w / factor * (1 - keep)
        out.append(w)
    return np.array(out), 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def rotate(x, positions, freq, magnitude, layout, backward=False):
    """x [n][heads][d] (fp64), positions [n]: rotated."""
    rot, y = 2 * len(freq), x.astype(np.float64).copy()
    angle = np.asarray(positions, np.float64)[:, None, None] * freq * (-1 if backward else 1)
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y

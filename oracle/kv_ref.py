"""Plain CPU oracle of the rotary positions and of the paged 8-bit key/value
cache with its attention.  Test infrastructure only.

Values and attention are formed in 64 bits.  What the library fixes bit for bit
(turned keys, steps and codes) is emulated here in IEEE fp32, one NumPy
operation for one rounding, in the documented order.
"""

from __future__ import annotations

import numpy as np

f32 = np.float32


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original: float = 0.0, low: float = 1.0, high: float = 4.0) -> np.ndarray:
    """Radians per position of each pair, fp64 [rot/2]."""
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "none":
        return f
    if scaling == "linear":
        return f / factor
    turns = original * f / (2 * np.pi)
    if scaling == "turns":
        keep = (turns - low) / (high - low)
    else:
        keep = (np.log(turns) - np.log(low)) / (np.log(high) - np.log(low))
    keep = np.clip(keep, 0.0, 1.0)
    return keep * f + (1 - keep) * f / factor


def rope_table(n_pos: int, rot: int, magnitude: float = 1.0, **kw) -> np.ndarray:
    """(cos, sin) times magnitude, fp64 [n_pos, rot/2, 2]."""
    a = np.arange(n_pos, dtype=np.float64)[:, None] * rope_frequencies(rot, **kw)
    return np.stack((np.cos(a), np.sin(a)), -1) * magnitude


def pair_columns(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope(x: np.ndarray, table: np.ndarray, positions, interleaved: bool = False,
         transpose: bool = False) -> np.ndarray:
    """x [..., rows, heads, D] turned by table[position of the row] in x's own precision
    (fp32: every product and every sum one rounding)."""
    one, two = pair_columns(2 * table.shape[1], interleaved)
    cs = table[np.asarray(positions)].astype(x.dtype)[..., :, None, :, :]
    c, s = cs[..., 0], cs[..., 1]
    s = -s if transpose else s
    y = x.copy()
    x1, x2 = x[..., one], x[..., two]
    y[..., one] = x1 * c - x2 * s
    y[..., two] = x2 * c + x1 * s
    return y


def codes_of(x: np.ndarray) -> np.ndarray:
    """clamp(rint(x), -127, 127), 0 for NaN."""
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(x), -127, 127)
    return np.where(np.isnan(q), 0, q).astype(np.int32)


class Cache:
    """Codes uint8 [pages, heads, page, D] (keys) and [pages, heads, D, page] (values), steps fp32."""

    def __init__(self, k_codes, v_codes, k_steps, v_steps):
        self.k_codes, self.v_codes = np.array(k_codes), np.array(v_codes)
        self.k_steps, self.v_steps = np.array(k_steps, f32), np.array(v_steps, f32)
        self.n_pages, self.heads, self.page, self.dim = self.k_codes.shape

    def _put(self, codes, steps, new, lo):
        """codes [heads, page, D] (a view), steps [heads] (a view), new fp32 [tokens, heads, D] at place lo."""
        with np.errstate(all="ignore"):
            was = steps.copy() if lo > 0 else np.zeros_like(steps)
            top = np.abs(new).max(axis=(0, 2)) / f32(127)       # NaN stays NaN
            step = np.maximum(was, top)
            for h in range(len(steps)):
                if lo > 0 and step[h] != was[h]:
                    c = codes[h, :lo].astype(f32) - f32(128)
                    codes[h, :lo] = codes_of(c * (was[h] / step[h])) + 128
                q = new[:, h] / step[h] if step[h] > 0 else np.zeros_like(new[:, h])
                codes[h, lo: lo + len(new)] = codes_of(q) + 128
            steps[:] = step

    def append(self, k, v, lens, pages, starts):
        """k, v fp32 [T, heads, D], already turned."""
        for b, length in enumerate(lens):
            rows = range(starts[b], starts[b + 1])
            first = length - len(rows)
            for p in range(max(first, 0) // self.page, -(-length // self.page)):
                if p >= pages.shape[1] or not 0 <= pages[b, p] < self.n_pages:
                    continue
                lo, hi = max(first, p * self.page), min(length, (p + 1) * self.page)
                if lo >= hi:
                    continue
                at, r = pages[b, p], starts[b] - first
                self._put(self.k_codes[at], self.k_steps[at], k[r + lo: r + hi], lo - p * self.page)
                self._put(self.v_codes[at].transpose(0, 2, 1), self.v_steps[at], v[r + lo: r + hi],
                          lo - p * self.page)

    def tokens(self, b, lo, hi, pages):
        """Keys and values fp32 [hi - lo, heads, D] and whether each token's page is there."""
        k = np.zeros((hi - lo, self.heads, self.dim), f32)
        v, there = np.zeros_like(k), np.zeros(hi - lo, bool)
        for j in range(lo, hi):
            p = j // self.page
            if p >= pages.shape[1] or not 0 <= pages[b, p] < self.n_pages:
                continue
            at, t = pages[b, p], j % self.page
            there[j - lo] = True
            k[j - lo] = (self.k_codes[at, :, t].astype(f32) - f32(128)) * self.k_steps[at][:, None]
            v[j - lo] = (self.v_codes[at, :, :, t].astype(f32) - f32(128)) * self.v_steps[at][:, None]
        return k, v, there

    def attention(self, q, lens, pages, starts, scale, window=0, causal=True):
        """q [T, Hq, D] -> (out fp64 [T, Hq, D], lse fp64 [T, Hq], sum_j p_j |v_j| [T, Hq, D],
        largest key value [T, Hq] that the row sees)."""
        T, hq, d = q.shape
        group = hq // self.heads
        out = np.zeros((T, hq, d))
        lse = np.full((T, hq), -np.inf)
        spread, top = np.zeros((T, hq, d)), np.zeros((T, hq))
        for b, length in enumerate(lens):
            k, v, there = self.tokens(b, 0, max(length, 0), pages)
            n = starts[b + 1] - starts[b]
            for i in range(n):
                at, r = length - n + i, starts[b] + i
                j = np.arange(max(length, 0))
                see = there.copy()
                if causal:
                    see &= j <= at
                if window:
                    see &= j > at - window
                if not see.any():
                    continue
                for h in range(hq):
                    kk, vv = (t[see, h // group].astype(np.float64) for t in (k, v))
                    s = kk @ q[r, h].astype(np.float64) * scale
                    m = s.max()
                    e = np.exp(s - m)
                    out[r, h] = e @ vv / e.sum()
                    spread[r, h] = e @ np.abs(vv) / e.sum()
                    lse[r, h] = m + np.log(e.sum())
                    top[r, h] = np.abs(kk).max()
        return out, lse, spread, top

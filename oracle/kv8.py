"""8-bit paged cache, float64 (test infrastructure only).

Restates, from the definitions alone, what the 8-bit cache holds and what its attention and page selection return:

* a page is quantised when its last token arrives, one scale per (page, kv head, K or V) block;
* with m = max |x| over the block's finite values and M = 127 (INT8) or 448 (E4M3): scale = m / M as float32,
  code = x M / m rounded to nearest even; m < 2^-100 stores zeros with scale 0; infinities saturate, NaNs store 0;
* lo and hi are the smallest and largest K code of each channel over the page's tokens;
* the tokens of the incomplete page are BF16 rows.
"""
from __future__ import annotations

import math

import numpy as np

INT8, E4M3 = 0, 1
TOP = {INT8: 127, E4M3: 448}


def code_values(fmt: int) -> np.ndarray:
    """The number each of the 256 code bytes stands for."""
    b = np.arange(256)
    if fmt == INT8:
        return b - 128.0
    e, f = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    mag[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -mag, mag)


def place(P: int, d: int, is_v: bool) -> np.ndarray:
    """Byte offset of (token, channel) in a code section, [P][d]."""
    out = np.empty((P, d), np.int64)
    for t in range(P):
        turn = 2 * ((t >> 1) & 3) if is_v else (4 * (t & 1) if d == 128 else 0)
        for c in range(d):
            line, chunk, byte = (t * d + c) // 128, ((t * d + c) % 128) // 16, c % 16
            out[t, c] = line * 128 + (chunk ^ turn) * 16 + byte
    return out


def block_bytes(P: int, d: int) -> int:
    return -(-(2 * P * d + 16 + 2 * d) // 128) * 128


def encode(x: np.ndarray, fmt: int):
    """x [P][d] BF16 values as float64: (bytes [P][d], scale float32).  Nearest code, to the even one at a tie."""
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    m = float(fin.max())
    zero = 128 if fmt == INT8 else 0
    if m < 2.0 ** -100:
        return np.full(x.shape, zero, np.uint8), np.float32(0)
    scale = np.float32(m) / np.float32(TOP[fmt])
    if fmt == INT8:
        y = np.where(np.isnan(x), 0.0, np.clip(np.where(np.isnan(x), 0, x) * 127.0 / m, -127, 127))
        return (np.rint(y) + 128).astype(np.uint8), scale
    vals = code_values(fmt)
    pos = vals[:127]                                     # ascending magnitudes, byte = index
    y = np.clip(np.where(np.isnan(x), 0, np.abs(x)) * 448.0 / m, 0, 448)
    j = np.clip(np.searchsorted(pos, y), 1, 126)
    low, high = pos[j - 1], pos[j]
    up = (y - low > high - y) | ((y - low == high - y) & (j % 2 == 0))
    byte = np.where(up, j, j - 1)
    return np.where((x < 0) | ((x == 0) & np.signbit(x)), byte + 128, byte).astype(np.uint8), scale



class Cache:
    """Pool bytes [pages][heads][block] and tail rows [slots][heads][2][P][d] (BF16 values in float64) of one layer."""

    def __init__(self, P, d, heads, fmt, pool, tail):
        self.P, self.d, self.heads, self.fmt = P, d, heads, fmt
        self.pool, self.tail = pool, tail
        self.at = [place(P, d, False), place(P, d, True)]

    def store(self, page: int, h: int, kv: int, x: np.ndarray):
        P, d = self.P, self.d
        code, scale = encode(x, self.fmt)
        blk = self.pool[page, h]
        blk[kv * P * d + self.at[kv]] = code
        blk[2 * P * d + 4 * kv:2 * P * d + 4 * kv + 4] = np.frombuffer(scale.tobytes(), np.uint8)
        if kv == 0:
            v = code_values(self.fmt)[code] + 0.0
            for off, val in ((16, v.min(0)), (16 + d, v.max(0))):
                if self.fmt == INT8:
                    b = val + 128
                else:
                    table = code_values(E4M3)
                    b = np.array([int(np.flatnonzero(table == y)[0]) for y in val])
                blk[2 * P * d + off:2 * P * d + off + d] = b.astype(np.uint8)

    def write(self, bt, slot: int, start: int, K, V, append=False):
        """Tokens start .. of one request; K, V [tokens][heads][d]."""
        P, n = self.P, K.shape[0]
        if n == 0:
            return
        for h in range(self.heads):
            for kv, x in enumerate((K, V)):
                base = start // P * P
                rows = np.concatenate([self.tail[slot, h, kv, :start - base], x[:, h]])     # tokens base ..
                whole = rows.shape[0] // P
                for j in range(whole):
                    self.store(bt[base // P + j], h, kv, rows[j * P:(j + 1) * P])
                rest = rows[whole * P:]
                self.tail[slot, h, kv, :rest.shape[0]] = rest
                if append and whole:
                    self.tail[slot, h, kv, P - 1] = x[-1, h]

    def rows(self, bt, slot: int, n: int, h: int, pages=None):
        """Dequantised K, V [tokens][d] of a kv head: the listed complete pages (all by default), then the tail rows."""
        P, d = self.P, self.d
        table, out = code_values(self.fmt), []
        pages = range(n // P) if pages is None else pages
        for kv in range(2):
            parts = []
            for p in pages:
                blk = self.pool[bt[p], h]
                scale = blk[2 * P * d + 4 * kv:2 * P * d + 4 * kv + 4].view(np.float32)[0]
                parts.append(table[blk[kv * P * d + self.at[kv]]] * float(scale))
            parts.append(self.tail[slot, h, kv, :n % P])
            out.append(np.concatenate(parts) if parts else np.zeros((0, d)))
        return out

    def attend(self, q, bt, slot: int, n: int, pages=None):
        """q [heads G][d]: output [heads G][d], and a bound of a float32 evaluation's error (see attend_bound)."""
        G = q.shape[0] // self.heads
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        for h in range(self.heads):
            k, v = self.rows(bt, slot, n, h, None if pages is None else [p for p in pages[h] if p >= 0])
            if k.shape[0] == 0:
                continue
            for i in range(h * G, (h + 1) * G):
                out[i], bound[i] = attend_bound(q[i], k, v, self.P)
        return out, bound

    def bounds(self, q, bt, n: int, h: int):
        """U_p of every complete page for one kv head; q [G][d]."""
        P, d = self.P, self.d
        a, b = np.maximum(q, 0).sum(0), np.maximum(-q, 0).sum(0)
        table, u = code_values(self.fmt), np.zeros(n // P)
        for p in range(n // P):
            blk = self.pool[bt[p], h]
            lo, hi = (table[blk[2 * P * d + o:2 * P * d + o + d]] for o in (16, 16 + d))
            u[p] = math.fsum(list(a * hi) + list(-b * lo)) * float(blk[2 * P * d:2 * P * d + 4].view(np.float32)[0])
        return u

    def select(self, q, bt, n: int, first: int, last: int, k: int):
        """[heads][k] logical pages, ascending, -1 after the last; q [heads G][d]."""
        G, pages = q.shape[0] // self.heads, n // self.P
        out = np.full((self.heads, k), -1, np.int32)
        for h in range(self.heads):
            if pages <= k:
                ids = np.arange(pages)
            else:
                u = self.bounds(q[h * G:(h + 1) * G], bt, n, h)
                p = np.arange(pages)
                kept = (p < first) | (p >= pages - last)
                ids = np.sort(np.lexsort((p, np.where(kept, -np.inf, -u)))[:k])
            out[h, :len(ids)] = ids
        return out


U = 2.0 ** -24          # half a step of float32, relative


def attend_bound(q, k, v, P: int):
    """softmax(q k^T / sqrt d) v in float64, and how far a float32 evaluation may be off.

    A score is a sum of d products: off by at most s = (d + 8) U sum |q k| / sqrt d in any order of summation (the 8
    cover the scaling by sqrt d and log2 e, the products' own rounding and the block's scale).  The exponential is off
    by at most 2^-21 relative (two halves of 2^-22: the hardware's and its argument's), and the weighted sums over n
    tokens, their rescalings and the division by (n + 32) U.  A weight may enter its product as a number of 24 bits
    relative to the largest weight of its page: U e^(m_page - lse) |v|.
    """
    d, n = q.shape[0], k.shape[0]
    s = k @ q / math.sqrt(d)
    m = s.max()
    w = np.exp(s - m)
    p = w / w.sum()
    out = p @ v
    off = (d + 8) * U * (np.abs(k) @ np.abs(q)).max() / math.sqrt(d)
    rel = 2 * off + 2.0 ** -21 + 2 * (n + 32) * U
    top = np.concatenate([np.full(min(P, n - i), p[i:i + P].max()) for i in range(0, n, P)])
    return out, rel * (p @ np.abs(v)) + U * (top @ np.abs(v)) + 1e-38

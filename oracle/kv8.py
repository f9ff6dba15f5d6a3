"""The 8-bit block cache and its attention, restated plainly in float64.

A block of 64 positions x D values of one (sequence, kv head) has one float32
scale s = amax / 448 (e4m3) or amax / 127 (int8), 1 where amax is 0; codes are
round(x / s) with the quotient in float32.  A block is read quantised once all
its 64 positions are cached, in 16 bits until then.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_round

BLOCK = 64
TOP = {"e4m3": 448.0, "int8": 127.0}


def quantise(x, fmt: str):
    """(codes' values float64 [.., 64, D], scales float32 [..]) of blocks x [.., 64, D] (values exact in float32)."""
    x32 = np.asarray(x).astype(np.float32)
    amax = np.abs(x32).max(axis=(-1, -2))
    with np.errstate(invalid="ignore"):
        s = np.where(amax == 0, np.float32(1), amax / np.float32(TOP[fmt])).astype(np.float32)
    bad = ~np.isfinite(x32).all(axis=(-1, -2))
    s = np.where(bad, np.float32(np.nan), s)
    with np.errstate(invalid="ignore"):
        y = (x32 / s[..., None, None]).astype(np.float32)
    y = np.where(bad[..., None, None], np.float32(0), y)
    if fmt == "e4m3":
        c = e4m3_round(np.clip(y.astype(np.float64), -448, 448))
    else:
        c = np.clip(np.rint(y), -127, 127).astype(np.float64)
    return c, s


def k_index(r, d):
    """Byte of K element (position r of the page, d) in its page."""
    return ((r // 8 * 2 + d // 64) * 8 + r % 8) * 64 + d % 64


def v_index(r, d):
    """Byte of V element (r, d) after the page's 8192 K codes."""
    return r // 16 * 2048 + d // 32 * 512 + (d % 8 * 4 + r % 8 // 2) * 16 + d // 16 % 2 * 8 + d // 8 % 2 * 4 + r // 8 % 2 * 2 + r % 2


def page_rows(codes, which: int):
    """Codes of pages uint8 [.., 8192] as rows [.., 64, 128]."""
    r, d = np.arange(64)[:, None], np.arange(128)[None]
    return codes[..., (k_index, v_index)[which](r, d)]


def code_values(codes, fmt: str):
    """uint8 codes -> the numbers they stand for, float64."""
    c = np.asarray(codes).astype(np.int64)
    if fmt == "int8":
        return np.where(c > 127, c - 256, c).astype(np.float64)
    e, m = c % 128 // 8, c % 8
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c >= 128, -x, x)


class Kv8Ref:
    """One sequence: x[0], x[1] are the K and V rows [Hkv, len, D] as appended (float64)."""

    def __init__(self, Hkv: int, fmt: str, D: int = 128):
        self.fmt, self.x = fmt, [np.zeros((Hkv, 0, D)) for _ in range(2)]

    @property
    def len(self):
        return self.x[0].shape[1]

    def append(self, k, v, at: int = None):
        """Rows k, v [n, Hkv, D]; at: position of the first (default: the end), later rows are dropped."""
        at = self.len if at is None else at
        for i, y in enumerate((k, v)):
            self.x[i] = np.concatenate((self.x[i][:, :at], np.asarray(y, np.float64).transpose(1, 0, 2)), axis=1)

    def blocks(self, which: int):
        """(codes' values [Hkv, full, 64, D], scales [Hkv, full]) of the complete blocks."""
        x = self.x[which]
        full = x.shape[1] // BLOCK
        return quantise(x[:, :full * BLOCK].reshape(x.shape[0], full, BLOCK, x.shape[2]), self.fmt)

    def cached(self, which: int):
        """Rows as attention reads them, float64 [Hkv, len, D]; a non-finite 16-bit row reads as NaN."""
        x = self.x[which]
        c, s = self.blocks(which)
        y = (c * s.astype(np.float64)[..., None, None]).reshape(x.shape[0], BLOCK * s.shape[1], x.shape[2])
        rest = x[:, y.shape[1]:]
        rest = np.where(np.isfinite(rest).all(-1, keepdims=True), rest, np.nan)
        return np.concatenate((y, rest), axis=1)

    def attend(self, q, sm_scale: float, window: int = 0):
        """q [n, Hq, D] at the last n positions -> (out [n, Hq, D], lse2 [n, Hq], sum p |v| [n, Hq, D],
        largest sum_d |q_d k_d| [n, Hq] over the visible keys)."""
        q = np.asarray(q, np.float64)
        n, Hq, D = q.shape
        k, v = self.cached(0), self.cached(1)
        G = Hq // k.shape[0]
        out, lse = np.zeros((n, Hq, D)), np.zeros((n, Hq))
        mass, size = np.zeros((n, Hq, D)), np.zeros((n, Hq))
        for i in range(n):
            t = self.len - n + i
            lo = max(0, t - window + 1) if window > 0 else 0
            for h in range(Hq):
                K, V = k[h // G, lo:t + 1], v[h // G, lo:t + 1]
                s = K @ q[i, h] * sm_scale
                m = s.max()
                p = np.exp(s - m)
                out[i, h] = p @ V / p.sum()
                mass[i, h] = p @ np.abs(V) / p.sum()
                lse[i, h] = (m + np.log(p.sum())) / np.log(2)
                size[i, h] = (np.abs(K) @ np.abs(q[i, h])).max() * sm_scale
        return out, lse, mass, size

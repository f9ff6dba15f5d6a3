"""Rotary positions in float64 (angles in extended precision)."""
from __future__ import annotations

import numpy as np

KINDS = ("plain", "linear", "ntk", "yarn", "bands")


def frequencies(rot: int, base: float, kind: str = "plain", factor: float = 1.0, orig_len: float = 0.0, low: float = None,
                high: float = None):
    """(w_i in radians per position as long doubles [rot/2], factor of the rotated values)."""
    L = np.longdouble
    pi2 = L(2) * L("3.14159265358979323846264338327950288")
    i = np.arange(rot // 2).astype(L)
    bs = L(base)
    if kind == "ntk":
        bs = bs * L(factor) ** (L(rot) / L(rot - 2))
    w = bs ** (-2 * i / L(rot))
    amp = 1.0
    if kind == "linear":
        w = w / L(factor)
    elif kind == "yarn":
        low, high = low or 1.0, high or 32.0
        dim = lambda turns: L(rot) * np.log(L(orig_len) / (pi2 * L(turns))) / (2 * np.log(bs))
        a, c = max(np.floor(dim(high)), L(0)), min(np.ceil(dim(low)), L(rot - 1))
        r = np.clip((i - a) / max(c - a, L("0.001")), L(0), L(1))
        w = (1 - r) * w + r * w / L(factor)
        amp = 1 + 0.1 * np.log(factor) if factor > 1 else 1.0
    elif kind == "bands":
        low, high = low or 1.0, high or 4.0
        r = np.clip((L(orig_len) * w / pi2 - L(low)) / (L(high) - L(low)), L(0), L(1))
        w = (1 - r) * w / L(factor) + r * w
    return w, float(amp)


def rotate(x, pos, w, amp, layout: str, grad: bool = False):
    """x [..., T, H, D] float64, pos int [..., T]: the first 2 len(w) elements of each head rotated."""
    x = np.asarray(x, dtype=np.float64)
    n = len(w)
    pi2 = 8 * np.arctan(np.longdouble(1))
    turns = np.asarray(pos).astype(np.longdouble)[..., None] * w / pi2
    ang = ((turns - np.rint(turns)) * pi2).astype(np.float64)   # modulo one turn while all its bits are there
    c, s = np.cos(ang)[..., None, :] * amp, np.sin(ang)[..., None, :] * amp
    if grad:
        s = -s
    y = x.copy()
    u, v = (x[..., :n], x[..., n:2 * n]) if layout == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    a, b = u * c - v * s, v * c + u * s
    if layout == "half":
        y[..., :n], y[..., n:2 * n] = a, b
    else:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a, b
    return y

"""CPU oracle of the serving step (NumPy, fp64): rotary positions, norms per head and their gradient, the rows a ragged
batch appends and attends to, the f8_block format, and chunk attention with score modifications.  Written from the definitions in include/tq.h, not from the kernels; the
quantisers are those of tq_oracle."""
from __future__ import annotations

import math

import numpy as np

from . import tq_oracle as O


def rope_angles(rotary: int, scaling: str = "none", base: float = 10000.0, factor: float = 1.0,
                original_ctx: float = 0.0, low: float = 0.0, high: float = 0.0, attn_factor: float = 0.0):
    """(angles per position of the rotary / 2 pairs, factor on the rotated coordinates)."""
    i = np.arange(rotary // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = base ** (-2.0 * i / rotary)
    attn = 1.0
    low = low or 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "wavelength":
        turns = original_ctx * f / (2 * math.pi)
        s = np.clip((turns - low) / ((high or 4.0) - low), 0.0, 1.0)
        f = s * f + (1 - s) * f / factor
    elif scaling == "yarn":
        def dim(t):
            return rotary * math.log(original_ctx / (2 * math.pi * t)) / (2 * math.log(base))
        a = max(math.floor(dim(high or 32.0)), 0)
        b = min(math.ceil(dim(low)), rotary - 1)
        g = np.clip((i - a) / max(b - a, 0.001), 0.0, 1.0)
        f = g * f / factor + (1 - g) * f
        attn = 0.1 * math.log(factor) + 1.0
    return f, attn_factor or attn


def rope(x, positions, angles, m: float = 1.0, layout: str = "half", inverse: bool = False) -> np.ndarray:
    """x [tokens, heads, d] rotated to positions [tokens]; coordinates behind the 2 len(angles) first unchanged."""
    y = np.array(x, np.float64)
    n = len(angles)
    a = np.asarray(positions, np.float64)[:, None] * angles * (-1.0 if inverse else 1.0)
    c, s = (m * np.cos(a))[:, None], (m * np.sin(a))[:, None]
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    p, q = np.array(y[..., first]), np.array(y[..., second])
    y[..., first] = p * c - q * s
    y[..., second] = p * s + q * c
    return y


def norm_rope(x, weight, positions, angles, eps: float, m: float = 1.0, layout: str = "half") -> np.ndarray:
    """x [tokens, heads, d] normed per head, times weight [d] (None: ones), rotated."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rope(y if weight is None else y * weight, positions, angles, m, layout)


def norm_rope_grad(x, dout, weight, positions, angles, eps: float, m: float = 1.0, layout: str = "half"):
    """(dx, dweight) of norm_rope for the gradient dout of its result: the chain rule through 1 / sqrt(mean + eps)."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    g = rope(dout, positions, angles, m, layout, inverse=True)
    ms = (x * x).mean(-1, keepdims=True) + eps
    gw = g if weight is None else g * weight
    dx = gw * ms ** -0.5 - x * ms ** -1.5 * (gw * x).sum(-1, keepdims=True) / d
    return dx, (g * x * ms ** -0.5).sum((0, 1))


def batch_positions(new, lens):
    """(sequence, position) of every row of a batch of new[b] tokens at the ends of sequences of lens[b] tokens."""
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)]) if len(new) else np.zeros(0, np.int64)
    return seq, pos.astype(np.int64)


def visible(pos: int, length: int, window: int = 0, first_key: int = 0, prefix: int = 0):
    """The keys [lo, hi) that the token at a position sees (empty if hi <= lo), without sinks."""
    hi = min(length, max(pos + 1, prefix))
    lo = max(0, first_key)
    if window:
        lo = max(lo, pos - window + 1)
    return lo, hi


def seen(pos: int, length: int, window: int = 0, first_key: int = 0, prefix: int = 0, sinks: int = 0) -> np.ndarray:
    """The keys that the token at a position sees: those of visible(), and the first `sinks` ones from first_key on of
    those that only the window would hide."""
    lo, hi = visible(pos, length, window, first_key, prefix)
    first = max(0, first_key)
    return np.concatenate([np.arange(first, min(first + sinks, lo, hi)), np.arange(lo, max(lo, hi))])


def chunk_attention(q, k, v, positions, scale: float, *, softcap: float = 0.0, window: int = 0, slopes=None,
                    first_keys=None, prefix: int = 0, missing=None, sinks: int = 0) -> np.ndarray:
    """One sequence: q [n, Hq, d] at positions [n], k and v [T, H, d] its stored tokens; missing [T] marks keys that
    are not there.  Returns [n, Hq, d]."""
    n, Hq, d = q.shape
    T, H, _ = k.shape
    out = np.zeros((n, Hq, d))
    for i in range(n):
        j = seen(int(positions[i]), T, window, 0 if first_keys is None else int(first_keys[i]), prefix, sinks)
        if missing is not None:
            j = j[~missing[j]]
        if len(j) == 0:
            continue
        for h in range(Hq):
            s = k[j, h * H // Hq] @ np.asarray(q[i, h], np.float64) * scale
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(int(positions[i]) - j)
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ v[j, h * H // Hq]
    return out


def q8_0_values(x) -> np.ndarray:
    """What x reads back as after q8_0: q * fp16(delta), q from the unrounded fp64 delta."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    delta = np.abs(b).max(-1, keepdims=True) / 127.0
    t = np.divide(b, delta, out=np.zeros_like(b), where=delta > 0)
    q = np.sign(t) * np.floor(np.abs(t) + 0.5)
    return (q * delta.astype(np.float16).astype(np.float64)).reshape(x.shape)


def turbo_mse_encode(x, fmt: str, signs) -> dict:
    """Stage 1 of a turbo format on unrounded values (tq_oracle.turbo_encode takes fp16 inputs)."""
    x = np.asarray(x, np.float64)
    n = np.sqrt(np.sum(x * x, axis=-1))
    y = O.rotate(x / np.where(n > 0, n, 1.0)[..., None], signs)
    _, b = O.codebook(O.TURBO_FORMATS[fmt][0], x.shape[-1])
    return {"n16": n.astype(np.float16), "idx": O.quantize(y, b), "y": y, "n": n}


F8_BLOCK, F8_TOP, F8_MIN, F8_MAX = 16, 448.0, -80, 80


def e4m3_values() -> np.ndarray:
    """What the 256 codes stand for: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x[(c & 127) == 127] = np.nan
    return np.where(c & 128, -x, x)


def e4m3_round(x) -> np.ndarray:
    """The nearest finite e4m3 value of |x| <= 448, found among all of them; a tie goes to the even code."""
    grid = e4m3_values()[:127]
    a = np.abs(np.asarray(x, np.float64))
    up = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[up - 1], grid[up]
    right = (a - lo > hi - a) | ((a - lo == hi - a) & (up % 2 == 0))
    return np.copysign(np.where(right, hi, lo), x)


def f8_exponent(top: float) -> int:
    """The smallest e in [-80, 80] with top <= 448 * 2^e."""
    e = F8_MIN
    while top > F8_TOP * 2.0 ** e:
        e += 1
    return e


class F8Block:
    """One block of one head: at most 16 tokens, in the order in which a sequence gets them."""

    def __init__(self, d: int):
        self.codes, self.marks, self.e = np.zeros((0, d)), np.zeros(0, bool), F8_MIN

    def append(self, x, at: int):
        """New tokens x [n, d] from offset `at` on; what was there before `at` stays, what was behind is gone."""
        x = np.array(x, np.float64)
        bad = ~(np.abs(x) <= F8_TOP * 2.0 ** F8_MAX).all(-1)
        x[bad] = 0.0
        e = f8_exponent(np.abs(x).max(initial=0.0))
        codes, marks = self.codes[:at], self.marks[:at]
        if at:
            e = max(e, self.e)
            codes = e4m3_round(codes * 2.0 ** (self.e - e))
        self.codes = np.concatenate([codes, e4m3_round(x * 2.0 ** -e)])
        self.marks, self.e = np.concatenate([marks, bad]), e

    def values(self) -> np.ndarray:
        return np.where(self.marks[:, None], np.nan, self.codes * 2.0 ** self.e)


__all__ = ["O", "turbo_mse_encode", "rope_angles", "rope", "batch_positions", "visible", "seen", "chunk_attention", "q8_0_values",
           "norm_rope", "norm_rope_grad", "e4m3_values", "e4m3_round", "f8_exponent", "F8Block"]

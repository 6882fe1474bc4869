"""CPU oracle of the serving step (NumPy, fp64): rotary positions, the rows a ragged batch appends and attends to, and
chunk attention with score modifications.  Written from the definitions in include/tq.h, not from the kernels; the
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


def batch_positions(new, lens):
    """(sequence, position) of every row of a batch of new[b] tokens at the ends of sequences of lens[b] tokens."""
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)]) if len(new) else np.zeros(0, np.int64)
    return seq, pos.astype(np.int64)


def visible(pos: int, length: int, window: int = 0, first_key: int = 0, prefix: int = 0):
    """The keys [lo, hi) that the token at a position sees (empty if hi <= lo)."""
    hi = min(length, max(pos + 1, prefix))
    lo = max(0, first_key)
    if window:
        lo = max(lo, pos - window + 1)
    return lo, hi


def chunk_attention(q, k, v, positions, scale: float, *, softcap: float = 0.0, window: int = 0, slopes=None,
                    first_keys=None, prefix: int = 0, missing=None) -> np.ndarray:
    """One sequence: q [n, Hq, d] at positions [n], k and v [T, H, d] its stored tokens; missing [T] marks keys that
    are not there.  Returns [n, Hq, d]."""
    n, Hq, d = q.shape
    T, H, _ = k.shape
    out = np.zeros((n, Hq, d))
    for i in range(n):
        lo, hi = visible(int(positions[i]), T, window, 0 if first_keys is None else int(first_keys[i]), prefix)
        j = np.arange(lo, max(lo, hi))
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


__all__ = ["O", "turbo_mse_encode", "rope_angles", "rope", "batch_positions", "visible", "chunk_attention", "q8_0_values"]

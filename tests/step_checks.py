"""Checks of the serving step's attention that no output escapes: every row is finite, and every row, each for itself,
is within the bound of tests/test_gpu_step.py (a NaN is within none)."""
import math

import numpy as np

from kv_cache_quantization_turbo_gb300 import workloads as W
from oracle import step_oracle as S
import gpu_common as C
import test_gpu_step as T


def assert_rows(got, want, bound):
    """got and want [rows, heads, d], bound [rows, heads] relative to the row; a row that is zeros in want is zeros."""
    assert np.isfinite(got).all(), f"{int((~np.isfinite(got)).any(-1).sum())} rows are not finite"
    empty = ~want.any(-1)
    assert not got[empty].any(), "a row without keys is not zeros"
    bad = ~(C.rel_err_per_head(got, want) < bound) & ~empty
    assert not bad.any(), (np.argwhere(bad)[:8].tolist(), float(C.rel_err_per_head(got, want)[bad].max()))


def check_attend(P, G, dtype, out_dtype=None, *, seed=3, softcap=0.0, window=0, bias=False, first=None, prefix=None,
                 rows=None, scale=None, q=None):
    """The call on N(0, 1) queries (or q) against the oracle over what the cache holds."""
    Hq = P.H * G
    if q is None:
        q = W.normal_tensor((P.n_tokens, Hq + 2, P.d), seed=seed, device="cuda").to(dtype)[:, 1:1 + Hq]
    m = T.mods_of(P, Hq, softcap, window, bias, first, prefix)
    out = T.attend(P, q, out_dtype, m, scale=scale)
    assert T.status(P.ctx) == 0
    got, q64, scale = T.f64(out), T.f64(q), scale or 1 / math.sqrt(P.d)
    assert np.all(got[P.rows:] == 9.0)
    slopes = None if m.slopes is None else T.f64(m.slopes)
    for b in range(len(P.new)):
        at = np.nonzero(P.seq == b)[0]
        if rows is not None:
            at = at[np.isin(at, rows)]
        if not len(at):
            continue
        k, v = P.stored(b)
        kw = dict(softcap=softcap, window=window, slopes=slopes,
                  first_keys=None if first is None else np.asarray(first)[at],
                  prefix=0 if prefix is None else int(prefix[b]))
        want = S.chunk_attention(q64[at], k, v, P.pos[at], scale, **kw)
        bound = T.row_bound(q64[at], k, v, P.pos[at], want, dtype, scale, **kw)
        assert_rows(got[at], want, np.maximum(bound, C.ATTN_RTOL) + T.half_step(out.dtype))
    return out

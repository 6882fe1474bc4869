"""Attention over f8_block caches whose blocks' scales lie far apart, in the kernels for few rows, for many and over staged
tiles, against the fp64 oracle.

Tolerances, fixed before the first run, per coordinate: the bound of tests/test_gpu_f8.py with every term weighted by what
the row sees, so that neither a hidden key nor one without weight widens it.
  sum_j w_j e_j (|v_j| + |o|) + A (2^-11 + 2^-20) + n 2^-28 2^s 448 max_j w_j 2^E_j, A = sum_j w_j |v_j|, plus half a step of
the output.  e_j, the error of a score: (d + 16) 2^-23 S_j for the sum, 2^-24 q_max scale sum_i |k_ji| for what fp16 leaves
of a query, 2^-22 (|s_j| + |s_max|) for the products with log2 e and the scales (fp32 queries in the kernels for many rows:
2^-11 S_j more).  The last term: a weight in fp16 is off by 2^-25 at most below the normal numbers, the row's largest weight
times its V block's scale 2^E_j is 2^3 or more of the same unit, and a code at most 448; s: exponents by which the scales
of one staged tile may differ while its weights count by the largest one, 8.
"""
import math

import numpy as np
import pytest
import torch

import test_gpu_f8 as F
from test_gpu_f8 import DT, S, W, ctxs, f64, rounding, status, tq  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu

KERNELS = ["few", "many", "staged"]
# query heads of the KV head, new tokens, context
SIZES = {"few": (2, 3, 609), "many": (2, 100, 601), "staged": (8, 700, 1301)}


def bound(q, k, v, exps, pos, scale, kernel, dtype, missing=None, softcap=0.0, slopes=None, **seen):
    """The oracle's row of query head vectors q [Hq, d] at a position (one KV head), and each coordinate's bound."""
    j = S.seen(pos, len(k), **seen)
    want = S.chunk_attention(q[None], k[:, None], v[:, None], [pos], scale, missing=missing, softcap=softcap, slopes=slopes,
                             **seen)[0]
    if missing is not None:
        j = j[~missing[j]]
    kk, vv = k[j], v[j]
    tol = np.zeros_like(want)
    for h in range(len(q)):
        s = kk @ q[h] * scale
        size = np.abs(kk) @ np.abs(q[h]) * abs(scale)
        e = (k.shape[1] + 16) * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(q[h]).max() * abs(scale) * np.abs(kk).sum(-1)
        if dtype == torch.float32 and kernel != "few":
            e = e + 2.0 ** -11 * size
        if softcap:
            s = softcap * np.tanh(s / softcap)
            e = e + 1e-6 * np.abs(s)
        if slopes is not None:
            s = s - float(slopes[h]) * np.abs(pos - j)
        w = np.exp(s - s.max())
        w /= w.sum()
        e = e + 2.0 ** -22 * (np.abs(s) + abs(s.max()))
        # keys of no weight have none with their error either
        none = s < s.max() - 60
        assert (s[none] + e[none] < s.max() - 50).all() and e[~none].max() < 1
        e = np.where(none, 0.0, e)
        a = w @ np.abs(vv)
        tail = 2.0 ** (-28 + (8 if kernel == "staged" else 0)) * 448 * (w * 2.0 ** exps[j]).max()
        tol[h] = (w * e) @ (np.abs(vv) + np.abs(want[h])) + a * (2.0 ** -11 + 2.0 ** -20) + len(j) * tail
    return want, tol


def exponents(c, view):
    word = view.header.view(torch.int32).cpu().numpy().view(np.uint32)[c.vectors(0, np.arange(c.lens[0]))[:, 0] // 16]
    return (word >> 23).astype(np.int64) - 127


def filled(ctx, d, kernel, k_of, v_of, dtype=torch.float16, seed=5, **kw):
    """One sequence, one KV head; k_of, v_of: factors of the keys [total]."""
    G, new, total = SIZES[kernel]
    c = F.Cache(ctx, d, 1, [new], [total], 16, **kw)
    i = torch.arange(total, device="cuda")
    k = W.normal_tensor((total, 1, d), seed=seed, device="cuda") * k_of(i)[:, None, None]
    v = W.normal_tensor((total, 1, d), seed=seed + 1, device="cuda") * v_of(i)[:, None, None]
    return c, k, v, G


def rows_of(new):
    return np.unique(np.concatenate([np.linspace(0, new - 1, 12).astype(int), [min(new - 1, 63), min(new - 1, 64)]]))


def check(c, G, q, kernel, scale, rows=None, missing=None, stored=None, exps=None, **kw):
    mods = tq.ScoreMods(**kw | ({"slopes": torch.as_tensor(kw["slopes"], dtype=torch.float32, device="cuda")} if "slopes" in kw
                                else {})) if kw else None
    out = F.attend(c, q, mods, torch.float32, scale=scale, least=kernel != "staged")
    torch.cuda.synchronize()
    assert status(c.ctx) == (0 if missing is None else 2)
    if kernel == "staged":
        least = tq.tq_chunk_workspace_bytes(c.ctx.h, c.batch, G, 1)
        assert tq.tq_chunk_workspace_for(c.ctx.h, c.batch, G, c.kv, c.vv, mods) > least
    k, v = (x[:, 0] for x in (stored or c.stored(0)))
    exps, got, q64 = exponents(c, c.vv) if exps is None else exps, f64(out), f64(q)
    for i in rows_of(c.rows) if rows is None else rows:
        want, tol = bound(q64[i], k, v, exps, int(c.pos[i]), scale, kernel, q.dtype, missing, **kw)
        err = np.abs(got[i] - want)
        ok = err <= tol + rounding(out.dtype, want)
        assert ok.all(), (int(i), np.argwhere(~ok)[:4].tolist(), float((err / (tol + 1e-300)).max()), float(np.abs(want).max()))
    return out


def kernels_of(d):
    return [x for x in KERNELS if x != "staged" or d != 256]


CASES = [(d, x) for d in (64, 128, 256) for x in kernels_of(d)]


@pytest.mark.parametrize("d,kernel", CASES)
@pytest.mark.parametrize("power", [12, 20, 30, 60])
def test_values_of_keys_without_weight(ctxs, d, kernel, power):  # noqa: F811
    """Values 2^power larger in keys that every row sees and none weighs (scores 80 lower), ahead of the others, among them
    and behind them."""
    for place in (lambda i: i < 128, lambda i: i // 16 % 3 == 1, lambda i: (i >= 448) & (i < 560), lambda i: i < 16):
        c, k, v, G = filled(ctxs[d], d, kernel, lambda i: torch.zeros_like(i, dtype=torch.float32),
                            lambda i: torch.where(place(i), 2.0 ** power, 1.0))
        k[place(torch.arange(len(k), device="cuda")), 0, 0] = -1.0
        c.append([len(k)], [len(k)], k, v, oracle=False)
        q = torch.zeros((c.n_tokens, G, d), dtype=torch.float16, device="cuda")
        q[:, :, 0] = 80.0
        check(c, G, q, kernel, 1.0)


@pytest.mark.parametrize("d,kernel", CASES)
@pytest.mark.parametrize("power", [12, 30, 70])
def test_values_of_hidden_keys(ctxs, d, kernel, power):  # noqa: F811
    """Values 2^power larger from a block on: rows before it are those of the cache without, up to their bounds, in the same
    tile and the same warp as rows that see them."""
    G, new, total = SIZES[kernel]
    begin = (total - new // 2) // 16 * 16  # a block in the new tokens
    if kernel == "few":
        begin = total // 16 * 16  # the last token alone
    for up in (power, 0):
        c, k, v, _ = filled(ctxs[d], d, kernel, torch.ones_like, lambda i: torch.where(i >= begin, 2.0 ** up, 1.0))
        c.append([total], [total], k.float(), v, oracle=False)
        q = W.normal_tensor((c.n_tokens, G, d), seed=9, device="cuda").half()
        near = [i for i in (begin - 1, begin - 2, begin - 16, begin, begin + 1) if total - new <= i < total]
        out = check(c, G, q, kernel, 1 / math.sqrt(d), rows=[i - (total - new) for i in near])
        if up:
            first = out
    same = int(begin - (total - new))
    big = (first[:same] - out[:same]).abs().max() / out[:same].abs().max()
    assert big < 2.0 ** -9  # (each is within 2^-11 of the weights' sizes and its scores' errors)


@pytest.mark.parametrize("d,kernel", CASES)
def test_keys_of_hidden_blocks(ctxs, d, kernel):  # noqa: F811
    """Keys 2^40 larger from a block on, which no checked row sees; the softmax scale makes scores of the small ones."""
    G, new, total = SIZES[kernel]
    begin = (total - new // 2) // 16 * 16 if kernel != "few" else total // 16 * 16
    c, k, v, _ = filled(ctxs[d], d, kernel, lambda i: torch.where(i >= begin, 1.0, 2.0 ** -40), torch.ones_like)
    c.append([total], [total], k, v.float(), oracle=False)
    q = W.normal_tensor((c.n_tokens, G, d), seed=9, device="cuda").half()
    near = [i for i in (begin - 1, begin - 2, begin - 17) if total - new <= i < total]
    check(c, G, q, kernel, 2.0 ** 40 / math.sqrt(d), rows=[i - (total - new) for i in near])


@pytest.mark.parametrize("d,kernel", CASES)
@pytest.mark.parametrize("dtype", list(DT))
def test_values_that_grow_and_fall(ctxs, d, kernel, dtype):  # noqa: F811
    """Scales that change by powers of two from block to block, up to 2^50 along the context, falling where the weight falls
    and rising where it falls."""
    G, new, total = SIZES[kernel]
    for sign in (1, -1):
        def v_of(i):
            b = torch.div(i, 16, rounding_mode="floor").float()
            return 2.0 ** ((sign * 50.0 * (b * 16 / total - 0.5)).floor() + b * 7 % 11)
        c, k, v, _ = filled(ctxs[d], d, kernel, lambda i: 0.1 * torch.ones_like(i, dtype=torch.float32), v_of)
        k[:, 0, 0] = torch.arange(total, device="cuda") / total
        c.append([total], [total], k, v, oracle=False)
        q = W.normal_tensor((c.n_tokens, G, d), seed=9, device="cuda")
        for slope in (0.0, 30.0, -30.0):
            q[:, :, 0] = slope
            check(c, G, q.to(DT[dtype]), kernel, 1.0)


@pytest.mark.parametrize("d,kernel", CASES)
@pytest.mark.parametrize("span", [7, 8, 9, 10, 23, 40])
def test_spans_within_a_tile(ctxs, d, kernel, span):  # noqa: F811
    """Every other block 2^span larger, of keys, of values and of both, the larger ones heavier, lighter or alike."""
    for of_k, of_v, heavy in ((span, 0, 0), (0, span, 1), (0, span, -1), (span, span, 0)):
        def up(i, n):
            return 2.0 ** (i // 16 % 2 * n).float()
        c, k, v, G = filled(ctxs[d], d, kernel, lambda i: up(i, of_k), lambda i: up(i, of_v))
        k[:, 0, 0] = torch.arange(len(k), device="cuda") // 16 % 2 * heavy
        c.append([len(k)], [len(k)], k, v, oracle=False)
        q = W.normal_tensor((c.n_tokens, G, d), seed=9, device="cuda").half()
        if heavy:
            q[:, :, 0] = 10.0
        # Scores of the large keys of order 1, or of the small ones, as far as an error e_j stays below 1 (fp32's step of a
        # score of 2^40 is 2^17: no weight follows from it).
        for scale in (2.0 ** -of_k / math.sqrt(d), 1 / math.sqrt(d))[:2 if of_k <= 10 else 1]:
            check(c, G, q, kernel, scale, rows=rows_of(c.rows)[::3])


@pytest.mark.parametrize("d,kernel", CASES)
def test_windows_over_scales_far_apart(ctxs, d, kernel):  # noqa: F811
    """A window whose sinks have values 2^40 larger and scores 60 lower; scores from -3000 to 3000."""
    G, new, total = SIZES[kernel]
    c, k, v, _ = filled(ctxs[d], d, kernel, torch.zeros_like, lambda i: torch.where(i < 16, 2.0 ** 40, 1.0))
    k = k.float()
    k[:16, 0, 0] = -1.0
    c.append([total], [total], k, v, oracle=False)
    q = torch.zeros((c.n_tokens, G, d), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 60.0
    check(c, G, q, kernel, 1.0, window=500 if kernel == "staged" else 300, sinks=16)
    c, k, v, _ = filled(ctxs[d], d, kernel, torch.zeros_like, lambda i: 2.0 ** (i // 16 % 5 * 6).float())
    k = k.float()
    k[:, 0, 0] = torch.linspace(-1, 1, total, device="cuda")
    c.append([total], [total], k, v, oracle=False)
    for s in (3000.0, -3000.0):
        q[:, :, 0] = s
        check(c, G, q, kernel, 1.0)


@pytest.mark.parametrize("d,kernel", CASES)
def test_modified_scores_marks_and_missing_pages_over_scales_far_apart(ctxs, d, kernel):  # noqa: F811
    """Blocks 2^30 apart under capped and biased scores; a marked vector makes NaN of the rows that see it alone, a
    page out of range is left out."""
    G, new, total = SIZES[kernel]
    c, k, v, _ = filled(ctxs[d], d, kernel, lambda i: 2.0 ** -(i // 16 % 4 * 10.0), lambda i: 2.0 ** (i // 16 % 3 * 15.0))
    c.append([total], [total], k, v, oracle=False)
    q = W.normal_tensor((c.n_tokens, G, d), seed=9, device="cuda").half()
    scale, mods = 1 / math.sqrt(d), dict(softcap=30.0, slopes=np.full(G, 0.0078125))
    stored, exps = c.stored(0), exponents(c, c.vv)
    for kw in ({}, mods):
        check(c, G, q, kernel, scale, **kw)
    marked = total - max(2, new // 2)
    vec = int(c.vectors(0, [marked])[0, 0])
    c.vv.header.view(torch.int32)[vec // 16] |= 1 << vec % 16
    before = int(marked - (total - new))
    for kw in ({}, mods):
        out = check(c, G, q, kernel, scale, rows=rows_of(before), stored=stored, exps=exps, **kw)
        assert torch.isnan(out[before:new]).all()
    c.vv.header.view(torch.int32)[vec // 16] &= ~(1 << vec % 16)
    c.table = c.table.copy()
    c.table[0, [3, 20]] = [10 ** 6, -5]
    c.set_batch([new], [total])
    missing = np.isin(np.arange(total) // 16, [3, 20])
    for kw in ({}, mods):
        check(c, G, q, kernel, scale, missing=missing, stored=stored, exps=exps, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("G,new", [(1, 1), (4, 1), (2, 3), (8, 2)])
def test_weights_of_few_rows_are_not_rounded(ctxs, d, dtype, G, new):  # noqa: F811
    """Kernel for few rows: weights have 22 bits.  Keys and queries of one coordinate have scores of one product, so a row of
    few keys is off by 2^-22 (|s_j| + |s_max|) for the product with log2 e and the scales, 2^-22 |s_j| for what two fp16 numbers
    leave of an fp32 query, 2^-21 of the weights (2^-22 for what two fp16 numbers leave of one, 2^-22 for the exponential),
    2^-28 448 of the largest product of weight and scale for what of a small one is below fp16, and 2^-20 for its sums in
    fp32 (16 additions at most).  The output is fp32."""
    if new * G > (8 if d == 256 else 16):
        pytest.skip("these are many rows")
    for total in (16, 5, 37):
        c = F.Cache(ctxs[d], d, 1, [new], [total], 16)
        k, v = torch.zeros((total, 1, d), device="cuda"), W.normal_tensor((total, 1, d), seed=32 + total, device="cuda")
        k[:, 0, 3] = W.normal_tensor((total, 1), seed=31, device="cuda")[:, 0]
        c.append([total], [total], k, v, oracle=False)
        q = torch.zeros((new, G, d), device="cuda")
        q[:, :, 3] = 1 + 0.3 * W.normal_tensor((new, G), seed=9, device="cuda")
        q = q.to(DT[dtype])
        out = F.attend(c, q, None, torch.float32, scale=1.0)
        torch.cuda.synchronize()
        assert status(c.ctx) == 0
        k, v = (y[:, 0] for y in c.stored(0))
        exps = exponents(c, c.vv)
        for t in range(new):
            j = np.arange(int(c.pos[t]) + 1)
            for h in range(G):
                s = k[j] @ f64(q)[t, h]
                w = np.exp(s - s.max())
                w /= w.sum()
                want = w @ v[j]
                e = 2.0 ** -22 * (2 * np.abs(s) + abs(s.max())) + 2.0 ** -21 + 2.0 ** -20
                tol = (w * e) @ (np.abs(v[j]) + np.abs(want)) + len(j) * 2.0 ** -28 * 448 * (w * 2.0 ** exps[j]).max()
                assert (np.abs(f64(out)[t, h] - want) <= tol).all(), (t, h, float((np.abs(f64(out)[t, h] - want) / tol).max()))

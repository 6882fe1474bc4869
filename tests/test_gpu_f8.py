"""GPU parity of f8_block caches (tq_append_kv, tq_read_kv, tq_dequantize, tq_chunk_attention) and of windows with sinks over
every format, against the fp64 oracle.

Tolerances, fixed before the first run.
  * append: without a rotation every code, scale and mark equals the oracle's (x / 2^e is exact, so is its rounding).  With
    one, a key's coordinates are off by 6e-7 (|x_p| + |x_q|), so a code may be that of a value so far away: the stored value
    is within half a step of e4m3 (2^-4 relative, 2^-10 2^e below the normal numbers) of the exact one, plus that error; the
    scale is equal unless the block's maximum is that near to 448 * 2^k (the inputs here are not: asserted).
  * attention.  K and V are exact operands.  To first order a row is off by sum_j w_j (r_j v_j + e_j (v_j - o)): r_j, the
    rounding of a weight to fp16, is at most 2^-11, plus 2^-21 for ex2 (2^-22) and its argument's last product; e_j the
    error of a score: (d + 16) 2^-23 S_j for the sum, S_j = scale sum_i |q_i k_ji|, plus 2^-22 max |s| for the product with
    log2 e and the reference, plus the queries' rounding: fp16 and bf16 queries are exact in fp16 down to 2^-24 of the row's
    largest, q_max: 2^-24 q_max scale sum_i |k_ji|; fp32 ones in the kernel for many rows 2^-11 S_j.  A weight below fp16's
    normal numbers is off by 2^-25 absolute where the row's largest is 2^4 or more, and V blocks of smaller scale count
    relative to the largest: n 2^-29 max |v|.  So |error| <= A (2^-11 + 2^-20) + 2 A max_j e_j + n 2^-29 max |v| per
    coordinate, A = sum_j w_j |v_j| (|o| <= A), plus half a step of the output.
"""
import math

import numpy as np
import pytest
import torch

import step_checks as K
import test_gpu_step as T
from test_gpu_step import DT, ctxs, f64, rounding, status  # noqa: F401  (ctxs: the fixture)
from kv_cache_quantization_turbo_gb300 import tq
from kv_cache_quantization_turbo_gb300 import workloads as W
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


class Cache:
    """A paged f8_block cache of a ragged batch, and what the oracle holds: blocks[kind][sequence][block][head].  Everything
    that no token owns is filled with codes and words of other scales."""

    def __init__(self, ctx, d, H, new, lens, page, *, seed=0, n_layers=1, layer=0, contiguous=False, padding=0):
        self.ctx, self.d, self.H, self.page, self.layer = ctx, d, H, page, layer
        self.new, self.lens = np.asarray(new, np.int64), np.asarray(lens, np.int64)
        B = len(self.new)
        if contiguous:
            self.table, n_pages = None, B + 1
        else:
            self.table, n_pages = W.shuffled_block_table(self.lens, page, seed=seed + 9, extra_pages=3)
        self.kv, self.vv = (tq.alloc_view("f8_block", d, H, page, n_pages, n_layers) for _ in range(2))
        g = torch.Generator(device="cuda").manual_seed(seed)
        for view in (self.kv, self.vv):
            view.payload.copy_(torch.randint(0, 256, view.payload.shape, dtype=torch.uint8, device="cuda", generator=g))
            e = torch.randint(47, 208, (view.header.numel() // 4,), device="cuda", generator=g, dtype=torch.int32)
            view.header.view(torch.int32).copy_(e << 23 | 0xFFFF)
        self.blocks = {x: [dict() for _ in range(B)] for x in "kv"}
        self.padding = padding
        self.set_batch(self.new, self.lens)

    def batch_of(self, new, lens, padding=0, **kw):
        new, lens = np.asarray(new, np.int64), np.asarray(lens, np.int64)
        dev = dict(dtype=torch.int32, device="cuda")
        cu = torch.as_tensor(np.concatenate([[0], np.cumsum(new)]), **dev)
        a = dict(max_tokens=int(max(new, default=0)), max_ctx=int(max(lens, default=0))) | kw
        return tq.Batch(cu, torch.as_tensor(lens, **dev), None if self.table is None else torch.as_tensor(self.table, **dev),
                        int(new.sum()) + padding, a["max_tokens"], a["max_ctx"])

    def set_batch(self, new, lens, **kw):
        self.new, self.lens = np.asarray(new, np.int64), np.asarray(lens, np.int64)
        self.seq, self.pos = S.batch_positions(self.new, self.lens)
        self.rows, self.n_tokens = len(self.seq), len(self.seq) + self.padding
        self.batch = self.batch_of(new, lens, self.padding, **kw)

    def append(self, new, lens, k, v, *, rope=None, stream=None, oracle=True):
        """k, v [tokens (+ padding), H, d] of any type, to the cache and to the oracle's blocks."""
        b = self.batch_of(new, lens, k.shape[0] - int(np.sum(new)))
        table, angles, m, layout = rope or (None, None, 1.0, "half")
        st = tq.tq_append_kv(self.ctx.h, b, k, v, self.kv, self.vv, self.layer, rope=table, stream=stream)
        assert st == tq.TQ_OK, tq.tq_status_string(st)
        if not oracle:
            return
        seq, pos = S.batch_positions(np.asarray(new), np.asarray(lens))
        x = {"k": f64(k)[:len(seq)], "v": f64(v)[:len(seq)]}
        if rope is not None:
            x["k"] = S.rope(x["k"], pos, angles, m, layout)
        for name in "kv":
            for s in range(len(new)):
                at = np.flatnonzero(seq == s)
                blocks = self.blocks[name][s]
                for n in np.unique(pos[at] // 16):
                    rows = at[pos[at] // 16 == n]
                    for h in range(self.H):
                        blocks.setdefault((n, h), S.F8Block(self.d)).append(x[name][rows, h], int(pos[rows[0]] % 16))

    def fill(self, seed=100, scale=None, outliers=0.0):
        """Whole sequences at once, through the call itself."""
        n = int(self.lens.sum())
        x = [W.kv_tensor(n, self.H, self.d, seed=seed + i, device="cuda", outlier_frac=outliers).float() for i in range(2)]
        if scale is not None:
            x = [y * scale(torch.arange(n, device="cuda"), i)[:, None, None] for i, y in enumerate(x)]
        self.append(self.lens, self.lens, *x, oracle=False)
        return self

    def vectors(self, b, pos):
        page = np.full(len(pos), b) if self.table is None else self.table[b, np.asarray(pos) // self.page].astype(np.int64)
        first = (self.layer * self.kv.num_pages + page) * self.H
        return (first[:, None] + np.arange(self.H)) * self.page + (np.asarray(pos) % self.page)[:, None]

    def stored(self, b):
        """Values [T, H, d] of sequence b's tokens as the bytes have them, by the documented layout."""
        out = []
        for view in (self.kv, self.vv):
            v = self.vectors(b, np.arange(self.lens[b]))
            pay = view.payload.view(-1, self.d).cpu().numpy()[v]
            word = view.header.view(torch.int32).cpu().numpy().view(np.uint32)[v // 16]
            scale = (word & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)
            x = S.e4m3_values()[pay] * scale[..., None]
            x[(word >> (v % 16).astype(np.uint32)) & 1 == 1] = np.nan
            out.append(x)
        return out

    def check_blocks(self, rotated=False):
        """Every token that the oracle has against the stored bytes."""
        torch.cuda.synchronize()
        assert status(self.ctx) == 0
        for s in range(len(self.lens)):
            for name, got in zip("kv", self.stored(s)):
                for (n, h), block in self.blocks[name][s].items():
                    want = block.values()
                    have = got[16 * n:16 * n + len(want), h]
                    if rotated and name == "k":
                        # a code's neighbour where the exact value is that near to the middle of two
                        step = np.maximum(2.0 ** -3 * np.abs(want), 2.0 ** (block.e - 9))
                        off = np.abs(have - want)
                        assert ((off == 0) | (off <= 1.001 * step)).all() and (off > 0).mean() < 1e-2
                        continue
                    np.testing.assert_array_equal(have, want, err_msg=f"{name} of sequence {s}, block {n}, head {h}")


def tokens(n, H, d, dtype, seed):
    """k and v as slices of a fused projection, some channels larger."""
    buf = W.normal_tensor((n, 3 * H, d), seed=seed, device="cuda")
    buf[..., 3] *= 20.0
    return buf.to(dtype)[:, H:2 * H], buf.to(dtype)[:, 2 * H:]


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48])
def test_append_in_steps(ctxs, dtype, d, page):  # noqa: F811
    """Chunks and single tokens one after the other, growing values (scales that rise under earlier tokens) and falling
    ones, blocks entered at every offset, a sequence without tokens."""
    lens = [70, 33, 5, 50]
    c = Cache(ctxs[d], d, 3, lens, lens, page, padding=2)
    at = np.zeros(4, np.int64)
    rng = np.random.default_rng(d + page)
    step = 0
    while (at < lens).any():
        new = np.minimum(rng.choice([0, 1, 1, 2, 7, 17, 30], 4), lens - at)
        at = at + new
        k, v = tokens(int(new.sum()) + 2, 3, d, torch.float32, 10 + step)
        size = 2.0 ** rng.integers(-3, 4, 2) * (1.3 ** step if step < 20 else 0.1)
        c.append(new, at, (k * size[0]).to(DT[dtype]), (v * size[1]).to(DT[dtype]))
        step += 1
    c.check_blocks()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rotary", [(128, 128), (64, 20), (256, 126), (128, 32)])
def test_append_rotated(ctxs, layout, d, rotary):  # noqa: F811
    t = tq.tq_rope_build(d, rotary, layout, "yarn", base=1e4, factor=4.0, original_ctx=2048.0)
    rope = (t, *S.rope_angles(rotary, "yarn", base=1e4, factor=4.0, original_ctx=2048.0), layout)
    for dtype in DT.values():
        c = Cache(ctxs[d], d, 2, [40, 9], [40, 9], 16)
        for new, lens in (([20, 1], [20, 1]), ([3, 8], [23, 9]), ([17, 0], [40, 9])):
            k, v = tokens(sum(new), 2, d, dtype, sum(lens))
            c.append(new, lens, k, v, rope=rope)
        for blocks in c.blocks["k"]:  # the scales' maxima are not at a border, so they are the same
            for b in blocks.values():
                top = np.abs(b.codes).max()
                assert abs(top - 448) > 1e-3 or top == 448
        c.check_blocks(rotated=True)


def test_append_positions_of_the_callers(ctxs):  # noqa: F811
    """Positions given by the caller turn the keys, the places stay those of the sequence."""
    d = 64
    t = tq.tq_rope_build(d)
    k, v = tokens(20, 1, d, torch.float32, 1)
    pos = torch.arange(20, dtype=torch.int32, device="cuda") * 31 + 1000
    turned = torch.empty((20, 1, d), device="cuda")
    assert tq.tq_rope(ctxs[d].h, t, k, pos, turned) == tq.TQ_OK
    outs = []
    for kk, kw in ((k, dict(rope=t, positions=pos)), (turned, {})):
        c = Cache(ctxs[d], d, 1, [20], [20], 16)
        assert tq.tq_append_kv(c.ctx.h, c.batch, kk, v, c.kv, c.vv, 0, **kw) == tq.TQ_OK
        torch.cuda.synchronize()
        outs.append(c.stored(0))
    off = np.abs(outs[0][0] - outs[1][0])  # the two rotations differ in their last bits: a code's neighbour now and then
    assert (off <= np.maximum(2.0 ** -3, np.abs(outs[1][0]) * 2.0 ** -3)).all() and (off > 0).mean() < 1e-3
    np.testing.assert_array_equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("H,new", [(1, [1]), (11, [600]), (16, [2048, 1]), (5, [1] * 70), (8, [37, 16, 15, 17] * 40)])
def test_append_sizes(ctxs, H, new):  # noqa: F811
    c = Cache(ctxs[64], 64, H, new, new, 32)
    k, v = tokens(sum(new), H, 64, torch.float16, 3)
    c.append(new, new, k, v)
    c.check_blocks()


def test_append_rolls_back(ctxs):  # noqa: F811
    """Tokens taken back and others written in their place (speculative steps): earlier tokens keep their values, the
    block's scale stays."""
    d = 128
    c = Cache(ctxs[d], d, 2, [6], [30], 16)
    spare = sorted(set(range(c.kv.num_pages)) - set(c.table[0].tolist()))[0]
    c.table = np.array([[*c.table[0], spare]], np.int32)
    for new, total in ((30, 30), (4, 24), (1, 25), (9, 34), (20, 20)):
        k, v = tokens(new, 2, d, torch.bfloat16, total)
        c.blocks = {x: [{b: y for b, y in c.blocks[x][0].items() if 16 * b[0] < total}] for x in "kv"}
        c.append([new], [total], k * (3.0 if new == 4 else 1.0), v)
        c.lens = np.array([total])
        c.check_blocks()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_marks_of_vectors_that_are_not_finite(ctxs, d):  # noqa: F811
    """NaN, infinities and magnitudes above 448 * 2^80: their vectors alone read back as NaN, later appends keep the marks
    of earlier tokens and clear those of replaced ones."""
    c = Cache(ctxs[d], d, 2, [20], [20], 16)
    k, v = tokens(20, 2, d, torch.float32, 1)
    k, v = k.clone(), v.clone()
    k[0, 0, 5], k[3, 1, d - 1], k[7, 0, 0] = float("nan"), float("inf"), 448 * 2.0 ** 80
    v[2, 1, 1], v[17, 0, 9], v[5, 0, 2] = -float("inf"), 5.42e26 * 1.01, -448 * 2.0 ** 80 * 1.0001
    c.append([20], [20], k, v)
    c.check_blocks()
    assert np.isnan(c.stored(0)[0][0, 0]).all() and np.isnan(c.stored(0)[1][17, 0]).all()
    assert np.isfinite(c.stored(0)[0][7, 0]).all()
    k, v = tokens(4, 2, d, torch.float32, 2)
    c.append([4], [7], k, v)  # over positions 3 to 6
    c.lens = np.array([7])
    c.blocks = {x: [{b: y for b, y in c.blocks[x][0].items() if b[0] == 0}] for x in "kv"}
    c.check_blocks()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_and_dequantize(ctxs, d, dtype):  # noqa: F811
    """Every stored value, rounded once to the output type; padding rows stay; both views, one, and mixed formats."""
    c = Cache(ctxs[d], d, 3, [40, 5], [40, 5], 16, padding=3)
    k, v = tokens(45, 3, d, torch.float32, 4)
    k = k.clone()
    k[2, 1, 0] = float("nan")
    c.append([40, 5], [40, 5], k, v)
    outs = [torch.full((48, 3, d), 9.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    assert tq.tq_read_kv(c.ctx.h, c.batch, c.kv, outs[0], c.vv, outs[1], 0) == tq.TQ_OK
    alone = torch.full_like(outs[1], 9.0)
    assert tq.tq_read_kv(c.ctx.h, c.batch, None, None, c.vv, alone, 0) == tq.TQ_OK
    q8 = tq.alloc_view("q8_0", d, 3, 16, c.kv.num_pages)
    mixed = [torch.full_like(o, 9.0) for o in outs]
    assert tq.tq_read_kv(c.ctx.h, c.batch, q8, mixed[0], c.vv, mixed[1], 0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert torch.equal(alone, outs[1]) and torch.equal(mixed[1], outs[1]) and not mixed[0][:45].any()
    for i, o in enumerate(outs):
        want = np.concatenate([c.stored(s)[i] for s in range(2)])
        np.testing.assert_array_equal(f64(o)[:45], f64(torch.as_tensor(want).to(DT[dtype])))
        assert (o[45:] == 9.0).all()
    slots = torch.as_tensor((c.table[0, np.arange(40) // 16].astype(np.int64) * 16 + np.arange(40) % 16), device="cuda")
    deq = torch.empty((40, 3, d), device="cuda")
    assert tq.tq_dequantize(c.ctx.h, c.kv, 0, slots, 0, 40, 0, deq) == tq.TQ_OK
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(deq), c.stored(0)[0])


def test_append_and_read_skip_what_is_out_of_range(ctxs):  # noqa: F811
    d = 64
    c = Cache(ctxs[d], d, 2, [20, 20, 4], [40, 20, 4], 16)
    c.append([20, 0, 0], [20, 0, 0], *tokens(20, 2, d, torch.float16, 6), oracle=False)  # the first one's earlier tokens
    keep = [x.clone() for view in (c.kv, c.vv) for x in (view.payload, view.header)]
    c.table = c.table.copy()
    c.table[0, 2], c.table[1, 0] = -3, 10 ** 6
    k, v = tokens(44, 2, d, torch.float16, 5)
    b = c.batch_of([20, 20, 4], [40, 20, 3])  # the last: more new tokens than its length
    assert tq.tq_append_kv(c.ctx.h, b, k, v, c.kv, c.vv, 0) == tq.TQ_OK
    out = torch.full((44, 2, d), 9.0, device="cuda")
    assert tq.tq_read_kv(c.ctx.h, b, c.kv, out, None, None, 0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert status(c.ctx) == 3
    there = np.concatenate([np.arange(20) < 12, np.arange(20) >= 16, np.zeros(4, bool)])
    assert not out[torch.as_tensor(~there, device="cuda")].any()
    assert out[torch.as_tensor(there, device="cuda")].any(-1).all()
    touched = np.unique(np.concatenate([c.vectors(0, np.arange(20, 32)).ravel(), c.vectors(1, np.arange(16, 20)).ravel()]))
    now = [x for view in (c.kv, c.vv) for x in (view.payload, view.header)]
    for i, (a, b) in enumerate(zip(keep, now)):
        changed = (a != b).view(-1, d if i % 2 == 0 else 4).any(-1).cpu().numpy()
        allowed = touched if i % 2 == 0 else np.unique(touched // 16)
        # (earlier tokens of a block are brought to its new scale)
        block = np.unique(np.concatenate([(touched // 16 * 16)[:, None] + np.arange(16)])) if i % 2 == 0 else allowed
        assert np.isin(np.flatnonzero(changed), block).all()


def test_empty_batches(ctxs):  # noqa: F811
    c = Cache(ctxs[64], 64, 1, [0, 0], [20, 0], 16, padding=5)
    keep = c.kv.payload.clone()
    k, v = tokens(5, 1, 64, torch.float16, 1)
    out = torch.full((5, 1, 64), 9.0, device="cuda")
    assert tq.tq_append_kv(c.ctx.h, c.batch, k, v, c.kv, c.vv, 0) == tq.TQ_OK
    assert tq.tq_read_kv(c.ctx.h, c.batch, c.kv, out, None, None, 0) == tq.TQ_OK
    o = attend(c, k)
    torch.cuda.synchronize()
    assert torch.equal(keep, c.kv.payload) and (out == 9.0).all() and (o == 9.0).all() and status(c.ctx) == 0


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend(c, q, mods=None, out_dtype=None, scale=None, stream=None, ws=None, out=None, least=False):
    need = tq.tq_chunk_workspace_bytes(c.ctx.h, c.batch, q.shape[1], c.H)
    n = need if least else tq.tq_chunk_workspace_for(c.ctx.h, c.batch, q.shape[1], c.kv, c.vv, mods)
    assert n >= need > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) if ws is None else ws
    if out is None:
        out = torch.full(q.shape, 9.0, dtype=out_dtype or q.dtype, device="cuda")
    st = tq.tq_chunk_attention(c.ctx.h, c.batch, q, c.kv, c.vv, c.layer, 1 / math.sqrt(c.d) if scale is None else scale, ws,
                               n, out, mods=mods, stream=stream)
    assert st == tq.TQ_OK, tq.tq_status_string(st)
    return out


def mods_of(c, Hq, softcap=0.0, window=0, bias=False, first=None, prefix=None, sinks=0):
    m = T.mods_of(c, Hq, softcap, window, bias, first, prefix)
    return tq.ScoreMods(m.softcap, m.window, m.slopes, m.first_keys, m.prefix_lens, sinks)


def expected(q, k, v, positions, scale, many, dtype, *, softcap=0.0, window=0, slopes=None, first_keys=None, prefix=0, sinks=0):
    """The oracle's rows and the bound of each coordinate, without the output's rounding."""
    want = S.chunk_attention(q, k, v, positions, scale, softcap=softcap, window=window, slopes=slopes, first_keys=first_keys,
                             prefix=prefix, sinks=sinks)
    n, Hq, d = q.shape
    tol = np.zeros_like(want)
    for i in range(n):
        j = S.seen(int(positions[i]), len(k), window, 0 if first_keys is None else int(first_keys[i]), prefix, sinks)
        if not len(j):
            continue
        for h in range(Hq):
            kk, vv = k[j, h * k.shape[1] // Hq], v[j, h * k.shape[1] // Hq]
            s = kk @ q[i, h] * scale
            size = np.abs(kk) @ np.abs(q[i, h]) * abs(scale)
            e = (d + 16) * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(q[i, h]).max() * abs(scale) * np.abs(kk).sum(-1)
            if dtype == torch.float32 and many:
                e = e + 2.0 ** -11 * size
            if softcap:
                s = softcap * np.tanh(s / softcap)
                e = e + 1e-6 * np.abs(s)
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(int(positions[i]) - j)
            e = e + 2.0 ** -22 * np.abs(s).max()
            w = np.exp(s - s.max())
            a = (w / w.sum()) @ np.abs(vv)
            tol[i, h] = a * (2.0 ** -11 + 2.0 ** -20) + 2 * a * e.max() + len(j) * 2.0 ** -29 * np.abs(vv).max()
    return want, tol


def check(c, G, dtype, out_dtype=None, *, seed=3, rows=None, scale=None, q=None, least=False, **kw):
    Hq = c.H * G
    if q is None:
        q = W.normal_tensor((c.n_tokens, Hq + 2, c.d), seed=seed, device="cuda").to(dtype)[:, 1:1 + Hq]
    m = mods_of(c, Hq, **kw)
    out = attend(c, q, m, out_dtype, scale=scale, least=least)
    torch.cuda.synchronize()
    assert status(c.ctx) == 0
    got, q64, scale = f64(out), f64(q), 1 / math.sqrt(c.d) if scale is None else scale
    assert np.all(got[c.rows:] == 9.0)
    many = int(max(c.new)) * G > (8 if c.d == 256 else 16)
    for b in range(len(c.new)):
        at = np.nonzero(c.seq == b)[0]
        if rows is not None:
            at = at[np.isin(at, rows)]
        if not len(at):
            continue
        k, v = c.stored(b)
        first = kw.get("first")
        prefix = kw.get("prefix")
        want, tol = expected(q64[at], k, v, c.pos[at], scale, many, dtype, softcap=kw.get("softcap", 0.0),
                             window=kw.get("window", 0), slopes=None if m.slopes is None else f64(m.slopes),
                             first_keys=None if first is None else np.asarray(first)[at],
                             prefix=0 if prefix is None else int(prefix[b]), sinks=kw.get("sinks", 0))
        err = np.abs(got[at] - want)
        ok = err <= tol + rounding(out.dtype, want)
        assert ok.all(), (b, np.argwhere(~ok)[:6].tolist(), float((err / (tol + 1e-30)).max()), float(err.max()))
    return out


SHAPES = [  # G, new, lens, page
    (1, [1], [1], 16),
    (4, [1, 0, 1, 1], [15, 9, 16, 17], 16),
    (8, [1], [9000], 16),
    (2, [4, 1, 3], [4, 4000, 1537], 48),
    (5, [1] * 30, list(range(3, 3003, 100)), 32),
    (16, [1, 1], [129, 257], 64),
    (1, [16, 7], [500, 7], 16),
    (1, [130], [130], 16),
    (4, [70, 3, 300], [70, 900, 301], 16),
    (7, [33, 1, 1], [1000, 2, 640], 80),
    (2, [257], [4097], 256),
    (3, [129, 128, 127], [129, 2000, 140], 32),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,new,lens,page", SHAPES)
def test_attend_shapes(ctxs, d, G, new, lens, page):  # noqa: F811
    c = Cache(ctxs[d], d, 2, new, lens, page, padding=1).fill()
    rows = None if sum(new) <= 40 else np.unique(np.linspace(0, sum(new) - 1, 40).astype(int))
    check(c, G, torch.float16, rows=rows)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", [([3, 1], [300, 50]), ([90, 1], [300, 129])])
@pytest.mark.parametrize("mods", [dict(softcap=5.0), dict(window=1), dict(window=50), dict(bias=True),
                                  dict(prefix=[200, 30]), dict(softcap=20.0, window=70, bias=True, prefix=[30, 0]),
                                  dict(window=60, sinks=5, softcap=9.0, bias=True)])
def test_attend_score_modifications(ctxs, d, shape, mods):  # noqa: F811
    c = Cache(ctxs[d], d, 2, *shape, 16).fill(outliers=0.01)
    check(c, 2, torch.bfloat16, **mods)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out_dtype", list(DT))
@pytest.mark.parametrize("new", [2, 60])
def test_attend_types(ctxs, dtype, out_dtype, new):  # noqa: F811
    check(Cache(ctxs[128], 128, 2, [new], [333], 16).fill(), 2, DT[dtype], DT[out_dtype])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 100])
def test_attend_scales_of_every_size(ctxs, d, new):  # noqa: F811
    """Block scales that rise, fall and jump by powers up to 2^60 along the context, K's and V's each in their own way; whole
    blocks of zeros; and caches whose values are all tiny or all huge: the result scales with them."""
    def jumps(i, kind):
        b = torch.div(i, 16, rounding_mode="floor")
        if kind == 0:
            return 2.0 ** -((b * 7 % 13).float())
        return torch.where(b % 5 == 3, 0.0, 2.0 ** (b * 11 % 17 - 8).float())
    check(Cache(ctxs[d], d, 2, [new], [700], 16).fill(scale=jumps), 2, torch.float16, torch.float32)
    for up in (True, False):
        def ramp(i, kind):
            b = torch.div(i, 16, rounding_mode="floor").float()
            return torch.ones_like(b) if kind == 0 else 2.0 ** ((b if up else 43 - b) - 20)
        check(Cache(ctxs[d], d, 1, [new], [700], 16).fill(scale=ramp), 2, torch.float16, torch.float32)
    for p in (-60, 60):
        c = Cache(ctxs[d], d, 1, [new], [200], 16).fill(scale=lambda i, kind: torch.full_like(i, 2.0 ** p, dtype=torch.float32))
        check(c, 2, torch.bfloat16, torch.float32, scale=2.0 ** -p / math.sqrt(d))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 100])
def test_attend_weightless_blocks_of_large_values(ctxs, d, new):  # noqa: F811
    """Values 2^30 larger in keys that no row weighs (its score is 80 lower), and small ones where the weight is."""
    c = Cache(ctxs[d], d, 1, [new], [600], 16)
    k = torch.zeros((600, 1, d), device="cuda")
    v = W.normal_tensor((600, 1, d), seed=5, device="cuda")
    large = (torch.arange(600, device="cuda") // 64) % 2 == 1
    k[large, 0, 0] = -1.0
    v[large] *= 2.0 ** 30
    c.append([600], [600], k, v, oracle=False)
    q = torch.zeros((c.n_tokens, 2, d), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 80.0
    out = attend(c, q, scale=1.0, out_dtype=torch.float32)
    torch.cuda.synchronize()
    kk, vv = c.stored(0)
    want, tol = expected(f64(q)[-4:], kk, vv, c.pos[-4:], 1.0, new > 8, torch.float16)
    small = np.abs(vv[~large.cpu().numpy()]).max()
    # what fp16 loses of a weight below 2^-14 2^-30 is nothing here: the weights are 1 and e^-80; small values count 2^-30 of
    # the large ones', so their weights of 2^4 lie at 2^-26, where fp16 keeps nothing finer than 2^-24: the bound says so
    assert (np.abs(f64(out)[-4:] - want) <= tol).all() and np.isfinite(f64(out)).all() and small < 10


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [6, 40])
def test_attend_marks_reach_those_who_see_them(ctxs, d, new):  # noqa: F811
    """A marked K or V vector: rows that see it are NaN, the others as without it."""
    for which in range(2):
        c = Cache(ctxs[d], d, 1, [new, 1], [260, 50], 16)
        x = [W.normal_tensor((310, 1, d), seed=i, device="cuda") for i in range(2)]
        c.append([260, 50], [260, 50], *x, oracle=False)
        q = W.normal_tensor((new + 1, 1, d), seed=4, device="cuda").half()
        first = np.zeros(new + 1, np.int64)
        first[[1, 3, 5]], first[2] = [131, 140, 259], 130
        m = mods_of(c, 1, first=first)
        clean = attend(c, q, m)
        x[which][130, 0, d // 2] = float("nan")
        c.append([260, 50], [260, 50], *x, oracle=False)
        got = attend(c, q, m)
        torch.cuda.synchronize()
        sees = torch.ones(new + 1, dtype=torch.bool)
        sees[[1, 3, 5, new]] = False
        assert torch.isnan(got[sees]).all()
        assert torch.equal(got[~sees], clean[~sees]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("new", [[2, 1], [40, 1]])
def test_attend_documents_empty_rows_and_pages_out_of_range(ctxs, d, new):  # noqa: F811
    ctx = ctxs[d]
    c = Cache(ctx, d, 1, new, [600, 40], 16).fill()
    n = sum(new)
    first = c.pos - c.pos % 37
    first[1] = 10 ** 9
    check(c, 2, torch.float16, first=first)
    check(c, 2, torch.float16, first=first, window=20, sinks=4)
    q = W.normal_tensor((n, 2, d), seed=8, device="cuda").half()
    k, v = c.stored(0)
    c.table = c.table.copy()
    c.table[0, [1, 20]] = [-7, 10 ** 6]
    c.set_batch(new, [600, 40])
    out = attend(c, q)
    torch.cuda.synchronize()
    assert status(ctx) == 2
    missing = np.zeros(600, bool)
    missing[16:32] = missing[320:336] = True
    at = np.flatnonzero(c.seq == 0)
    want = S.chunk_attention(f64(q)[at], k, v, c.pos[at], 1 / math.sqrt(d), missing=missing)
    _, tol = expected(f64(q)[at], k, v, c.pos[at], 1 / math.sqrt(d), True, torch.float16)
    assert (np.abs(f64(out)[at] - want) <= 2 * tol + rounding(out.dtype, want)).all()


def test_attend_contiguous_layers_and_neighbours(ctxs):  # noqa: F811
    for new in ([1, 2], [50, 20]):
        c = Cache(ctxs[128], 128, 2, new, [150, 96], 160, contiguous=True, n_layers=3, layer=1).fill()
        check(c, 2, torch.float16)


@pytest.mark.parametrize("new", [1, 300])
def test_attend_repeats_streams_and_graphs(ctxs, new):  # noqa: F811
    c = Cache(ctxs[128], 128, 2, [new, 1], [2000, 700], 16).fill()
    q = W.normal_tensor((c.n_tokens, 8, 128), seed=1, device="cuda").half()
    m = mods_of(c, 8, window=900, sinks=3)
    want = [attend(c, q), attend(c, q, m)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attend(c, q, m if i else None, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
    n = tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, c.kv, c.vv, m)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(c, q, m, stream=torch.cuda.current_stream(), ws=ws, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[1])


def test_refusals(ctxs):  # noqa: F811
    ctx, d = ctxs[64], 64
    c = Cache(ctx, d, 2, [3], [20], 16).fill()
    q = torch.zeros((3, 2, d), dtype=torch.float16, device="cuda")
    q8 = tq.alloc_view("q8_0", d, 2, 16, c.kv.num_pages)
    t3 = tq.alloc_view("turbo3_mse", d, 2, 16, c.kv.num_pages)
    n = tq.tq_chunk_workspace_for(ctx.h, c.batch, 2, c.kv, c.vv)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)

    def att(kv, vv, mods=None, batch=c.batch):
        return tq.tq_chunk_attention(ctx.h, batch, q, kv, vv, 0, 1.0, ws, n, out, mods=mods)
    assert att(c.kv, c.vv) == tq.TQ_OK
    for kv, vv in ((q8, c.vv), (c.kv, q8), (c.kv, t3)):
        assert att(kv, vv) == tq.TQ_ERR_UNSUPPORTED
        assert tq.tq_append_kv(ctx.h, c.batch, q, q, kv, vv, 0) == tq.TQ_ERR_UNSUPPORTED
    assert att(c.kv, c.vv, tq.ScoreMods(window=5, sinks=-1)) == tq.TQ_ERR_INVALID_ARG
    odd = tq.CacheView("f8_block", d, 2, 24, 2, 1, c.kv.payload, c.kv.header)
    assert att(odd, odd) == tq.TQ_ERR_INVALID_ARG
    x = torch.zeros((3, 2, d), dtype=torch.float16, device="cuda")
    assert tq.tq_encode_kv(ctx.h, c.kv, x, None, None, 0, 1, 3, 3 * 2 * d, 2 * d) == tq.TQ_ERR_UNSUPPORTED
    assert tq.tq_encode_kv(ctx.h, None, None, c.vv, x, 0, 1, 3, 3 * 2 * d, 2 * d) == tq.TQ_ERR_UNSUPPORTED
    assert tq.tq_encode_kv_layers(ctx.h, [q8, c.kv], [0, 0], None, None, 2, x, None, 1, 2 * d, 2 * d) == \
        tq.TQ_ERR_UNSUPPORTED
    dec = torch.empty((1, 1, 2, d), device="cuda")
    nb = tq.tq_decode_workspace_bytes(ctx.h, 1, 1, 2, 20)
    assert tq.tq_decode_attention(ctx.h, x[:1], 1, 1, 1, 2, c.kv, c.vv, 0, c.batch.seq_lens, 20, c.batch.block_table,
                                  c.table.shape[1], 1.0, 0.0, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb, dec) == \
        tq.TQ_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert status(ctx) == 0 and not q8.payload.any()


# ---------------------------------------------------------------------------
# windows with sinks, every format
# ---------------------------------------------------------------------------

SINKS = [dict(window=64, sinks=4), dict(window=1, sinks=1), dict(window=200, sinks=130), dict(window=37, sinks=17),
         dict(window=64, sinks=2 ** 31 - 1), dict(window=300, sinks=300), dict(window=2 ** 31 - 1, sinks=9)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([1, 1, 2], [700, 65, 3000]), ([200, 1], [200, 90]), ([40, 300], [2000, 1500])])
@pytest.mark.parametrize("kw", SINKS)
def test_sinks_over_f8(ctxs, d, new, lens, kw):  # noqa: F811
    c = Cache(ctxs[d], d, 1, new, lens, 48).fill()
    rows = np.unique(np.linspace(0, sum(new) - 1, 24).astype(int))
    check(c, 2, torch.float16, rows=rows, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vfmt", ["q8_0", "turbo2_mse", "turbo4_mse"])
@pytest.mark.parametrize("new,lens", [([1, 2], [700, 3000]), ([200, 40], [900, 2000])])
@pytest.mark.parametrize("page", [16, 24])
def test_sinks_over_the_other_formats(ctxs, d, vfmt, new, lens, page):  # noqa: F811
    """The bound of tests/test_gpu_step.py: six deviations of the operands' rounding over the keys that a row sees."""
    P = T.Paged(ctxs[d], d, 1, new, lens, page, vfmt)
    q = W.normal_tensor((P.n_tokens, 2, d), seed=3, device="cuda").half()
    for kw in (dict(window=64, sinks=4), dict(window=37, sinks=150), dict(window=300, sinks=17)):
        out = T.attend(P, q, mods=tq.ScoreMods(**kw))
        torch.cuda.synchronize()
        assert status(P.ctx) == 0
        for b in range(2):
            at = np.nonzero(P.seq == b)[0]
            at = at[np.unique(np.linspace(0, len(at) - 1, 8).astype(int))]
            k, v = P.stored(b)
            for i in at:  # a row at a time, over its keys alone
                j = S.seen(int(P.pos[i]), len(k), **kw)
                one = f64(q)[i:i + 1]
                want = S.chunk_attention(one, k[j], v[j], [len(j) - 1], 1 / math.sqrt(d))
                bound = T.row_bound(one, k[j], v[j], [len(j) - 1], want, torch.float16, 1 / math.sqrt(d))
                K.assert_rows(f64(out)[i:i + 1], want, np.maximum(bound, T.C.ATTN_RTOL) + T.half_step(out.dtype))


@pytest.mark.parametrize("vfmt", ["f8_block", "q8_0"])
@pytest.mark.parametrize("new", [4, 150])
def test_sinks_of_documents_and_prefixes(ctxs, vfmt, new):  # noqa: F811
    """Each document keeps its own first tokens; a prefix beyond a row's own position."""
    d, total = 64, 1500
    first = {4: np.array([0, 700, 1400, -50])}.get(new)
    pos = np.arange(total - new, total)
    if first is None:
        first = np.where(np.arange(new) < 60, 3, np.where(np.arange(new) < 100, 700, pos - pos % 11))
    kw = dict(window=20, sinks=6)
    if vfmt == "f8_block":
        c = Cache(ctxs[d], d, 1, [new], [total], 16).fill()
        check(c, 2, torch.float16, first=first, rows=np.arange(0, new, 7), **kw)
        check(c, 2, torch.float16, first=first, prefix=[total], rows=np.arange(0, new, 29), **kw)
        return
    P = T.Paged(ctxs[d], d, 1, [new], [total], 16)
    q = W.normal_tensor((new, 2, d), seed=3, device="cuda").half()
    m = T.mods_of(P, 2, 0.0, 20, False, first)
    out = T.attend(P, q, mods=tq.ScoreMods(window=20, first_keys=m.first_keys, sinks=6))
    torch.cuda.synchronize()
    k, v = P.stored(0)
    for i in range(0, new, 7 if new > 4 else 1):
        j = S.seen(int(P.pos[i]), total, first_key=int(first[i]), **kw)
        one = f64(q)[i:i + 1]
        want = S.chunk_attention(one, k[j], v[j], [len(j) - 1], 1 / math.sqrt(d))
        bound = T.row_bound(one, k[j], v[j], [len(j) - 1], want, torch.float16, 1 / math.sqrt(d))
        K.assert_rows(f64(out)[i:i + 1], want, np.maximum(bound, T.C.ATTN_RTOL) + T.half_step(out.dtype))


def test_sinks_without_a_window_change_nothing(ctxs):  # noqa: F811
    for new in (1, 100):
        c = Cache(ctxs[128], 128, 2, [new], [300], 16).fill()
        q = W.normal_tensor((new, 4, 128), seed=1, device="cuda").half()
        a, b = attend(c, q), attend(c, q, tq.ScoreMods(sinks=50))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_serving_loop(ctxs, d):  # noqa: F811
    """Prefill and decode of a ragged batch with normed, rotated queries and keys, a window and sinks: every step's rows
    against the oracle over what the cache holds, and the cache against the oracle's blocks."""
    ctx, H, G = ctxs[d], 2, 2
    table = tq.tq_rope_build(d, d // 2, "half", base=10000.0)
    f, m = S.rope_angles(d // 2, base=10000.0)
    w = 1 + 0.2 * W.normal_tensor((2, d), seed=1, device="cuda")
    c = Cache(ctx, d, H, [1, 1, 1], [150, 60, 90], 16)
    lens = np.zeros(3, np.int64)
    mods = dict(window=40, sinks=4)
    for step, new in enumerate([[100, 17, 33], [1, 1, 1], [20, 0, 1], [1, 1, 50], [1, 1, 1]]):
        lens = lens + new
        n = sum(new)
        qkv = W.normal_tensor((n, H * (G + 2), d), seed=50 + step, device="cuda").half()
        c.set_batch(new, lens)
        pos = torch.as_tensor(c.pos.astype(np.int32), device="cuda")
        q, k, v = qkv[:, :H * G], qkv[:, H * G:H * (G + 1)], qkv[:, H * (G + 1):]
        want_k = S.norm_rope(f64(k), f64(w[1]), c.pos, f, 1e-6, m)
        want_q = S.norm_rope(f64(q), f64(w[0]), c.pos, f, 1e-6, m)
        assert tq.tq_norm_rope(ctx.h, table, q, q, w[0], k, k, w[1], 1e-6, pos) == tq.TQ_OK  # in place
        torch.cuda.synchronize()
        for got, want in ((q, want_q), (k, want_k)):
            assert (np.abs(f64(got) - want) <= 4e-6 * np.abs(want).max() + rounding(torch.float16, want)).all()
        c.append(new, lens, k, v)
        c.check_blocks()
        check(c, G, torch.float16, q=q, **mods)


# ---------------------------------------------------------------------------
# chunks whose key tiles are staged once for all their entries
# ---------------------------------------------------------------------------

STAGED = [  # G, new, lens, page: eight entries (of 256 rows) and more for a sequence
    (4, [600], [600], 16),
    (8, [300], [4000], 64),
    (2, [1030, 1100], [1030, 2500], 48),
    (8, [260, 0, 600], [1000, 0, 601], 256),
    (7, [300], [32000], 16),
]


def staged_cache(ctx, d, G, new, lens, page, H=2, mods=None, **kw):
    """The cache, and that a call over it asks for the larger workspace."""
    c = Cache(ctx, d, H, new, lens, page, padding=2, **kw)
    least = tq.tq_chunk_workspace_bytes(ctx.h, c.batch, H * G, H)
    assert tq.tq_chunk_workspace_for(ctx.h, c.batch, H * G, c.kv, c.vv, mods) > least
    return c


def some(n):
    return np.unique(np.concatenate([np.linspace(0, n - 1, 14).astype(int), [63 % n, 64 % n, 127 % n, 128 % n]]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new,lens,page", STAGED)
def test_staged_shapes(ctxs, d, G, new, lens, page):  # noqa: F811
    """Both kernels, the one for the least workspace and the staged one, on the same call."""
    c = staged_cache(ctxs[d], d, G, new, lens, page).fill(outliers=0.01)
    for least in (False, True):
        check(c, G, torch.float16, rows=some(sum(new)), least=least)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mods", [dict(softcap=5.0), dict(bias=True), dict(prefix=[2550]), dict(window=300),
                                  dict(softcap=20.0, window=1000, bias=True, prefix=[1400]), dict(window=700, sinks=5),
                                  dict(window=300, sinks=900, bias=True), dict(window=1000, sinks=130)])
def test_staged_score_modifications(ctxs, d, mods):  # noqa: F811
    window = tq.ScoreMods(window=mods.get("window", 0))
    c = staged_cache(ctxs[d], d, 8, [1500], [2600], 16, H=1, mods=window).fill()
    check(c, 8, torch.bfloat16, torch.float32, rows=some(1500), **mods)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 128])
def test_staged_scales_marks_and_missing_pages(ctxs, d, dtype):  # noqa: F811
    """Scales that jump by up to 2^16 and blocks of zeros; a marked K and a marked V vector; pages out of range, those behind
    the window never looked at."""
    def jumps(i, kind):
        b = torch.div(i, 16, rounding_mode="floor")
        return 2.0 ** -((b * 7 % 13).float()) if kind == 0 else torch.where(b % 5 == 3, 0.0, 2.0 ** (b * 11 % 17 - 8).float())
    c = staged_cache(ctxs[d], d, 4, [520], [900], 16).fill(scale=jumps)
    check(c, 4, DT[dtype], torch.float32, rows=some(520))
    q = W.normal_tensor((522, 8, d), seed=3, device="cuda").to(DT[dtype])
    clean = attend(c, q)
    for view, key in ((c.kv, 500), (c.vv, 700)):
        vec = c.vectors(0, [key])[0, 1]
        view.header.view(torch.int32)[int(vec // 16)] |= 1 << int(vec % 16)
    got = attend(c, q)
    torch.cuda.synchronize()
    pos = torch.as_tensor(c.pos)
    assert torch.isnan(got[:520, 4:][pos >= 500]).all() and torch.equal(got[:520, :4], clean[:520, :4])
    assert torch.equal(got[:520][pos < 500], clean[:520][pos < 500]) and status(c.ctx) == 0
    n, total = 1500, 2600
    c = staged_cache(ctxs[d], d, 8, [n], [total], 16, H=1, mods=tq.ScoreMods(window=300)).fill()
    q = W.normal_tensor((n + 2, 8, d), seed=3, device="cuda").to(DT[dtype])
    k, v = c.stored(0)
    c.table = c.table.copy()
    c.table[0, [2, 100]] = [-1, 10 ** 6]
    c.set_batch([n], [total])
    for kw, lost in ((dict(), [2, 100]), (dict(window=300), [100]), (dict(window=300, sinks=20), [100]),
                     (dict(window=300, sinks=40), [2, 100])):
        out = attend(c, q, mods_of(c, 8, **kw))
        torch.cuda.synchronize()
        assert status(c.ctx) == 2
        missing = np.isin(np.arange(total) // 16, lost)
        at = some(n)
        want = S.chunk_attention(f64(q)[at], k, v, c.pos[at], 1 / math.sqrt(d), missing=missing, **kw)
        _, tol = expected(f64(q)[at], k, v, c.pos[at], 1 / math.sqrt(d), True, DT[dtype], **kw)
        assert (np.abs(f64(out)[at] - want) <= 2 * tol + rounding(out.dtype, want)).all(), kw


def test_staged_repeats_streams_graphs_and_layers(ctxs):  # noqa: F811
    d = 128
    c = staged_cache(ctxs[d], d, 4, [700, 500], [2000, 900], 32, H=2, n_layers=3, layer=2).fill()
    q = W.normal_tensor((c.n_tokens, 8, d), seed=1, device="cuda").half()
    m = mods_of(c, 8, window=1900, sinks=3)
    assert tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, c.kv, c.vv, m) > tq.tq_chunk_workspace_bytes(c.ctx.h, c.batch, 8, 2)
    want = [attend(c, q), attend(c, q, m)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attend(c, q, m if i else None, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
    n = tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, c.kv, c.vv)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(c, q, m, stream=torch.cuda.current_stream(), ws=ws, out=out)
        attend(c, q, None, stream=torch.cuda.current_stream(), ws=ws, out=out)  # the same workspace, one after the other
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:c.rows], want[0][:c.rows])
    # lengths that break the bounds: zeros in their rows.  (The others' work is cut elsewhere then, so that their sums differ
    # in the last bits: weights and values of order 1, a rounding of 2^-11 on each side and of the outputs.)
    c.batch = c.batch_of([700, 500], [2000, 300], 2, max_ctx=2000)
    out = attend(c, q, out=torch.full_like(q, 9.0))
    torch.cuda.synchronize()
    assert status(c.ctx) == 1 and not out[700:1200].any() and (out[1200:] == 9.0).all()
    assert (out[:700].float() - want[0][:700].float()).abs().max() < 2.0 ** -9


def test_staged_is_not_for_documents_or_too_large_batches(ctxs):  # noqa: F811
    c = staged_cache(ctxs[64], 64, 4, [600], [600], 16).fill()
    least = tq.tq_chunk_workspace_bytes(c.ctx.h, c.batch, 8, 2)
    first = np.concatenate([c.pos - c.pos % 200, [0, 0]])
    m = mods_of(c, 8, first=first)
    assert tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, c.kv, c.vv, m) == least
    check(c, 4, torch.float16, first=first, rows=some(600))
    assert tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, c.kv, c.vv, tq.ScoreMods(window=10)) == least
    huge = tq.Batch(c.batch.cu_tokens, c.batch.seq_lens, torch.zeros((1, 1 << 24), dtype=torch.int32, device="cuda"), 600, 600,
                    1 << 28)
    assert tq.tq_chunk_workspace_for(c.ctx.h, huge, 8, c.kv, c.vv) == tq.tq_chunk_workspace_bytes(c.ctx.h, huge, 8, 2)
    q8 = tq.alloc_view("q8_0", 64, 2, 16, 40)
    assert tq.tq_chunk_workspace_for(c.ctx.h, c.batch, 8, q8, q8) == least


def test_staging_stays_within_a_grid(ctxs):  # noqa: F811
    """65535 sequences of 64 tokens may be staged, one more is not (nothing runs: the sizes alone)."""
    view = tq.alloc_view("f8_block", 64, 1, 16, 1)
    tables = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (65537, 65536)]
    table = torch.zeros((65536, 8), dtype=torch.int32, device="cuda")
    for n, staged in ((65535, True), (65536, False)):
        b = tq.Batch(tables[0][:n + 1], tables[1][:n], table[:n], 64 * n, 64, 128)
        least = tq.tq_chunk_workspace_bytes(ctxs[64].h, b, 32, 1)
        assert (tq.tq_chunk_workspace_for(ctxs[64].h, b, 32, view, view) > least) == staged


# Batches of many entries of like lengths, which the plan does not cut between blocks; and of more entries than it looks at.
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,new,H,G", [(48, 64, 8, 4), (47, 63, 7, 4), (152, 40, 2, 8), (600, 5, 1, 4)])
def test_attend_many_like_entries(ctxs, d, n, new, H, G):  # noqa: F811
    c = Cache(ctxs[d], d, H, [new] * n, [new + 7 * (b % 60) for b in range(n)], 16, padding=2).fill()
    rows = some(n * new)
    check(c, G, torch.float16, rows=rows, least=True, window=100, sinks=5)
    # documents of 50 tokens, and one sequence in four that sees nothing
    first = np.concatenate([np.where(c.seq % 4 == 3, 1 << 20, c.pos - c.pos % 50), [0, 0]])
    out = check(c, G, torch.bfloat16, rows=rows, least=True, first=first)
    assert not out[:c.rows][torch.from_numpy(c.seq[:c.rows] % 4 == 3).cuda()].any()

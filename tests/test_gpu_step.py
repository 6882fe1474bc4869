"""GPU parity of the serving step (tq_rope, tq_append_kv, tq_read_kv, tq_chunk_attention) against the fp64 oracle.

Tolerances, fixed before the first run:
  * rotation: the angle is off by at most 2^-25 half turns (9.4e-8 rad), sincospi and the two products by a few 2^-24:
    |error| <= 6e-7 m (|x_p| + |x_q|) per pair, plus half a step of the output type;
  * q8_0 codes: equal wherever x / delta is further from a half-integer than the rotation's error can move it
    (127 * 2 * 6e-7 < 2e-4); elsewhere one apart; scales within one fp16 step; without a rotation the bytes are those of
    tq_encode_kv; turbo codes equal outside the 1e-6 band of a boundary, norms within one fp16 step;
  * attention: the framework's bound of 2e-3 per row, plus half a step of the output type, wherever the operands' own
    rounding does not pass it.  The products' operands are fp16: keys, values, weights, and queries that come in fp32
    are each off by up to 2^-11 relative, uniformly, 2^-11 / sqrt(3) rms.  A key's score is then off by e_j with rms
    2^-11 / sqrt(3) scale sqrt(sum_i (q_i k_ji)^2) (sqrt(2) times that for fp32 queries) where every e_j is independent,
    and to first order the row by sum_j w_j (e_j (v_j - o) + v_j (r_j + r'_j)) with r, r' of rms 2^-11 / sqrt(3): its
    variance is sum_j w_j^2 (var e_j |v_j - o|^2 + 2 (2^-22 / 3) |v_j|^2).  Few keys and coordinates can carry a row
    (channels 20 times larger than the rest), so six times that standard deviation is allowed: row_bound() below.
"""
import math

import numpy as np
import pytest
import torch

from kv_cache_quantization_turbo_gb300 import tq
from kv_cache_quantization_turbo_gb300 import workloads as W
from oracle import step_oracle as S
import gpu_common as C

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, want):
    """Half a step of the type around the wanted values.  Below the smallest normal number the step no longer shrinks
    with the value: it stays tiny * eps, so half of it is eps / 2 * tiny (fp16: 2^-25)."""
    return half_step(dtype) * np.maximum(np.abs(want), torch.finfo(dtype).tiny)


@pytest.fixture(scope="module")
def ctxs():
    C.require_cuda()
    c = {d: C.Ctx(d) for d in (64, 128, 256)}
    yield c
    for x in c.values():
        x.close()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def run_rope(ctx, d, rotary, layout, dtype, tokens, heads, positions, *, inverse=False, in_place=False, pad=0,
             scaling="none", seed=0):
    kw = dict(base=500000.0, factor=8.0, original_ctx=8192.0)
    table = tq.tq_rope_build(d, rotary, layout, scaling, **kw)
    buf = W.normal_tensor((tokens, heads + pad, d), seed=seed, device="cuda").to(dtype)
    x = buf[:, :heads]
    keep = buf.clone()
    out = x if in_place else torch.full((tokens, heads, d), float("nan"), dtype=dtype, device="cuda")
    pos = torch.as_tensor(np.asarray(positions, np.int32), device="cuda")
    assert tq.tq_rope(ctx.h, table, x, pos, out, inverse=inverse) == tq.TQ_OK
    torch.cuda.synchronize()
    f, m = S.rope_angles(rotary, scaling, **kw)
    x64 = f64(keep[:, :heads])
    want = S.rope(x64, positions, f, m, layout, inverse)
    got = f64(out)
    r2 = rotary // 2
    size = np.abs(x64[..., :rotary])
    pair = size[..., :r2] + size[..., r2:] if layout == "half" else size[..., 0::2] + size[..., 1::2]
    pair = np.concatenate([pair, pair], -1) if layout == "half" else np.repeat(pair, 2, -1)
    tol = 6e-7 * m * pair + rounding(dtype, want[..., :rotary])
    assert np.all(np.abs(got[..., :rotary] - want[..., :rotary]) <= tol)
    np.testing.assert_array_equal(got[..., rotary:], x64[..., rotary:])
    if in_place:
        assert torch.equal(buf[:, heads:], keep[:, heads:])
    else:
        assert torch.equal(buf, keep)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 128), (128, 64), (256, 40), (64, 20), (128, 126), (256, 2)])
def test_rope_layouts_types_and_parts(ctxs, dtype, layout, d, rotary):
    """Whole and partial rotations, pairs of every access width, one to several heads per thread."""
    pos = np.random.default_rng(rotary).integers(0, 200000, 37)
    run_rope(ctxs[d], d, rotary, layout, DT[dtype], 37, 5, pos, seed=rotary)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "wavelength", "yarn"])
def test_rope_scalings_and_far_positions(ctxs, scaling):
    """Positions up to the ends of int32, negative ones too: the angle does not lose bits."""
    run_rope(ctxs[128], 128, 128, "half", torch.float32, 8, 3,
             [0, 1, -1, 131071, 16777217, 2**31 - 1, -2**31, 123456789], scaling=scaling, seed=3)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 40), (700, 33), (5000, 7)])
def test_rope_sizes_strides_and_in_place(ctxs, tokens, heads):
    pos = np.arange(tokens) * 3
    run_rope(ctxs[64], 64, 64, "half", torch.bfloat16, tokens, heads, pos, pad=3, seed=4)
    run_rope(ctxs[64], 64, 32, "interleaved", torch.float16, tokens, heads, pos, pad=2, in_place=True, seed=5)


def test_rope_inverse_is_the_gradient(ctxs):
    """Against the formula, as the transpose (<R x, g> = <x, R^T g>), and against differences of the forward pass."""
    ctx, n, h, d = ctxs[128], 29, 4, 128
    run_rope(ctx, d, 96, "half", torch.float32, n, h, np.arange(n) * 1000, inverse=True, scaling="yarn", seed=6)
    table = tq.tq_rope_build(d, 96, "interleaved", "yarn", base=1e4, factor=4.0, original_ctx=2048.0)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 777
    x, g, v = (W.normal_tensor((n, h, d), seed=7 + i, device="cuda") for i in range(3))
    step = 2.0 ** -3  # linear in x: any step serves, a power of two adds no rounding of its own
    y, yv, gx = (torch.empty_like(x) for _ in range(3))
    for src, dst, inv in ((x, y, False), (x + step * v, yv, False), (g, gx, True)):
        assert tq.tq_rope(ctx.h, table, src, pos, dst, inverse=inv) == tq.TQ_OK
    torch.cuda.synchronize()
    # per sum of n h d terms: errors of 1e-6 relative to the terms, which have both signs
    size = float((y.double() * g.double()).abs().sum())
    assert abs(float((y.double() * g.double()).sum() - (x.double() * gx.double()).sum())) < 2e-6 * size
    num = float(((yv.double() - y.double()) / step * g.double()).sum())
    # a difference of values near |x| (errors 1e-6 each) over the step
    assert abs(num - float((v.double() * gx.double()).sum())) < (2e-6 + 4e-6 / step) * size


def test_rope_refusals(ctxs):
    ctx, t = ctxs[64], tq.tq_rope_build(64)
    x = torch.zeros((4, 2, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    call = tq._lib.tq_rope
    import ctypes
    ok = [ctx.h, ctypes.byref(t), x.data_ptr(), 0, 4, 2, 128, pos.data_ptr(), 0, x.data_ptr(), 128, None]

    def change(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return call(*a)
    assert change() == tq.TQ_OK
    assert change(a4=0) == tq.TQ_OK
    for kw in (dict(a2=x.data_ptr() + 4), dict(a2=None), dict(a3=3), dict(a4=-1), dict(a5=0), dict(a6=127),
               dict(a6=129), dict(a7=None), dict(a8=2), dict(a9=None), dict(a10=132), dict(a0=ctxs[128].h)):
        assert change(**kw) == tq.TQ_ERR_INVALID_ARG, kw
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        tq.tq_rope(ctx.h, t, x, pos.long(), x)
    with pytest.raises(ValueError):
        tq.tq_rope(ctx.h, t, x.transpose(0, 1), pos[:2], x.transpose(0, 1))


# ---------------------------------------------------------------------------
# batches over a paged cache
# ---------------------------------------------------------------------------

class Paged:
    """A paged q8_0 / V cache of a ragged batch in which everything that no token owns is NaN, and its batch."""

    def __init__(self, ctx, d, H, new, lens, page, vfmt="q8_0", *, seed=0, n_layers=1, layer=0, contiguous=False,
                 padding=0, fill=True, outliers=0.0):
        self.ctx, self.d, self.H, self.page, self.vfmt, self.layer = ctx, d, H, page, vfmt, layer
        self.new, self.lens = np.asarray(new, np.int64), np.asarray(lens, np.int64)
        B = len(self.new)
        if contiguous:
            self.table, n_pages = None, B + 1
        else:
            self.table, n_pages = W.shuffled_block_table(self.lens, page, seed=seed + 9, extra_pages=3)
        self.kv = tq.alloc_view("q8_0", d, H, page, n_pages, n_layers)
        self.vv = tq.alloc_view(vfmt, d, H, page, n_pages, n_layers)
        for view in (self.kv, self.vv):
            g = torch.Generator(device="cuda").manual_seed(seed)
            view.payload.copy_(torch.randint(0, 256, view.payload.shape, dtype=torch.uint8, device="cuda", generator=g))
            view.header.view(torch.int16).fill_(0x7E01)  # an fp16 NaN
        self.seq, self.pos = S.batch_positions(self.new, self.lens)
        self.rows = len(self.seq)
        self.n_tokens = self.rows + padding
        cu = np.concatenate([[0], np.cumsum(self.new)])
        self.set_batch(cu, self.lens)
        if fill:
            for b in range(B):
                T = int(self.lens[b])
                if T == 0:
                    continue
                k = W.kv_tensor(T, H, d, seed=seed + 100 + b, device="cuda", outlier_frac=outliers)
                v = W.kv_tensor(T, H, d, seed=seed + 200 + b, device="cuda", outlier_frac=outliers)
                slots = torch.as_tensor(self.slots(b, np.arange(T)), device="cuda")
                C.encode(ctx, self.kv, k, True, layer_begin=layer, slots=slots)
                C.encode(ctx, self.vv, v, False, layer_begin=layer, slots=slots)

    def set_batch(self, cu, lens, max_tokens=None, max_ctx=None, table="own"):
        dev = dict(dtype=torch.int32, device="cuda")
        t = self.table if isinstance(table, str) else table
        self.batch = tq.Batch(torch.as_tensor(np.asarray(cu, np.int32), device="cuda"),
                              torch.as_tensor(np.asarray(lens, np.int32), device="cuda"),
                              None if t is None else torch.as_tensor(t, **dev), self.n_tokens,
                              int(max(self.new, default=0)) if max_tokens is None else max_tokens,
                              int(max(self.lens, default=0)) if max_ctx is None else max_ctx)

    def slots(self, b, pos):
        pos = np.asarray(pos, np.int64)
        page = np.full_like(pos, b) if self.table is None else self.table[b, pos // self.page].astype(np.int64)
        return page * self.page + pos % self.page

    def stored(self, b, fmt=None, view=None):
        """Oracle values [T, H, d] of sequence b's stored tokens."""
        out = []
        for view, fmt in ((self.kv, "q8_0"), (self.vv, self.vfmt)):
            p, h = C.read_vectors(view, self.layer)
            s = self.slots(b, np.arange(self.lens[b]))
            p, h = C.slot_major(p, s, self.page), C.slot_major(h, s, self.page)
            out.append(C.oracle_dequant(fmt, C.gpu_codes(fmt, self.d, p, h), self.ctx.signs, self.ctx.S))
        return out


    def stored_all(self):
        """Oracle values of every slot (one KV head): [slots, 1, d]."""
        out = []
        for view, fmt in ((self.kv, "q8_0"), (self.vv, self.vfmt)):
            p, h = C.read_vectors(view, self.layer)
            s = np.arange(view.num_pages * self.page)
            out.append(C.oracle_dequant(fmt, C.gpu_codes(fmt, self.d, C.slot_major(p, s, self.page),
                                                         C.slot_major(h, s, self.page)), self.ctx.signs, self.ctx.S))
        return out


def status(ctx):
    return tq.tq_get_status(ctx.h)[1]


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

def check_append(P, dtype, *, rope=None, positions=None, seed=1, oracle_kw=None, qkv=True):
    """Appends random rows; compares every stored vector, and that nothing else changed."""
    d, H, n = P.d, P.H, P.n_tokens
    buf = W.normal_tensor((n, 3 * H if qkv else H, d), seed=seed, device="cuda").to(dtype)
    k = buf[:, H:2 * H] if qkv else buf
    v = buf[:, 2 * H:] if qkv else buf.flip(0).contiguous()
    before = [(x.payload.clone(), x.header.clone()) for x in (P.kv, P.vv)]
    pos_t = None if positions is None else torch.as_tensor(np.asarray(positions, np.int32), device="cuda")
    assert tq.tq_append_kv(P.ctx.h, P.batch, k, v, P.kv, P.vv, P.layer, rope=rope, positions=pos_t) == tq.TQ_OK
    torch.cuda.synchronize()
    assert status(P.ctx) == 0
    slots = np.concatenate([P.slots(b, P.pos[P.seq == b]) for b in range(len(P.new))]).astype(np.int64)
    k64, v64 = f64(k)[:P.rows], f64(v)[:P.rows]
    if rope is not None:
        f, m = S.rope_angles(rope.rotary_dim, **(oracle_kw or {}))
        p = P.pos if positions is None else np.asarray(positions)[:P.rows]
        k64 = S.rope(k64, p, f, m, "half" if rope.layout == 0 else "interleaved")
    for x64, view, fmt, rotated in ((k64, P.kv, "q8_0", rope is not None), (v64, P.vv, P.vfmt, False)):
        pay, hdr = C.read_vectors(view, P.layer)
        pay, hdr = C.slot_major(pay, slots, P.page), C.slot_major(hdr, slots, P.page)
        if fmt == "q8_0":
            codes = pay.view(np.int8).astype(np.int64).reshape(P.rows, H, -1, 32)
            blocks = x64.reshape(P.rows, H, -1, 32)
            delta = np.abs(blocks).max(-1, keepdims=True) / 127
            t = np.divide(blocks, delta, out=np.zeros_like(blocks), where=delta > 0)
            want = (np.sign(t) * np.floor(np.abs(t) + 0.5)).astype(np.int64)
            near = np.abs(np.abs(t) % 1 - 0.5) < 2e-4
            assert np.all((codes == want) | near) and np.abs(codes - want).max(initial=0) <= 1
            from _layout import f16_ulp_diff
            assert f16_ulp_diff(hdr.view(np.float16).reshape(P.rows, H, -1), delta[..., 0].astype(np.float16)).max() <= 1
        else:
            enc = S.turbo_mse_encode(x64, fmt, P.ctx.signs)
            C.check_turbo_codes(fmt, d, pay, hdr, enc, band_limit=False)
    # every byte that no new token owns is as it was
    for (pay0, hdr0), view in zip(before, (P.kv, P.vv)):
        shape = (view.n_layers, view.num_pages, view.n_kv_heads, view.page_size, -1)
        for old, new in ((pay0, view.payload), (hdr0, view.header)):
            o, w = (x.view(shape).cpu().numpy().copy() for x in (old, new))
            o[P.layer, slots // P.page, :, slots % P.page] = 0
            w[P.layer, slots // P.page, :, slots % P.page] = 0
            np.testing.assert_array_equal(o, w)
    return slots


ROPE_KW = dict(scaling="yarn", base=10000.0, factor=4.0, original_ctx=4096.0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vfmt", ["q8_0", "turbo2_mse", "turbo3_mse", "turbo4_mse"])
def test_append_formats_types_and_dims(ctxs, dtype, d, vfmt):
    """A ragged batch (an empty sequence, single tokens, chunks across pages) into layer 1 of 2, padding rows behind."""
    P = Paged(ctxs[d], d, 3, [5, 0, 1, 40, 17], [5, 9, 64, 300, 33], 16, vfmt, n_layers=2, layer=1, padding=4,
              fill=False)
    rope = tq.tq_rope_build(d, d, "half", **ROPE_KW)
    check_append(P, DT[dtype], rope=rope, oracle_kw=ROPE_KW)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [2, 20, 32, 64, 126])
@pytest.mark.parametrize("page", [1, 24])
def test_append_rotations_and_pages(ctxs, layout, rotary, page):
    P = Paged(ctxs[128], 128, 2, [3, 30, 1], [100, 31, 1], page, fill=False)
    rope = tq.tq_rope_build(128, rotary, layout, **ROPE_KW)
    pos = np.random.default_rng(rotary).integers(-5, 1000000, P.n_tokens)
    check_append(P, torch.float16, rope=rope, positions=pos, oracle_kw=ROPE_KW)
    check_append(P, torch.float32, rope=rope, oracle_kw=ROPE_KW, seed=8, qkv=False)


@pytest.mark.parametrize("H,new", [(1, [1]), (11, [600]), (16, [2048, 1]), (5, [1] * 70)])
def test_append_sizes(ctxs, H, new):
    P = Paged(ctxs[64], 64, H, new, [n + 7 * i for i, n in enumerate(new)], 32, "turbo3_mse", fill=False)
    check_append(P, torch.float16, rope=tq.tq_rope_build(64, **ROPE_KW), oracle_kw=ROPE_KW)


def test_append_without_rotation_gives_the_encoder_bytes(ctxs):
    for d in (64, 128, 256):
        P = Paged(ctxs[d], d, 4, [50, 3], [50, 70], 128, fill=False, contiguous=True)
        slots = check_append(P, torch.float16, qkv=False, seed=21)
        x = W.normal_tensor((P.n_tokens, 4, d), seed=21, device="cuda").half()
        ref = tq.alloc_view("q8_0", d, 4, P.page, P.kv.num_pages)
        C.encode(ctxs[d], ref, x, True, slots=torch.as_tensor(slots, device="cuda"))
        torch.cuda.synchronize()
        for a, b in zip(C.read_vectors(ref), C.read_vectors(P.kv)):
            np.testing.assert_array_equal(C.slot_major(a, slots, P.page), C.slot_major(b, slots, P.page))


def test_append_zero_vectors_and_empty_batches(ctxs):
    P = Paged(ctxs[64], 64, 2, [3], [3], 4, "turbo2_mse", fill=False)
    z = torch.zeros((3, 2, 64), device="cuda")
    assert tq.tq_append_kv(P.ctx.h, P.batch, z, z, P.kv, P.vv, 0) == tq.TQ_OK
    out = torch.full((2, 3, 2, 64), 7.0, device="cuda")
    assert tq.tq_read_kv(P.ctx.h, P.batch, P.kv, out[0], P.vv, out[1], 0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert not out.any()
    none = tq.Batch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                    None, 3, 0, 0)
    before = P.kv.payload.clone()
    assert tq.tq_append_kv(P.ctx.h, none, z + 1, z, P.kv, P.vv, 0) == tq.TQ_OK  # no sequence: every row is padding
    assert tq.tq_read_kv(P.ctx.h, none, P.kv, out[0], None, None, 0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert torch.equal(before, P.kv.payload) and not out.any()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vfmt", ["q8_0", "turbo2_mse", "turbo3_mse", "turbo4_mse"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_returns_the_stored_values(ctxs, d, vfmt, dtype):
    """fp32 arithmetic on the stored values (1e-6 relative to the vector), then half a step of the type; padding rows
    stay."""
    P = Paged(ctxs[d], d, 3, [30, 0, 1, 9], [64, 5, 1, 40], 16, vfmt, padding=3)
    k = torch.full((P.n_tokens, 3, d), 5.0, dtype=DT[dtype], device="cuda")
    v = k.clone()
    assert tq.tq_read_kv(P.ctx.h, P.batch, P.kv, k, P.vv, v, 0) == tq.TQ_OK
    torch.cuda.synchronize()
    for got, i in ((f64(k), 0), (f64(v), 1)):
        want = np.concatenate([P.stored(b)[i][P.lens[b] - P.new[b]:] for b in range(4)])
        tol = rounding(DT[dtype], want) + 1e-6 * np.linalg.norm(want, axis=-1, keepdims=True)
        assert np.all(np.abs(got[:P.rows] - want) <= tol)
        assert np.all(got[P.rows:] == 5.0)
    k2 = torch.zeros_like(k)
    assert tq.tq_read_kv(P.ctx.h, P.batch, P.kv, k2, None, None, 0) == tq.TQ_OK
    v2 = torch.zeros_like(v)
    assert tq.tq_read_kv(P.ctx.h, P.batch, None, None, P.vv, v2, 0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert torch.equal(k2[:P.rows], k[:P.rows]) and torch.equal(v2[:P.rows], v[:P.rows])


def test_append_and_read_skip_what_is_out_of_range(ctxs):
    """Bad pages and sequences that break the call's bounds: flagged, nothing written, zeros read."""
    ctx = ctxs[64]
    P = Paged(ctx, 64, 2, [4, 4, 4], [20, 20, 20], 8, fill=False)
    P.table = P.table.copy()
    P.table[1, 2] = 10**6  # the page of sequence 1's positions 16 ..
    P.set_batch([0, 4, 8, 12], [20, 20, 20])
    x = W.normal_tensor((12, 2, 64), seed=1, device="cuda")
    before = P.kv.payload.clone()
    assert tq.tq_append_kv(ctx.h, P.batch, x, x, P.kv, P.vv, 0) == tq.TQ_OK
    assert status(ctx) == 2
    out = torch.full_like(x, 3.0)
    assert tq.tq_read_kv(ctx.h, P.batch, P.kv, out, None, None, 0) == tq.TQ_OK
    assert status(ctx) == 2
    assert not out[4:8].any() and out[:4].any() and out[8:].any()
    changed = int((P.kv.payload.view(-1, 64) != before.view(-1, 64)).any(-1).sum())
    assert changed == 2 * 8
    for cu, lens, kw in (([0, 4, 8, 12], [20, 3, 20], {}), ([0, 4, 8, 12], [20, 21, 20], {}),
                         ([0, 4, 8, 13], [20, 20, 20], {}), ([0, 4, 8, 12], [20, 20, -1], {}),
                         ([0, 4, 8, 12], [20] * 3, dict(max_tokens=3))):
        P.set_batch(cu, lens, table=W.shuffled_block_table(P.lens, 8, seed=9, extra_pages=3)[0], **kw)
        assert tq.tq_append_kv(ctx.h, P.batch, x, x, P.kv, P.vv, 0) == tq.TQ_OK
        assert status(ctx) == 1, (cu, lens)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def row_bound(q, k, v, positions, want, dtype, scale, softcap=0.0, window=0, slopes=None, first_keys=None, prefix=0):
    """Six standard deviations of the first-order effect of the operands' rounding, relative to each row [n, Hq]."""
    n, Hq, d = q.shape
    T, H, _ = k.shape
    u = 2.0 ** -22 / 3
    out = np.zeros((n, Hq))
    for i in range(n):
        lo, hi = S.visible(int(positions[i]), T, window, 0 if first_keys is None else int(first_keys[i]), prefix)
        if hi <= lo:
            continue
        j = np.arange(lo, hi)
        for h in range(Hq):
            kk, vv = k[j, h * H // Hq], v[j, h * H // Hq]
            s = kk @ q[i, h] * scale
            var = u * (2 if dtype == torch.float32 else 1) * scale ** 2 * ((kk * q[i, h]) ** 2).sum(-1)
            if softcap:
                s = softcap * np.tanh(s / softcap)  # its slope is at most 1
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(int(positions[i]) - j)
            w = np.exp(s - s.max())
            w /= w.sum()
            o = want[i, h]
            t = (w ** 2 * (var * ((vv - o) ** 2).sum(-1) + 2 * u * (vv ** 2).sum(-1))).sum()
            out[i, h] = 6 * math.sqrt(t) / max(np.linalg.norm(o), 1e-30)
    return out


def attend(P, q, out_dtype=None, mods=None, workspace=None, scale=None, stream=None, out=None):
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, q.shape[1], P.H)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    if out is None:
        out = torch.full(q.shape, 9.0, dtype=out_dtype or q.dtype, device="cuda")
    st = tq.tq_chunk_attention(P.ctx.h, P.batch, q, P.kv, P.vv, P.layer, scale or 1 / math.sqrt(P.d), ws, n, out,
                               mods=mods, stream=stream)
    assert st == tq.TQ_OK, tq.tq_status_string(st)
    return out


def mods_of(P, Hq, softcap=0.0, window=0, bias=False, first=None, prefix=None):
    dev = dict(device="cuda")
    return tq.ScoreMods(softcap, window,
                        2.0 ** (-8.0 * torch.arange(1, Hq + 1, **dev).float() / Hq) if bias else None,
                        None if first is None else torch.as_tensor(np.asarray(first, np.int32), **dev),
                        None if prefix is None else torch.as_tensor(np.asarray(prefix, np.int32), **dev))


def check_attend(P, G, dtype, out_dtype=None, *, seed=3, softcap=0.0, window=0, bias=False, first=None, prefix=None,
                 rows=None, scale=None):
    Hq = P.H * G
    q = W.normal_tensor((P.n_tokens, Hq + 2, P.d), seed=seed, device="cuda").to(dtype)[:, 1:1 + Hq]
    m = mods_of(P, Hq, softcap, window, bias, first, prefix)
    out = attend(P, q, out_dtype, m, scale=scale)
    torch.cuda.synchronize()
    assert status(P.ctx) == 0
    got, q64 = f64(out), f64(q)
    assert np.all(got[P.rows:] == 9.0)
    slopes = None if m.slopes is None else f64(m.slopes)
    worst = -1.0
    for b in range(len(P.new)):
        at = np.nonzero(P.seq == b)[0]
        if rows is not None:
            at = at[np.isin(at, rows)]
        if not len(at):
            continue
        k, v = P.stored(b)
        want = S.chunk_attention(q64[at], k, v, P.pos[at], scale or 1 / math.sqrt(P.d), softcap=softcap, window=window,
                                 slopes=slopes, first_keys=None if first is None else np.asarray(first)[at],
                                 prefix=0 if prefix is None else int(prefix[b]))
        empty = ~want.any(-1)
        assert not got[at][empty].any()
        bound = row_bound(q64[at], k, v, P.pos[at], want, dtype, scale or 1 / math.sqrt(P.d), softcap, window, slopes,
                          None if first is None else np.asarray(first)[at], 0 if prefix is None else int(prefix[b]))
        err = C.rel_err_per_head(got[at], want) - np.maximum(bound, C.ATTN_RTOL) - half_step(out.dtype)
        worst = max(worst, err[~empty].max(initial=-1.0))
    assert worst < 0, worst
    return out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vfmt", ["q8_0", "turbo2_mse", "turbo3_mse", "turbo4_mse"])
def test_attend_formats_and_dims(ctxs, d, vfmt):
    """Chunks that span row tiles and key tiles with ragged ends, a decode row, an empty sequence, padding rows."""
    P = Paged(ctxs[d], d, 2, [140, 1, 0, 33], [170, 300, 4, 33], 16, vfmt, padding=5)
    check_attend(P, 2, torch.float16)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out_dtype", list(DT))
def test_attend_types(ctxs, dtype, out_dtype):
    P = Paged(ctxs[128], 128, 1, [20, 1], [200, 129], 24, outliers=0.01)
    check_attend(P, 4, DT[dtype], DT[out_dtype])


@pytest.mark.parametrize("d,H,G,new,lens,page", [
    (128, 1, 1, [1], [1], 1),
    (128, 2, 4, [1], [5000], 16),
    (64, 3, 7, [2, 1, 3], [129, 128, 127], 1),
    (256, 1, 16, [9], [1000], 64),
    (128, 1, 8, [257], [257], 256),
    (64, 1, 1, [300, 255, 256], [600, 255, 700], 24),
    (256, 2, 2, [65, 130], [400, 130], 100),
    (128, 1, 130, [3], [70], 16),
    (128, 4, 2, [1] * 40, list(range(1, 3201, 80)), 16),
])
def test_attend_shapes(ctxs, d, H, G, new, lens, page):
    """Lengths of one, key counts at and around tile borders, group sizes up to more than a row tile."""
    check_attend(Paged(ctxs[d], d, H, new, lens, page, "turbo4_mse" if d == 64 else "q8_0"), G, torch.float16)


def test_attend_contiguous_cache_and_layers(ctxs):
    P = Paged(ctxs[128], 128, 2, [3, 70], [50, 90], 100, n_layers=3, layer=2, contiguous=True)
    check_attend(P, 2, torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mods", [dict(softcap=5.0), dict(window=1), dict(window=50), dict(bias=True),
                                  dict(prefix=[40, 500, 0, 33]), dict(softcap=20.0, window=140, bias=True)])
def test_attend_score_modifications(ctxs, d, mods):
    P = Paged(ctxs[d], d, 2, [150, 1, 0, 33], [310, 290, 4, 33], 16)
    check_attend(P, 2, torch.float16, **mods)


@pytest.mark.parametrize("d", [64, 256])
def test_attend_documents_and_empty_rows(ctxs, d):
    """Packed documents, rows that see nothing (a first key behind their position or past the end), also whole tiles."""
    P = Paged(ctxs[d], d, 1, [300, 20], [350, 400], 16, "turbo3_mse")
    first = P.pos // 37 * 37
    first[5::11] = P.pos[5::11] + 1
    first[128:260] = 10**9
    check_attend(P, 2, torch.float16, first=first, bias=True)
    check_attend(P, 2, torch.float16, first=first, window=30, prefix=[350, 350], softcap=10.0)


def test_attend_masked_values_do_not_leak(ctxs):
    """Infinite and NaN scales of stored keys and values: rows that see them are NaN, all others as without them."""
    d = 128
    for which in ("k", "v"):
        for vfmt in ("q8_0", "turbo4_mse"):
            P = Paged(ctxs[d], d, 1, [200], [260], 16, vfmt)
            q = W.normal_tensor((200, 2, d), seed=4, device="cuda").half()
            first = np.where(np.arange(200) < 120, 0, 131)  # the second part's documents begin behind key 130
            m = mods_of(P, 2, first=first)
            clean = attend(P, q, mods=m)
            view = P.kv if which == "k" else P.vv
            s = int(P.slots(0, [130])[0])
            per = view.header.numel() // (view.num_pages * P.page)
            h = view.header.view(torch.float16).view(-1, per // 2)
            h[s, -1] = float("inf") if which == "v" else float("nan")
            got = attend(P, q, mods=m)
            torch.cuda.synchronize()
            sees = (first <= 130) & (P.pos >= 130)
            assert sees.any() and torch.isnan(got[torch.as_tensor(sees)]).all()
            keep = torch.as_tensor(~sees)
            assert torch.equal(got[keep], clean[keep])


def test_attend_query_range_and_isolation(ctxs):
    """bf16 queries far outside fp16's range (a tiny scale brings the scores back); a NaN query row stays alone."""
    P = Paged(ctxs[64], 64, 2, [40], [90], 16)
    q = W.normal_tensor((40, 4, 64), seed=5, device="cuda").to(torch.bfloat16)
    a = attend(P, q)
    big = attend(P, q * 2.0 ** 40, scale=2.0 ** -40 / 8)
    small = attend(P, q * 2.0 ** -60, scale=2.0 ** 60 / 8)
    torch.cuda.synchronize()
    assert torch.equal(a, big) and torch.equal(a, small)
    q2 = q.clone()
    q2[7, 1] = float("nan")
    b = attend(P, q2)
    torch.cuda.synchronize()
    assert torch.isnan(b[7, 1]).all()
    b[7, 1] = a[7, 1]
    assert torch.equal(a, b)


def test_attend_large_key_magnitudes_stay_finite(ctxs):
    """Stored values at the top of fp16: read within the documented 511.5 * 127."""
    P = Paged(ctxs[64], 64, 1, [4], [40], 16, fill=False)
    x = W.normal_tensor((40, 1, 64), seed=6, device="cuda").clamp(-1, 1).half() * 65504.0
    slots = torch.as_tensor(P.slots(0, np.arange(40)), device="cuda")
    C.encode(P.ctx, P.kv, x * 2.0 ** -14, True, slots=slots)
    C.encode(P.ctx, P.vv, x, False, slots=slots)
    q = W.normal_tensor((4, 1, 64), seed=7, device="cuda").half()
    got = f64(attend(P, q, torch.float32))
    k, v = P.stored(0)
    want = S.chunk_attention(f64(q), k, v, P.pos, 1 / 8)
    # scales are read up to 0.9 % smaller (516 as 511.5), on top of the usual bound
    assert C.rel_err_per_head(got, want).max() < 0.009 + C.ATTN_RTOL


def test_attend_out_of_range(ctxs):
    """Bad pages are left out, sequences that break the bounds give zeros; both are flagged."""
    ctx = ctxs[128]
    P = Paged(ctx, 128, 1, [20, 4], [60, 40], 16)
    q = W.normal_tensor((24, 2, 128), seed=8, device="cuda").half()
    good = P.table
    P.table = good.copy()
    P.table[0, 1] = -7
    P.set_batch([0, 20, 24], [60, 40])
    out = attend(P, q)
    torch.cuda.synchronize()
    assert status(ctx) == 2
    P.table = good
    k, v = P.stored(0)
    missing = (np.arange(60) // 16) == 1
    want = S.chunk_attention(f64(q)[:20], k, v, P.pos[:20], 1 / math.sqrt(128), missing=missing)
    assert C.rel_err_per_head(f64(out)[:20], want).max() < C.ATTN_RTOL + half_step(out.dtype)
    for cu, lens, kw in (([0, 20, 24], [60, 3], {}), ([0, 20, 24], [60, 61], {}), ([0, 20, 25], [60, 40], {}),
                         ([0, 20, 24], [60, -5], {}), ([0, 4, 24], [60, 40], dict(max_tokens=19))):
        P.set_batch(cu, lens, **kw)
        out = attend(P, q)
        torch.cuda.synchronize()
        assert status(ctx) == 1, (cu, lens)
        assert out[:cu[1]].any() and not out[cu[1]:24].any(), (cu, lens)


def test_attend_is_deterministic_and_ignores_old_workspaces(ctxs):
    P = Paged(ctxs[128], 128, 2, [100, 1, 1], [3000, 2000, 700], 16)
    q = W.normal_tensor((102, 8, 128), seed=9, device="cuda").half()
    a = attend(P, q)
    ws = torch.full((tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 8, 2),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b = attend(P, q, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_attend_full_width_sampled_rows(ctxs):
    """A 2048-token chunk at the end of 6000 tokens, 8 query heads of 2 KV heads: sampled rows around tile borders."""
    P = Paged(ctxs[128], 128, 2, [2048], [6000], 64, outliers=0.01)
    rows = [0, 1, 31, 32, 63, 64, 127, 128, 500, 1023, 1024, 2016, 2046, 2047]
    check_attend(P, 4, torch.bfloat16, rows=rows)


def test_attend_more_sequences_than_the_plan_keeps_near(ctxs):
    """1500 sequences of one or two tokens (their entry counts go through the workspace), some without any."""
    new = [1 + (i % 7 == 0) - (i % 11 == 5) for i in range(1500)]
    lens = [max(n, 1 + (i * 37) % 50) for i, n in enumerate(new)]
    P = Paged(ctxs[64], 64, 1, new, lens, 16, fill=False)
    x = W.normal_tensor((int(sum(lens)), 1, 64), seed=3, device="cuda").half()
    slots = torch.as_tensor(np.concatenate([P.slots(b, np.arange(n)) for b, n in enumerate(lens)]), device="cuda")
    C.encode(P.ctx, P.kv, x, True, slots=slots)
    C.encode(P.ctx, P.vv, x.flip(0).contiguous(), False, slots=slots)
    q = W.normal_tensor((P.n_tokens, 2, 64), seed=4, device="cuda").half()
    got = f64(attend(P, q))
    q64, keys, worst = f64(q), P.stored_all(), 0.0
    for b in list(range(0, 60)) + [1022, 1023, 1024, 1025, 1498, 1499]:
        at = np.nonzero(P.seq == b)[0]
        if len(at):
            k, v = (y[P.slots(b, np.arange(lens[b]))] for y in keys)
            want = S.chunk_attention(q64[at], k, v, P.pos[at], 1 / 8)
            worst = max(worst, C.rel_err_per_head(got[at], want).max())
    assert worst < C.ATTN_RTOL + half_step(torch.float16)
    assert np.isfinite(got).all() and (got != 9.0).any(-1).all()


def test_pages_beyond_32_bit_offsets(ctxs):
    """A cache of more than 4 GiB per view: append, read and attention through pages at its end."""
    d, H, page = 128, 8, 16
    n_pages = (1 << 32) // (page * H * d) + 400
    kv, vv = (tq.alloc_view("q8_0", d, H, page, n_pages) for _ in range(2))
    assert kv.payload.numel() > 1 << 32
    T = 100
    table = (n_pages - 1 - 3 * torch.arange(7, device="cuda")).to(torch.int32).view(1, 7)
    dev = dict(dtype=torch.int32, device="cuda")
    batch = tq.Batch(torch.tensor([0, T], **dev), torch.tensor([T], **dev), table, T, T, T)
    k, v, q = (W.normal_tensor((T, H, d), seed=i, device="cuda").half() for i in range(3))
    ctx = ctxs[128]
    assert tq.tq_append_kv(ctx.h, batch, k, v, kv, vv, 0) == tq.TQ_OK
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    assert tq.tq_read_kv(ctx.h, batch, kv, rk, vv, rv, 0) == tq.TQ_OK
    out = torch.empty_like(q)
    n = tq.tq_chunk_workspace_bytes(ctx.h, batch, H, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert tq.tq_chunk_attention(ctx.h, batch, q, kv, vv, 0, 1 / math.sqrt(d), ws, n, out) == tq.TQ_OK
    torch.cuda.synchronize()
    assert status(ctx) == 0
    want_k = S.q8_0_values(f64(k))
    # scales rounded once to fp16 on both sides, values to fp16; ties of codes are the encoder's own (fp32 quotients)
    assert np.abs(f64(rk) - want_k).max() < 1.5 * np.abs(f64(k)).max() / 127
    want = S.chunk_attention(f64(q), f64(rk), f64(rv), np.arange(T), 1 / math.sqrt(d))
    # the values read back are rounded to fp16 once more: 2^-11 each on K and V
    assert C.rel_err_per_head(f64(out), want).max() < C.ATTN_RTOL + 3 * half_step(torch.float16)
    del kv, vv
    torch.cuda.empty_cache()


def test_attend_refusals(ctxs):
    P = Paged(ctxs[128], 128, 2, [3], [10], 16)
    q = torch.zeros((3, 4, 128), dtype=torch.float16, device="cuda")
    out = torch.zeros_like(q)
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 4, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(q=q, out=out, kv=P.kv, vv=P.vv, layer=0, scale=0.1, ws=ws, n=n, mods=None, batch=P.batch, ctx=P.ctx):
        return tq.tq_chunk_attention(ctx.h, batch, q, kv, vv, layer, scale, ws, n, out, mods=mods)
    assert call() == tq.TQ_OK
    bad = tq.TQ_ERR_INVALID_ARG
    assert call(n=n - 1) == tq.TQ_ERR_WORKSPACE and call(ws=None) == tq.TQ_ERR_WORKSPACE
    assert call(ws=ws.data_ptr() + 16) == tq.TQ_ERR_WORKSPACE
    assert call(layer=1) == bad and call(layer=-1) == bad and call(scale=math.nan) == bad
    assert call(q=q.double(), out=out) == bad
    assert call(out=out.double()) == bad
    assert call(mods=tq.ScoreMods(softcap=-1.0)) == bad and call(mods=tq.ScoreMods(softcap=math.inf)) == bad
    assert call(mods=tq.ScoreMods(window=-1)) == bad
    assert call(kv=P.vv, vv=tq.alloc_view("q8_0", 128, 2, 8, 4)) == bad
    for kf, vf in (("turbo4", "q8_0"), ("q8_0", "turbo4")):
        assert call(kv=tq.alloc_view(kf, 128, 2, 16, P.kv.num_pages),
                    vv=tq.alloc_view(vf, 128, 2, 16, P.kv.num_pages)) == tq.TQ_ERR_UNSUPPORTED
    m = tq.alloc_view("minmax", 128, 2, 16, P.kv.num_pages, bits=4)
    assert call(vv=m) == tq.TQ_ERR_UNSUPPORTED
    q3 = torch.zeros((3, 3, 128), dtype=torch.float16, device="cuda")
    assert call(q=q3, out=torch.zeros_like(q3)) == tq.TQ_ERR_UNSUPPORTED
    assert tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 3, 2) == 0
    b = P.batch
    assert call(batch=tq.Batch(b.cu_tokens, b.seq_lens, b.block_table, 3, 3, 17)) == bad  # pages hold 16
    assert call(batch=tq.Batch(b.cu_tokens, b.seq_lens, None, 3, 3, 17)) == bad
    assert call(batch=tq.Batch(b.cu_tokens, b.seq_lens, b.block_table, 3, -1, 10)) == bad
    for kw in (dict(first_keys=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(slopes=torch.zeros(2, device="cuda")),
               dict(prefix_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(mods=tq.ScoreMods(**kw))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# the three together, as a serving loop uses them
# ---------------------------------------------------------------------------

def test_steps_together_on_a_stream_and_in_a_graph(ctxs):
    """Two sequences: a prefill chunk each, then decode steps replayed from one captured graph whose lengths move on
    the device.  Every step's attention is compared with the oracle over all keys appended so far (as they read back)
    with the oracle's rotation of the queries; the context's second graph on the same workspace runs in turn."""
    ctx, d, H, G, page = ctxs[128], 128, 2, 2, 16
    Hq, cap = H * G, 64
    table, n_pages = W.shuffled_block_table(np.array([cap, cap]), page, seed=5)
    kv, vv = (tq.alloc_view("q8_0", d, H, page, n_pages) for _ in range(2))
    kw = dict(scaling="wavelength", base=10000.0, factor=8.0, original_ctx=64.0)
    rope = tq.tq_rope_build(d, 64, "half", **kw)
    f, m = S.rope_angles(64, **kw)
    dev = dict(dtype=torch.int32, device="cuda")
    bt = torch.as_tensor(table, **dev)
    ws_n = max(tq.tq_chunk_workspace_bytes(ctx.h, tq.Batch(torch.zeros(3, **dev), torch.zeros(2, **dev), bt, n, mt, cap),
                                           Hq, H) for n, mt in ((29, 20), (2, 1)))
    ws = torch.empty(ws_n, dtype=torch.uint8, device="cuda")

    def step(batch, qkv, pos, qr, out, stream):
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        assert tq.tq_rope(ctx.h, rope, q, pos, qr, stream=stream) == tq.TQ_OK
        assert tq.tq_append_kv(ctx.h, batch, k, v, kv, vv, 0, rope=rope, stream=stream) == tq.TQ_OK
        assert tq.tq_chunk_attention(ctx.h, batch, qr, kv, vv, 0, 1 / math.sqrt(d), ws, ws_n, out,
                                     stream=stream) == tq.TQ_OK

    def check(lens, new, qkv, out):
        seq, pos = S.batch_positions(new, lens)
        q = S.rope(f64(qkv)[:, :Hq], pos, f, m)
        whole = tq.Batch(torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda"),
                         torch.as_tensor(np.asarray(lens, np.int32), device="cuda"), bt, int(sum(lens)), cap, cap)
        k, v = (torch.empty((int(sum(lens)), H, d), device="cuda") for _ in range(2))
        assert tq.tq_read_kv(ctx.h, whole, kv, k, vv, v, 0) == tq.TQ_OK
        torch.cuda.synchronize()
        off = np.concatenate([[0], np.cumsum(lens)])
        for b in range(2):
            at = seq == b
            want = S.chunk_attention(q[at], f64(k)[off[b]:off[b + 1]], f64(v)[off[b]:off[b + 1]], pos[at],
                                     1 / math.sqrt(d))
            # the rotated queries are rounded to fp16 once more: another 2^-11
            assert C.rel_err_per_head(f64(out)[at], want).max() < C.ATTN_RTOL + 2 * half_step(torch.float16)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        lens = np.array([20, 9])
        b0 = tq.Batch(torch.as_tensor([0, 20, 29], **dev), torch.as_tensor(lens.astype(np.int32), device="cuda"), bt, 29,
                      20, cap)
        qkv = W.normal_tensor((29, Hq + 2 * H, d), seed=1, device="cuda").half()
        pos = torch.as_tensor(S.batch_positions(lens, lens)[1].astype(np.int32), device="cuda")
        qr, out = (torch.empty((29, Hq, d), dtype=torch.float16, device="cuda") for _ in range(2))
        step(b0, qkv, pos, qr, out, stream)
        stream.synchronize()
        check(lens, [20, 9], qkv, out)
        # decode
        sl = torch.as_tensor(lens.astype(np.int32), device="cuda")
        b1 = tq.Batch(torch.as_tensor([0, 1, 2], **dev), sl, bt, 2, 1, cap)
        x1 = torch.empty((2, Hq + 2 * H, d), dtype=torch.float16, device="cuda")
        p1 = torch.empty(2, **dev)
        q1, o1, o2 = (torch.empty((2, Hq, d), dtype=torch.float16, device="cuda") for _ in range(3))
        stream.synchronize()
        graphs = []
        for o in (o1, o2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                sl.add_(1)
                p1.copy_(sl).sub_(1)
                step(b1, x1, p1, q1, o, stream)
            graphs.append(g)
        sl.copy_(torch.as_tensor(lens.astype(np.int32), device="cuda"))
        for i in range(6):
            x1.copy_(W.normal_tensor((2, Hq + 2 * H, d), seed=10 + i, device="cuda").half())
            graphs[i % 2].replay()
            stream.synchronize()
            lens = lens + 1
            check(lens, [1, 1], x1, (o1, o2)[i % 2])
    torch.cuda.current_stream().wait_stream(stream)
    assert status(ctx) == 0


def test_calls_on_two_streams_at_once(ctxs):
    """Two attention calls with workspaces of their own overlap on two streams; each equals its lone run."""
    P = Paged(ctxs[128], 128, 2, [64, 1], [1500, 3000], 16)
    qs = [W.normal_tensor((65, 8, 128), seed=i, device="cuda").half() for i in (1, 2)]
    alone = [attend(P, q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.empty_like(q) for q in qs]
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 8, 2)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, s, o, w in zip(qs, streams, outs, ws):
            attend(P, q, stream=s, out=o, workspace=w)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


# ---------------------------------------------------------------------------
# calls at the edges of what the documentation allows
# ---------------------------------------------------------------------------

def test_no_tokens_need_no_memory(ctxs):
    """Empty tensors have no address: every call with no tokens succeeds, with no sequences and with idle ones."""
    ctx, d, dev = ctxs[64], 64, dict(dtype=torch.int32, device="cuda")
    rope = tq.tq_rope_build(d)
    x = torch.empty((0, 2, d), device="cuda")
    assert x.data_ptr() == 0
    assert tq.tq_rope(ctx.h, rope, x, torch.empty(0, **dev), x) == tq.TQ_OK
    kv, vv = (tq.alloc_view("q8_0", d, 2, 16, 4) for _ in range(2))
    before = kv.payload.clone()
    for n, bt in ((0, None), (0, torch.empty((0, 3), **dev)), (2, torch.zeros((2, 3), **dev))):
        b = tq.Batch(torch.zeros(n + 1, **dev), torch.full((n,), 5, **dev), bt, 0, 0, 40)
        assert tq.tq_append_kv(ctx.h, b, x, x, kv, vv, 0, rope=rope) == tq.TQ_OK
        assert tq.tq_read_kv(ctx.h, b, kv, x, vv, x, 0) == tq.TQ_OK
        ws = torch.empty(max(1, tq.tq_chunk_workspace_bytes(ctx.h, b, 4, 2)), dtype=torch.uint8, device="cuda")
        q = torch.empty((0, 4, d), device="cuda")
        assert tq.tq_chunk_attention(ctx.h, b, q, kv, vv, 0, 0.1, ws, ws.numel(), q) == tq.TQ_OK
    torch.cuda.synchronize()
    assert torch.equal(before, kv.payload) and status(ctx) == 0


def test_only_padding_rows(ctxs):
    """Rows without a sequence that owns them: max_tokens 0, nothing is read or written."""
    P = Paged(ctxs[128], 128, 1, [0, 0], [30, 7], 16, padding=6)
    q = torch.ones((6, 2, 128), dtype=torch.float16, device="cuda")
    out = attend(P, q)
    torch.cuda.synchronize()
    assert (out == 9.0).all() and status(P.ctx) == 0


def test_one_token_slices_of_odd_strides(ctxs):
    """The stride of a single token does not matter; that of two has to keep rows 16-byte aligned."""
    ctx, t = ctxs[64], tq.tq_rope_build(64)
    buf = torch.zeros((3, 2 * 64 + 1), dtype=torch.float16, device="cuda")
    x = buf.as_strided((1, 2, 64), (129, 64, 1))
    assert tq.tq_rope(ctx.h, t, x, torch.ones(1, dtype=torch.int32, device="cuda"), x) == tq.TQ_OK
    two = buf.as_strided((2, 2, 64), (129, 64, 1))
    assert tq.tq_rope(ctx.h, t, two, torch.ones(2, dtype=torch.int32, device="cuda"), two) == tq.TQ_ERR_INVALID_ARG
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_scale_of_any_sign(ctxs, d):
    """A negative scale is the negated query; a scale of 0 weighs all seen keys alike."""
    P = Paged(ctxs[d], d, 2, [140, 1, 3], [300, 700, 3], 16)
    for mods in ({}, dict(softcap=8.0, window=90)):
        check_attend(P, 2, torch.float16, scale=-1 / math.sqrt(d), **mods)
    q = W.normal_tensor((P.n_tokens, 4, d), seed=2, device="cuda").half()
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 4, 2)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    assert tq.tq_chunk_attention(P.ctx.h, P.batch, q, P.kv, P.vv, 0, 0.0, ws, n, out) == tq.TQ_OK
    torch.cuda.synchronize()
    for b in range(3):
        at = np.nonzero(P.seq == b)[0]
        v = P.stored(b)[1].repeat(2, axis=1)
        want = np.stack([v[:p + 1].mean(0) for p in P.pos[at]])
        # weights of 1 are exact; the values' rounding as in row_bound, six deviations of a mean
        mean_sq = np.stack([np.sqrt((v[:p + 1] ** 2).sum((0, 2))) / (p + 1) for p in P.pos[at]])
        bound = 6 * 2.0 ** -11 / math.sqrt(3) * mean_sq / np.maximum(np.linalg.norm(want, axis=-1), 1e-30)
        err = C.rel_err_per_head(f64(out)[at], want)
        assert (err < bound + half_step(torch.float16) + 1e-6).all(), (b, (err - bound).max())


def test_attend_sequences_that_share_pages(ctxs):
    """Two sequences with the same leading pages (a shared prompt) and own last pages, and one sequence twice."""
    P = Paged(ctxs[128], 128, 2, [3, 3, 3], [64, 64, 64], 16)
    t = P.table.copy()
    t[1, :3] = t[0, :3]
    t[2] = t[0]
    P.table = t
    P.set_batch([0, 3, 6, 9], [64, 64, 64])
    q = W.normal_tensor((3, 4, 128), seed=6, device="cuda").half().repeat(3, 1, 1)
    out = attend(P, q)
    torch.cuda.synchronize()
    assert torch.equal(out[:3], out[6:])
    for b in range(2):
        k, v = P.stored(b)
        want = S.chunk_attention(f64(q)[:3], k, v, P.pos[:3], 1 / math.sqrt(128))
        assert C.rel_err_per_head(f64(out)[3 * b:3 * b + 3], want).max() < C.ATTN_RTOL + half_step(out.dtype)
    assert not torch.equal(out[:3], out[3:6])


def test_attend_prefixes_outside_the_sequence_and_rising_bias(ctxs):
    """Prefix lengths below zero and behind the end, slopes below zero (far keys favoured)."""
    P = Paged(ctxs[64], 64, 2, [130, 2], [200, 500], 16)
    check_attend(P, 2, torch.float16, prefix=[-5, 2 ** 31 - 1])
    check_attend(P, 2, torch.float16, prefix=[2 ** 31 - 1, -2 ** 31], window=2 ** 31 - 1)
    q = W.normal_tensor((132, 4, 64), seed=3, device="cuda").half()
    slopes = torch.tensor([-0.5, 0.0, -0.01, 2.0], device="cuda")
    out = attend(P, q, mods=tq.ScoreMods(slopes=slopes))
    torch.cuda.synchronize()
    for b in range(2):
        at = np.nonzero(P.seq == b)[0]
        k, v = P.stored(b)
        want = S.chunk_attention(f64(q)[at], k, v, P.pos[at], 1 / 8, slopes=f64(slopes))
        bound = row_bound(f64(q)[at], k, v, P.pos[at], want, torch.float16, 1 / 8, slopes=f64(slopes))
        assert (C.rel_err_per_head(f64(out)[at], want) < np.maximum(bound, C.ATTN_RTOL) + half_step(out.dtype)).all()


def test_batches_are_fixed_and_on_the_gpu(ctxs):
    P = Paged(ctxs[64], 64, 1, [1], [5], 16)
    b = P.batch
    with pytest.raises(AttributeError):
        b.max_ctx = 100
    with pytest.raises(AttributeError):
        tq.ScoreMods().window = 3
    with pytest.raises(ValueError):
        tq.Batch(b.cu_tokens.cpu(), b.seq_lens, b.block_table, 1, 1, 5)
    with pytest.raises(ValueError):
        tq.Batch(b.cu_tokens, b.seq_lens, b.block_table[:, :0].contiguous(), 1, 1, 5)
    with pytest.raises(ValueError):
        tq.ScoreMods(slopes=torch.zeros(2))


# ---------------------------------------------------------------------------
# entries of few rows (decode and short speculative steps take a kernel of their own)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,new,lens,page", [
    (1, [1], [1], 16),
    (4, [1, 0, 1, 1], [15, 9, 16, 17], 16),
    (8, [1], [9000], 16),
    (2, [4, 1, 3], [4, 4000, 1537], 24),
    (5, [1] * 30, list(range(3, 3003, 100)), 1),
    (7, [2, 1], [1000, 2], 100),
    (16, [1, 1], [129, 257], 64),
    (1, [16, 7], [500, 7], 8),
    (3, [5], [2100], 256),
])
def test_attend_few_rows(ctxs, d, G, new, lens, page):
    check_attend(Paged(ctxs[d], d, 2, new, lens, page, padding=1), G, torch.float16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mods", [dict(softcap=5.0), dict(window=1), dict(window=50), dict(bias=True),
                                  dict(prefix=[500, 8, 0, 10 ** 6]),
                                  dict(softcap=20.0, window=700, bias=True, prefix=[30, 0, 100, 9])])
def test_attend_few_rows_score_modifications(ctxs, d, mods):
    P = Paged(ctxs[d], d, 2, [4, 1, 0, 3], [1900, 290, 4, 33], 16)
    check_attend(P, 2, torch.float16, **mods)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_few_rows_documents_types_and_outliers(ctxs, d):
    P = Paged(ctxs[d], d, 1, [8, 2, 1], [777, 400, 64], 16, outliers=0.01)
    first = P.pos - P.pos % 37
    first[[1, 8]] = [10 ** 9, P.pos[8] + 1]  # rows that see nothing
    first[10] = 64                           # a whole entry
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)):
        check_attend(P, 1, dtype, out, first=first)
        check_attend(P, 1, dtype, out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_few_rows_masked_values_do_not_leak(ctxs, d):
    """Infinite and NaN scales, one key each: rows that see them are NaN, the others as without them."""
    for which, bad in (("k", float("nan")), ("v", float("inf")), ("k", float("-inf")), ("v", float("nan"))):
        P = Paged(ctxs[d], d, 1, [6, 1], [260, 50], 16)
        q = W.normal_tensor((7, 1, d), seed=4, device="cuda").half()
        first = np.array([0, 131, 130, 140, 0, 259, 0])
        m = mods_of(P, 1, first=first)
        clean = attend(P, q, mods=m)
        view = P.kv if which == "k" else P.vv
        s = int(P.slots(0, [130])[0])
        h = view.header.view(torch.float16).view(-1, d // 32)
        h[s, -1] = bad
        got = attend(P, q, mods=m)
        torch.cuda.synchronize()
        sees = torch.tensor([1, 0, 1, 0, 1, 0, 0], dtype=torch.bool)
        assert torch.isnan(got[sees]).all()
        assert torch.equal(got[~sees], clean[~sees]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_few_rows_out_of_range(ctxs, d):
    ctx = ctxs[d]
    P = Paged(ctx, d, 1, [2, 1], [600, 40], 16)
    q = W.normal_tensor((3, 2, d), seed=8, device="cuda").half()
    good = P.table
    P.table = good.copy()
    P.table[0, [1, 20]] = [-7, 10 ** 6]
    P.set_batch([0, 2, 3], [600, 40])
    out = attend(P, q)
    torch.cuda.synchronize()
    assert status(ctx) == 2
    P.table = good
    k, v = P.stored(0)
    missing = np.isin(np.arange(600) // 16, [1, 20])
    want = S.chunk_attention(f64(q)[:2], k, v, P.pos[:2], 1 / math.sqrt(d), missing=missing)
    assert C.rel_err_per_head(f64(out)[:2], want).max() < C.ATTN_RTOL + half_step(out.dtype)
    for cu, lens in (([0, 2, 3], [600, 0]), ([0, 2, 3], [600, 601]), ([0, 2, 4], [600, 40])):
        P.set_batch(cu, lens)
        out = attend(P, q)
        torch.cuda.synchronize()
        assert status(ctx) == 1 and out[:2].any() and not out[2:].any(), (cu, lens)


def test_attend_few_rows_is_deterministic_and_isolated(ctxs):
    """Repeats are equal, whatever the workspace held; a NaN query row stays alone; scaled queries give the same."""
    P = Paged(ctxs[128], 128, 2, [1, 3, 1], [30000, 2000, 700], 16)
    q = W.normal_tensor((5, 8, 128), seed=5, device="cuda").to(torch.bfloat16)
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 8, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    first = attend(P, q, workspace=ws)
    for fill in (0, 255, 77):
        assert torch.equal(attend(P, q, workspace=ws.fill_(fill)), first)
    assert torch.equal(attend(P, q * 2.0 ** 40, scale=2.0 ** -40 / math.sqrt(128)), first)
    q2 = q.clone()
    q2[2, 5] = float("nan")
    got = attend(P, q2)
    torch.cuda.synchronize()
    assert torch.isnan(got[2, 5]).all()
    got[2, 5] = first[2, 5]
    assert torch.equal(got, first)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vfmt", ["turbo2_mse", "turbo3_mse", "turbo4_mse"])
@pytest.mark.parametrize("page", [16, 24, 101])
def test_attend_few_rows_turbo_values(ctxs, d, vfmt, page):
    """Pages of whole slices, pages that end inside one, and contiguous sequences of an odd capacity (odd vectors)."""
    contiguous = page == 101
    lens = [100, 17, 99, 31] if contiguous else [1900, 17, 600, 31]
    P = Paged(ctxs[d], d, 3, [2, 1, 0, 3], lens, page, vfmt, contiguous=contiguous, padding=2, outliers=0.01)
    check_attend(P, 1, torch.float16)
    check_attend(P, 2, torch.bfloat16, torch.float32, window=40, bias=True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_few_rows_contiguous_and_layers(ctxs, d):
    P = Paged(ctxs[d], d, 2, [1, 4], [77, 90], 91, n_layers=3, layer=2, contiguous=True)
    check_attend(P, 2, torch.float16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24])
def test_attend_few_rows_bad_turbo_norms_do_not_leak(ctxs, d, page):
    for which, bad in (("k", float("inf")), ("v", float("inf")), ("v", float("nan"))):
        P = Paged(ctxs[d], d, 1, [4], [260], page, "turbo3_mse")
        q = W.normal_tensor((4, 1, d), seed=4, device="cuda").half()
        m = mods_of(P, 1, first=[0, 131, 130, 140])
        clean = attend(P, q, mods=m)
        view = P.kv if which == "k" else P.vv
        h = view.header.view(torch.float16).view(-1, d // 32 if which == "k" else 1)
        h[int(P.slots(0, [130])[0]), -1] = bad
        got = attend(P, q, mods=m)
        torch.cuda.synchronize()
        sees = torch.tensor([1, 0, 1, 0], dtype=torch.bool)
        assert torch.isnan(got[sees]).all()
        assert torch.equal(got[~sees], clean[~sees]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("vfmt", ["q8_0", "turbo4_mse"])
@pytest.mark.parametrize("page", [16, 24])
def test_attend_few_rows_beyond_32_bit_offsets(ctxs, vfmt, page):
    """Pages at the end of a cache of more than 4 GiB of keys, in its second layer."""
    d, H, T = 128, 8, 100
    n_pages = (1 << 31) // (page * H * d) + 400
    kv, vv = (tq.alloc_view(f, d, H, page, n_pages, 2) for f in ("q8_0", vfmt))
    assert kv.payload.numel() > 1 << 32
    table = (n_pages - 1 - 3 * torch.arange(7, device="cuda")).to(torch.int32).view(1, 7)
    dev = dict(dtype=torch.int32, device="cuda")
    whole = tq.Batch(torch.tensor([0, T], **dev), torch.tensor([T], **dev), table, T, T, T)
    k, v, q = (W.normal_tensor((T, H, d), seed=i, device="cuda").half() for i in range(3))
    ctx = ctxs[d]
    assert tq.tq_append_kv(ctx.h, whole, k, v, kv, vv, 1) == tq.TQ_OK
    rk, rv = (torch.empty((T, H, d), device="cuda") for _ in range(2))
    assert tq.tq_read_kv(ctx.h, whole, kv, rk, vv, rv, 1) == tq.TQ_OK
    last = tq.Batch(torch.tensor([0, 2], **dev), torch.tensor([T], **dev), table, 2, 2, T)
    q = q[:2].contiguous()
    out = torch.empty_like(q)
    n = tq.tq_chunk_workspace_bytes(ctx.h, last, H, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert tq.tq_chunk_attention(ctx.h, last, q, kv, vv, 1, 1 / math.sqrt(d), ws, n, out) == tq.TQ_OK
    torch.cuda.synchronize()
    assert status(ctx) == 0
    want = S.chunk_attention(f64(q), f64(rk), f64(rv), np.arange(T - 2, T), 1 / math.sqrt(d))
    assert C.rel_err_per_head(f64(out), want).max() < C.ATTN_RTOL + half_step(torch.float16)
    del kv, vv
    torch.cuda.empty_cache()


def test_attend_few_rows_on_two_streams_at_once(ctxs):
    P = Paged(ctxs[128], 128, 2, [2, 1], [5000, 900], 16, "turbo4_mse")
    qs = [W.normal_tensor((3, 8, 128), seed=i, device="cuda").half() for i in (1, 2)]
    alone = [attend(P, q) for q in qs]
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 8, 2)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in qs]
    outs, streams = [torch.empty_like(q) for q in qs], [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, s, o, w in zip(qs, streams, outs, ws):
            attend(P, q, stream=s, out=o, workspace=w)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)

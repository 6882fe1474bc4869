"""Calls of the serving step at the ends of what its documentation allows."""
import numpy as np
import pytest
import torch

import step_checks as K
import test_gpu_step as T
from test_gpu_step import ctxs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# one chunk of many rows, one batch of few rows (the two kernels of the attention)
SHAPES = {"many": ([70, 1], [300, 129]), "few": ([2, 1], [300, 129])}


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 1.0, 50.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38])
def test_attend_caps_of_any_size(ctxs, d, shape, softcap):  # noqa: F811
    """c tanh(s / c) for scores far below the cap (a large one changes nothing) and far above it (a tiny one leaves all
    keys alike).  The bound is that of every other call: the cap's own error has to vanish in it."""
    new, lens = SHAPES[shape]
    P = T.Paged(ctxs[d], d, 2, new, lens, 16)
    K.check_attend(P, 2, torch.float16, softcap=softcap)
    K.check_attend(P, 2, torch.float16, softcap=softcap, window=90, bias=True)
    # a query of zeros has scores of zero under every cap
    out = T.attend(P, torch.zeros((P.n_tokens, 4, d), dtype=torch.float16, device="cuda"), mods=T.mods_of(P, 4, softcap))
    plain = T.attend(P, torch.zeros((P.n_tokens, 4, d), dtype=torch.float16, device="cuda"))
    assert np.isfinite(T.f64(out)).all() and torch.equal(out, plain)


# ---------------------------------------------------------------------------
# scales that fp16 does not hold
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("vfmt", ["q8_0", "turbo2_mse", "turbo3_mse", "turbo4_mse"])
def test_values_beyond_fp16_scales_read_back_as_nan(ctxs, d, vfmt, dtype):  # noqa: F811
    """Finite or infinite values whose scale (or norm) overflows: NaN in the block of 32 (or the whole vector), and every
    other value as without them.  A vector along a row of the rotation's matrix has one large coordinate after it, whose
    reconstruction would add up infinities of one sign alone."""
    P = T.Paged(ctxs[d], d, 2, [6, 1], [20, 9], 16, vfmt)
    k, v = (T.W.normal_tensor((7, 2, d), seed=i, device="cuda") for i in (1, 2))
    outs = [torch.empty((7, 2, d), device="cuda") for _ in range(4)]

    def step(k, v, out):
        assert T.tq.tq_append_kv(P.ctx.h, P.batch, k.to(T.DT[dtype]), v.to(T.DT[dtype]), P.kv, P.vv, 0) == T.tq.TQ_OK
        assert T.tq.tq_read_kv(P.ctx.h, P.batch, P.kv, out[0], P.vv, out[1], 0) == T.tq.TQ_OK
        return out
    clean = step(k, v, outs[:2])
    for x in (k, v):
        x[0, 0, 5] = 1e8
        x[1, 1, 40] = -3e38
        x[2, 0, d - 1] = float("inf")
        x[3, 1, 0] = float("-inf")
        x[4, 0] = 1e6 * torch.as_tensor(P.ctx.signs, device="cuda")
    got = step(k, v, outs[2:])
    for name, fmt, c, g in (("k", "q8_0", clean[0], got[0]), ("v", vfmt, clean[1], got[1])):
        gone = torch.zeros((7, 2, d // 32), dtype=torch.bool, device="cuda")
        if fmt == "q8_0":  # 1e6 / 127 is a scale that fp16 holds
            for t, h, i in ((0, 0, 5), (1, 1, 40), (2, 0, d - 1), (3, 1, 0)):
                gone[t, h, i // 32] = True
        else:
            for t, h in ((0, 0), (1, 1), (2, 0), (3, 1), (4, 0)):
                gone[t, h] = True
        gone = gone.repeat_interleave(32, -1)
        assert torch.isnan(g[gone]).all(), (name, g[gone])
        same = ~gone
        if fmt == "q8_0":
            same[4, 0] = False
            # codes of 127 times the scale, off by half a step of fp16; 1e6 by half a step of its type
            assert (g[4, 0].abs() - 1e6).abs().max() < 1e6 * (2 ** -11 + T.half_step(T.DT[dtype]) + 1e-6)
        assert torch.equal(g[same], c[same]), name
    assert T.status(P.ctx) == 0
    # the stored bytes themselves read back as NaN for every other reader
    deq = torch.empty((1, 2, d), device="cuda")
    slot = torch.as_tensor(P.slots(0, P.pos[:1]), device="cuda")
    assert T.tq.tq_dequantize(P.ctx.h, P.kv, 0, slot, 0, 1, 0, deq) == T.tq.TQ_OK
    torch.cuda.synchronize()
    assert torch.isnan(deq[0, 0, :32]).all() and torch.isfinite(deq[0, 0, 32:]).all()
    # and a row of the attention that sees one of them is NaN, one that does not is not
    q = T.W.normal_tensor((7, 2, d), seed=3, device="cuda").half()
    out = T.attend(P, q, mods=T.mods_of(P, 2, window=1))
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[1, 1]).all()
    assert torch.isfinite(out[0, 1]).all() and torch.isfinite(out[1, 0]).all() and torch.isfinite(out[5:]).all()


# ---------------------------------------------------------------------------
# sequences that break their bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("G,limit", [(1, None), (1, 4), (4, None)])
def test_rows_of_a_refused_sequence_are_zeros_soon(ctxs, G, limit):  # noqa: F811
    """A chunk of 8192 tokens with a length that cannot be: zeros in its rows alone, without holding up the step (34 MB of
    zeros from one thread took 8.5 ms; 5 ms are allowed)."""
    d, H, n = 128, 8, 8192 // G
    new = [3, n, 2]
    P = T.Paged(ctxs[d], d, H, [3, 1, 2], [40, 1, 30], 16)
    P.n_tokens = sum(new) + 5
    cu = np.concatenate([[0], np.cumsum(new)])
    q = T.W.normal_tensor((P.n_tokens, H * G, d), seed=4, device="cuda")
    ws_batches = []
    for lens in ([40, 1, 30], [40, -1, 30]):
        P.set_batch(cu, lens, max_tokens=limit or n, max_ctx=48)
        ws_batches.append(P.batch)
    ws = torch.empty(T.tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, H * G, H), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 9.0)
    for batch in ws_batches:
        P.batch = batch
        T.attend(P, q, out=out.fill_(9.0), workspace=ws)
        torch.cuda.synchronize()
        assert T.status(P.ctx) == 1
        assert not out[3:3 + n].any() and (out[-5:] == 9.0).all()
        assert out[:3].any(-1).all() and out[3 + n:-5].any(-1).all() and torch.isfinite(out).all()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        T.attend(P, q, out=out, workspace=ws)
        end.record()
        torch.cuda.synchronize()
        assert start.elapsed_time(end) < 5.0
    T.status(P.ctx)


# ---------------------------------------------------------------------------
# many short entries
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
def test_entries_without_a_step_for_one_of_the_issuers(ctxs, d):  # noqa: F811
    """2400 entries of 20 rows, about 16 for a block: some see nothing (no product at all), some a single key tile (a step
    for one issuing warp alone), some three (one warp is a step ahead).  Repeats are equal, every row is written."""
    n_seqs, H, n = 300, 8, 20
    kind = np.random.default_rng(d).integers(0, 3, n_seqs)
    lens = np.where(kind == 2, 300, np.where(kind == 1, 60, 25)).tolist()
    P = T.Paged(ctxs[d], d, H, [n] * n_seqs, lens, 16, fill=False, padding=3)
    x = T.W.normal_tensor((int(sum(lens)), H, d), seed=1, device="cuda").half()
    slots = torch.as_tensor(np.concatenate([P.slots(b, np.arange(t)) for b, t in enumerate(lens)]), device="cuda")
    T.C.encode(P.ctx, P.kv, x, True, slots=slots)
    T.C.encode(P.ctx, P.vv, x.flip(0).contiguous(), False, slots=slots)
    first = np.where(kind[P.seq] == 0, 10 ** 9, 0)
    first = np.concatenate([first, np.zeros(3, np.int64)])
    some = np.flatnonzero(np.arange(n_seqs) % 37 == 0)
    out = K.check_attend(P, 1, torch.float16, first=first, rows=np.flatnonzero(np.isin(P.seq, some)))
    got, empty = T.f64(out)[:P.rows], kind[P.seq] == 0
    assert np.isfinite(got).all() and not got[empty].any() and got[~empty].any(-1).all()
    q = T.W.normal_tensor((P.n_tokens, H + 2, d), seed=3, device="cuda").half()[:, 1:1 + H]
    m = T.mods_of(P, H, first=first)
    for _ in range(20):
        again = T.attend(P, q, mods=m)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and T.status(P.ctx) == 0


# ---------------------------------------------------------------------------
# scores of any height
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
def test_attend_scores_that_rise_and_fall(ctxs, d, shape, order):  # noqa: F811
    """Scores from -20000 to 20000, exact in every operand (small integers), so that the softmax's reference rises in every
    part, in none, or now and then; what is left is the rounding of values and weights."""
    new, lens = SHAPES[shape]
    P = T.Paged(ctxs[d], d, 1, new, lens, 16)
    for b, n in enumerate(lens):
        k = np.zeros((n, 1, d), np.float32)
        k[:, 0, 0] = np.linspace(-126, 126, n).round()
        if order == "falling":
            k = k[::-1].copy()
        if order == "shuffled":
            k = k[np.random.default_rng(b).permutation(n)]
        k[:, 0, 1] = 127.0  # the block's scale is 1
        T.C.encode(P.ctx, P.kv, torch.as_tensor(k, device="cuda").half(), True,
                   slots=torch.as_tensor(P.slots(b, np.arange(n)), device="cuda"))
    q = torch.zeros((P.n_tokens, 2, d), dtype=torch.float16, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    for scale in (0.01, 1.0, 160.0):
        K.check_attend(P, 2, torch.float16, scale=scale, q=q)
        K.check_attend(P, 2, torch.float16, scale=scale, q=q, bias=True, window=150)


# ---------------------------------------------------------------------------
# queries in fp32
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d,G", [(d, G) for d in (64, 128, 256) for G in (1, 4, 8, 16) if (d, G) != (256, 16)])
def test_few_rows_take_fp32_queries_in_more_bits_than_fp16(ctxs, d, G):  # noqa: F811
    """Scores that are all in the bits that fp16 does not hold: q = 1 + n 2^-20 and -1 on two coordinates where a key has
    c twice gives n c 2^-20, exact in every product and sum here; the scale makes that up to 10.  So the bound is that of
    the rounding of values and weights alone."""
    P = T.Paged(ctxs[d], d, 1, [1], [200], 16, "q8_0")
    rng = np.random.default_rng(G)
    k = np.zeros((200, 1, d), np.float32)
    k[:, 0, 0::2] = k[:, 0, 1::2] = rng.integers(-127, 128, (200, d // 2))
    k[:, 0, 0::32] = k[:, 0, 1::32] = 127.0  # every block's scale is 1
    T.C.encode(P.ctx, P.kv, torch.as_tensor(k, device="cuda").half(), True,
               slots=torch.as_tensor(P.slots(0, np.arange(200)), device="cuda"))
    at = 2 * (16 * rng.integers(0, d // 32, G) + rng.integers(1, 16, G))
    q = np.zeros((1, G, d), np.float32)
    q[0, np.arange(G), at] = 1.0 + rng.choice([-511, -300, 200, 400, 511], G) * 2.0 ** -20
    q[0, np.arange(G), at + 1] = -1.0
    scale = 10.0 * 2 ** 20 / (127 * 511)
    out = T.attend(P, torch.as_tensor(q, device="cuda"), torch.float32, scale=scale)
    torch.cuda.synchronize()
    kk, vv = P.stored(0)
    assert np.array_equal(kk, k)
    q = q.astype(np.float64)
    want = T.S.chunk_attention(q, kk, vv, P.pos, scale)
    s = np.einsum("ghd,td->ght", q, kk[:, 0]) * scale
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    noise = np.einsum("ght,t->gh", w ** 2, 2 * (2.0 ** -22 / 3) * (vv[:, 0] ** 2).sum(-1))  # as in row_bound
    K.assert_rows(T.f64(out), want, np.maximum(6 * np.sqrt(noise) / np.linalg.norm(want, axis=-1), T.C.ATTN_RTOL))


def test_read_refuses_an_output_without_a_view(ctxs):  # noqa: F811
    P = T.Paged(ctxs[64], 64, 1, [2], [5], 16)
    out = torch.zeros((2, 1, 64), device="cuda")
    for views in ((None, out, P.vv, out), (P.kv, out, None, out)):
        with pytest.raises(ValueError):
            T.tq.tq_read_kv(P.ctx.h, P.batch, *views, 0)
    assert not out.any()

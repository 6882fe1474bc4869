"""What a program that was built against an earlier include/tq.h hands to tq_chunk_attention."""
import ctypes
import math

import pytest
import torch

import test_gpu_step as T
from test_gpu_step import W, ctxs, status, tq  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 60])
def test_score_modifications_end_with_the_prefixes(ctxs, new):  # noqa: F811
    """tq_score_mods is read up to prefix_lens: what lies behind it in the caller's memory changes nothing."""
    d = 64
    P = T.Paged(ctxs[d], d, 1, [new], [700], 16, "q8_0")
    q = W.normal_tensor((new, 2, d), seed=3, device="cuda").half()
    want = T.attend(P, q, mods=tq.ScoreMods(window=50))
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 2, 1)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)

    class Former(ctypes.Structure):
        _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("slopes", ctypes.c_void_p),
                    ("first_keys", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p), ("other", ctypes.c_int32)]
    for other in (0, 40, 2 ** 31 - 1, -1):
        m = Former(0.0, 50, None, None, None, other)
        ka, va = tq._view_arg(P.kv), tq._view_arg(P.vv)
        st = tq._lib.tq_chunk_attention(P.ctx.h, ctypes.byref(P.batch.c_batch()), q.data_ptr(), 1, 2 * d, 2, ka[0], va[0], 0,
                                        1 / math.sqrt(d), ctypes.cast(ctypes.byref(m), ctypes.POINTER(tq.tq_score_mods)),
                                        ws.data_ptr(), n, out.data_ptr(), 1, None)
        assert st == tq.TQ_OK
        torch.cuda.synchronize()
        assert torch.equal(out, want) and status(P.ctx) == 0


def test_sinks_have_a_call_of_their_own(ctxs):  # noqa: F811
    """tq_chunk_attention_sinks with sinks and without, its refusals, and the former structure's size."""
    assert ctypes.sizeof(tq.tq_score_mods) == 32
    d, new = 64, 3
    P = T.Paged(ctxs[d], d, 1, [new], [700], 16, "q8_0")
    q = W.normal_tensor((new, 2, d), seed=3, device="cuda").half()
    outs = [T.attend(P, q, mods=m) for m in (tq.ScoreMods(window=50), tq.ScoreMods(window=50, sinks=8))]
    n = tq.tq_chunk_workspace_bytes(P.ctx.h, P.batch, 2, 1)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    ka, va = tq._view_arg(P.kv), tq._view_arg(P.vv)
    m = tq.tq_score_mods(0.0, 50, None, None, None)

    def call(sinks, mods=ctypes.byref(m)):
        return tq._lib.tq_chunk_attention_sinks(P.ctx.h, ctypes.byref(P.batch.c_batch()), q.data_ptr(), 1, 2 * d, 2, ka[0],
                                                va[0], 0, 1 / math.sqrt(d), mods, sinks, ws.data_ptr(), n, out.data_ptr(), 1,
                                                None)
    for sinks, want in ((0, outs[0]), (8, outs[1])):
        assert call(sinks) == tq.TQ_OK
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert not torch.equal(*outs)
    assert call(-1) == tq.TQ_ERR_INVALID_ARG
    assert call(5, None) == tq.TQ_OK  # (without a window: no effect)
    torch.cuda.synchronize()
    assert torch.equal(out, T.attend(P, q))
    f8 = tq.alloc_view("f8_block", d, 1, 16, 1)
    for bad in (tq.ScoreMods(window=-1), tq.ScoreMods(softcap=-1.0), tq.ScoreMods(softcap=math.inf)):
        assert tq.tq_chunk_workspace_for(P.ctx.h, P.batch, 2, f8, f8, bad) == 0
    torch.cuda.synchronize()
    assert status(P.ctx) == 0

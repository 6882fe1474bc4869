"""The serving step without a GPU: the rotation table against the oracle, argument refusals, the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest

from oracle import step_oracle as S

tq = pytest.importorskip("kv_cache_quantization_turbo_gb300.tq", reason="libtq.so not built")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "wavelength", "yarn"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 128), (128, 32), (256, 250), (64, 4)])
def test_rope_table_equals_the_oracle(scaling, d, rotary):
    kw = dict(base=500000.0, factor=8.0, original_ctx=8192.0)
    t = tq.tq_rope_build(d, rotary, "half", scaling, **kw)
    f, m = S.rope_angles(rotary, scaling, **kw)
    got = np.array([t.turns[i] for i in range(rotary // 2)], np.float64) * 2.0 ** -64
    want = f / (2 * math.pi) % 1.0
    # one fp64 rounding per step of the formula: a few parts in 2^52
    np.testing.assert_allclose(got, want, rtol=2e-14, atol=1e-19)
    assert all(t.turns[i] == 0 for i in range(rotary // 2, 128))
    assert t.attn_factor == pytest.approx(m, rel=1e-7) and (t.head_dim, t.rotary_dim) == (d, rotary)


def test_rope_table_defaults_and_overrides():
    t = tq.tq_rope_build(128)
    assert t.rotary_dim == 128 and t.layout == 0 and t.attn_factor == 1.0
    f, _ = S.rope_angles(128, "wavelength", factor=4.0, original_ctx=1000.0, low=2.0, high=5.0)
    t = tq.tq_rope_build(128, scaling="wavelength", factor=4.0, original_ctx=1000.0, low=2.0, high=5.0,
                         attn_factor=0.5, layout="interleaved")
    got = np.array([t.turns[i] for i in range(64)], np.float64) * 2.0 ** -64
    np.testing.assert_allclose(got, f / (2 * math.pi), rtol=2e-14)
    assert t.attn_factor == 0.5 and t.layout == 1


@pytest.mark.parametrize("kw", [
    dict(head_dim=128, rotary_dim=3), dict(head_dim=128, rotary_dim=0), dict(head_dim=64, rotary_dim=66),
    dict(head_dim=128, base=1.0), dict(head_dim=128, base=math.inf), dict(head_dim=128, base=math.nan),
    dict(head_dim=128, scaling="linear", factor=0.0), dict(head_dim=128, scaling="linear", factor=math.nan),
    dict(head_dim=128, rotary_dim=2, scaling="ntk", factor=2.0), dict(head_dim=128, scaling="yarn", factor=2.0),
    dict(head_dim=128, scaling="wavelength", factor=2.0, original_ctx=100.0, low=4.0, high=4.0),
    dict(head_dim=128, attn_factor=-1.0), dict(head_dim=128, layout=2), dict(head_dim=128, scaling=5),
    dict(head_dim=96),
])
def test_rope_table_refusals(kw):
    with pytest.raises(tq.TQError) as e:
        tq.tq_rope_build(**kw)
    assert e.value.status == (tq.TQ_ERR_UNSUPPORTED if kw["head_dim"] == 96 else tq.TQ_ERR_INVALID_ARG)


def test_null_arguments_are_refused():
    L, bad = tq._lib, tq.TQ_ERR_INVALID_ARG
    assert L.tq_rope_build(None, None) == bad
    assert L.tq_rope(None, None, None, 0, 1, 1, 64, None, 0, None, 64, None) == bad
    b = tq.tq_batch(0, 0, 0, 0, 0, None, None, None)
    assert L.tq_append_kv(None, ctypes.byref(b), None, 0, None, 0, 0, None, None, None, None, 0, None) == bad
    assert L.tq_read_kv(None, ctypes.byref(b), None, None, None, None, 0, 0, None) == bad
    assert L.tq_chunk_workspace_bytes(None, ctypes.byref(b), 8, 8) == 0
    assert L.tq_chunk_attention(None, ctypes.byref(b), None, 0, 0, 1, None, None, 0, 1.0, None, None, 0, None, 0,
                                None) == bad


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):  # 3 sequences need 4 entries
        tq.Batch(torch.zeros(3, **i32), torch.zeros(3, **i32), None, 0, 0, 0)
    with pytest.raises(ValueError):
        tq.Batch(torch.zeros(4, dtype=torch.int64), torch.zeros(3, **i32), None, 0, 0, 0)
    with pytest.raises(ValueError):
        tq.Batch(torch.zeros(4, **i32), torch.zeros(3, **i32), torch.zeros((2, 5), **i32), 0, 0, 0)
    with pytest.raises(ValueError):
        tq.ScoreMods(slopes=torch.zeros(4, dtype=torch.float64))
    t = tq.tq_rope_build(64)
    x = torch.zeros((2, 3, 64))
    with pytest.raises(ValueError):  # on the CPU
        tq.tq_rope(0, t, x, torch.zeros(2, **i32), x)
    with pytest.raises(ValueError):  # other head_dim
        tq.tq_rope(0, t, torch.zeros((2, 3, 128)), torch.zeros(2, **i32), torch.zeros((2, 3, 128)))


# ---- the oracle's own pins ----

def test_oracle_rope_is_an_isometry_and_relative():
    """<R(p) q, R(j) k> depends on p - j alone, the inverse undoes, lengths stay."""
    rng = np.random.default_rng(0)
    f, _ = S.rope_angles(32)
    q, k = rng.standard_normal((1, 1, 48)), rng.standard_normal((1, 1, 48))
    for layout in ("half", "interleaved"):
        a = np.sum(S.rope(q, [1000], f, layout=layout) * S.rope(k, [990], f, layout=layout))
        b = np.sum(S.rope(q, [10], f, layout=layout) * S.rope(k, [0], f, layout=layout))
        assert a == pytest.approx(b, rel=1e-12)
        y = S.rope(q, [77], f, layout=layout)
        np.testing.assert_allclose(S.rope(y, [77], f, layout=layout, inverse=True), q, atol=1e-14)
        np.testing.assert_array_equal(y[..., 32:], q[..., 32:])


def test_oracle_chunk_attention_reduces_to_prefill():
    from oracle import tq_oracle as O
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((12, 2, 64)), rng.standard_normal((12, 2, 64))
    want = O.prefill_attention(q, k, v, 7, 0.125)
    np.testing.assert_allclose(S.chunk_attention(q, k, v, np.arange(7, 12), 0.125), want, atol=1e-13)
    # one visible key gives its value; none gives zeros
    got = S.chunk_attention(q, k, v, np.arange(7, 12), 0.125, window=1)
    np.testing.assert_allclose(got[:, 3], v[7:, 1], atol=1e-13)
    assert not S.chunk_attention(q, k, v, np.arange(7, 12), 0.125, first_keys=np.full(5, 12)).any()

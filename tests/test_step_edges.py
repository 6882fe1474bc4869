"""Calls of the serving step at the ends of what its documentation allows, without a GPU."""
import pytest

tq = pytest.importorskip("kv_cache_quantization_turbo_gb300.tq", reason="libtq.so not built")


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=1e-320), dict(scaling="wavelength", factor=1e-320, original_ctx=8192.0),
    dict(scaling="yarn", factor=1e-320, original_ctx=8192.0),
])
def test_rope_table_refuses_angles_without_a_number(kw):
    """1 / factor overflows: the fraction of a turn was that of an infinity, different from machine to machine."""
    with pytest.raises(tq.TQError) as e:
        tq.tq_rope_build(128, **kw)
    assert e.value.status == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=1e300), dict(scaling="linear", factor=1e-300),
                                dict(scaling="ntk", factor=1e-100),
                                # the stretched pairs' angles are below 3e-3: 3e307 at most
                                dict(scaling="yarn", factor=1e-310, original_ctx=8192.0, attn_factor=1.0)])
def test_rope_table_takes_factors_far_from_one(kw):
    t = tq.tq_rope_build(128, **kw)
    assert t.attn_factor == 1.0 and all(t.turns[i] == 0 for i in range(64, 128))


def test_rope_refuses_tensors_of_other_ranks():
    torch = pytest.importorskip("torch")
    t = tq.tq_rope_build(64)
    for shape in ((64,), (2, 64), (1, 2, 3, 64)):
        x = torch.zeros(shape)
        with pytest.raises(ValueError):
            tq.tq_rope(0, t, x, torch.zeros(shape[0], dtype=torch.int32), x)

"""Norms per head, the f8_block format and sinks without a GPU: the oracle's own pins, sizes, refusals, persistence."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

tq = pytest.importorskip("kv_cache_quantization_turbo_gb300.tq", reason="libtq.so not built")


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("weight", [True, False])
def test_oracle_norm_gradient_is_that_of_differences(layout, weight):
    """Central differences of <norm_rope(x, w), dout> in fp64: step h = 2^-17 leaves h^2 times third derivatives (below
    1e2 here) and 1e-16 / h of rounding: 1e-8 in all, of values of order 1."""
    rng = np.random.default_rng(1)
    x, g, w = rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 2, 16)), 1 + 0.3 * rng.standard_normal(16)
    w = w if weight else None
    pos, (f, m) = np.array([0, 5, 900]), S.rope_angles(12)
    m = 1.3

    def loss(x, w):
        return (S.norm_rope(x, w, pos, f, 1e-3, m, layout) * g).sum()
    dx, dw = S.norm_rope_grad(x, g, w, pos, f, 1e-3, m, layout)
    h = 2.0 ** -17
    for at in [(0, 0, 0), (1, 1, 7), (2, 0, 13), (2, 1, 15)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in (0, 6, 15):
        e = np.zeros(16)
        e[i] = h
        one = np.ones(16) if w is None else w
        assert abs((loss(x, one + e) - loss(x, one - e)) / (2 * h) - dw[i]) < 1e-7


def test_oracle_norm_by_hand():
    y = S.norm_rope(np.array([[[3.0, 4.0]]]), np.array([2.0, 1.0]), [0], np.ones(1), 0.0)
    np.testing.assert_allclose(y, [[[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]]])


def test_oracle_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(S.e4m3_values(), want)
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 10.0 ** np.random.default_rng(1).integers(-5, 2, 20000),
                        [0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 17.0, 19.0, 440.0, -0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(S.e4m3_round(x), want)


def test_oracle_block_scales():
    assert [S.f8_exponent(t) for t in (448.0, 448.0001, 0.0, 1.75, 1.7500001, 1e-30, 448 * 2.0 ** 80)] == \
        [0, 1, -80, -8, -7, -80, 80]
    b = S.F8Block(2)
    b.append(np.array([[1.0, -1.75]]), 0)
    assert b.e == -8 and b.values().tolist() == [[1.0, -1.75]]
    b.append(np.array([[3.0, np.nan], [448.0, 0.3]]), 1)
    assert b.e == 0 and np.isnan(b.values()[1]).all() and b.values()[2, 0] == 448.0
    assert b.values()[0].tolist() == [1.0, -1.75]  # the earlier token keeps its value at the new scale
    b.append(np.array([[0.5, 0.25]]), 1)            # the tokens behind are gone, the scale stays
    assert b.e == 0 and b.values().tolist() == [[1.0, -1.75], [0.5, 0.25]]
    b.append(np.array([[0.5, 0.25]]), 0)            # a fresh block
    assert b.e == -9


@pytest.mark.parametrize("kw,want", [
    (dict(pos=9, length=10, window=3, sinks=2), [0, 1, 7, 8, 9]),
    (dict(pos=9, length=10, window=3, sinks=100), list(range(10))),
    (dict(pos=9, length=10, window=3), [7, 8, 9]),
    (dict(pos=9, length=10, sinks=2), list(range(10))),
    (dict(pos=9, length=10, window=3, sinks=2, first_key=4), [4, 5, 7, 8, 9]),
    (dict(pos=9, length=10, window=3, sinks=2, first_key=-4), [0, 1, 7, 8, 9]),
    (dict(pos=9, length=10, window=3, sinks=5, first_key=50), []),
    (dict(pos=2, length=10, window=2, sinks=1, prefix=5), [0, 1, 2, 3, 4]),
])
def test_oracle_sinks(kw, want):
    assert S.seen(**kw).tolist() == want


# ---------------------------------------------------------------------------
# sizes, refusals
# ---------------------------------------------------------------------------

def view(fmt="f8_block", d=128, H=2, page=32, pages=3, layers=2, bits=0):
    return tq.tq_cache_view(tq.FORMATS[fmt], d, H, page, pages, layers, bits, None, None)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sizes(d):
    assert tq.tq_format_name("f8_block") == "f8_block"
    assert tq.tq_payload_bytes("f8_block", d) == d and tq.tq_header_bytes("f8_block", d) == 0
    assert tq.tq_vector_bytes("f8_block", d) == d
    assert tq.tq_view_header_bytes(view(d=d)) == 2 * 3 * 2 * 2 * 4  # layers, pages, heads, blocks, a word each
    for fmt, bits in (("q8_0", 0), ("turbo4", 0), ("turbo2_mse", 0), ("minmax", 3)):
        assert tq.tq_view_header_bytes(view(fmt, d, bits=bits)) == 2 * 3 * 2 * 32 * tq.tq_header_bytes(fmt, d, bits)
    for bad in (view(d=96), view(page=24), view(page=0), view(H=0), view(pages=0), view(layers=0), view("minmax")):
        assert tq.tq_view_header_bytes(bad) == 0
    assert tq._lib.tq_view_header_bytes(None) == 0


def test_views_of_pages_that_are_not_blocks_are_refused():
    with pytest.raises(ValueError):
        tq.alloc_view("f8_block", 128, 2, 24, 3, device="cpu")
    v = tq.alloc_view("f8_block", 64, 2, 16, 3, n_layers=2, device="cpu")
    assert v.payload.numel() == 2 * 3 * 2 * 16 * 64 and v.header.numel() == 2 * 3 * 2 * 4


def test_null_arguments_are_refused():
    L, bad = tq._lib, tq.TQ_ERR_INVALID_ARG
    b = tq.tq_batch(0, 0, 0, 0, 0, None, None, None)
    rows, grad = tq.tq_norm_rows(), tq.tq_norm_grad_rows()
    assert L.tq_norm_rope(None, None, ctypes.byref(rows), None, 0, 0, 1e-6, 0, None, None) == bad
    assert L.tq_norm_rope_grad(None, None, ctypes.byref(grad), None, 0, 0, 1e-6, 0, None, None, 0, None) == bad
    assert L.tq_norm_rope_grad_workspace_bytes(None, 1, 1) == 0
    assert L.tq_chunk_workspace_for(None, ctypes.byref(b), 8, None, None, None) == 0


def test_saved_and_loaded(tmp_path):
    """Host arrays through a file and back, every byte."""
    rng = np.random.default_rng(3)

    def fresh():
        v = tq.alloc_view("f8_block", 64, 2, 32, 3, n_layers=2, device="cpu")
        return v, v.payload.numpy(), v.header.numpy()
    v, pay, hdr = fresh()
    pay[:] = rng.integers(0, 256, pay.shape)
    hdr[:] = rng.integers(0, 256, hdr.shape)
    path = str(tmp_path / "cache")
    assert tq.tq_cache_save(None, v, path) == tq.TQ_OK
    st, geo, _ = tq.tq_cache_file_info(path)
    assert st == tq.TQ_OK and geo["format"] == 8 and geo["page_size"] == 32
    w, pay2, hdr2 = fresh()
    assert tq.tq_cache_load(None, w, path) == tq.TQ_OK
    assert (pay2 == pay).all() and (hdr2 == hdr).all()

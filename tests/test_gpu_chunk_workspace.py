"""The size of the larger workspace of tq_chunk_attention."""
import pytest
import torch

from test_gpu_step import ctxs, tq  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_the_larger_workspace_has_a_limit(ctxs, d):  # noqa: F811
    """At most 8 GiB beside the least one, keys and values together (nothing runs: the sizes alone)."""
    view = tq.alloc_view("f8_block", d, 8, 16, 1)
    dev = dict(dtype=torch.int32, device="cuda")
    tiles = 128 * d * 2 * 2 + 64  # bytes of a tile of 128 keys of a head
    seen = set()
    for ctx in [1 << n for n in range(15, 23)]:
        b = tq.Batch(torch.zeros(2, **dev), torch.zeros(1, **dev), torch.zeros((1, ctx // 16), **dev), 4096, 4096, ctx)
        more = tq.tq_chunk_workspace_for(ctxs[d].h, b, 64, view, view) - tq.tq_chunk_workspace_bytes(ctxs[d].h, b, 64, 8)
        need = ctx // 128 * 8 * tiles
        assert more <= 8 << 30
        assert (more >= need) if need <= 8 << 30 else more == 0
        seen.add(more > 0)
    assert seen == {True, False}

"""Scales and marks that tq_append_kv writes for rotated keys, word by word.

The rotation is off by 6e-7 (|x_p| + |x_q|) per coordinate, at most 1.2e-6 of the largest magnitude of its vector's pairs, so
the exponent is the oracle's unless the block's maximum lies within 1e-5 of 448 * 2^k: asserted of the unrounded maxima."""
import numpy as np
import pytest
import torch

import test_gpu_f8 as F
from test_gpu_f8 import DT, S, ctxs, status, tq  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu


class Block(S.F8Block):
    """Remembers the largest magnitude of each append."""

    def __init__(self, d):
        super().__init__(d)
        self.tops = []

    def append(self, x, at):
        good = (np.abs(x) <= S.F8_TOP * 2.0 ** S.F8_MAX).all(-1)
        self.tops.append(np.abs(x[good]).max(initial=0.0))
        super().append(x, at)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d,rotary", [(128, 128), (64, 20), (256, 126), (128, 32), (256, 256)])
def test_words_of_rotated_keys(ctxs, monkeypatch, layout, dtype, d, rotary):  # noqa: F811
    monkeypatch.setattr(S, "F8Block", Block)
    kw = dict(base=1e4, factor=4.0, original_ctx=2048.0)
    rope = (tq.tq_rope_build(d, rotary, layout, "yarn", **kw), *S.rope_angles(rotary, "yarn", **kw), layout)
    c = F.Cache(ctxs[d], d, 3, [70, 25], [70, 25], 16)
    for n, (new, lens) in enumerate((([20, 1], [20, 1]), ([3, 8], [23, 9]), ([30, 0], [53, 9]), ([1, 16], [54, 25]),
                                     ([16, 0], [70, 25]))):
        k, v = F.tokens(sum(new), 3, d, torch.float32, 7 * n + d)
        k = k * 1.7 ** n
        if n in (1, 2):
            k[2, 1, d - 1], v[0, 2, 0] = float("inf"), float("nan")
        c.append(new, lens, k.to(DT[dtype]), v.to(DT[dtype]), rope=rope)
    torch.cuda.synchronize()
    assert status(c.ctx) == 0
    seen = 0
    for name, view in (("k", c.kv), ("v", c.vv)):
        words = view.header.view(torch.int32).cpu().numpy().view(np.uint32)
        for s in range(2):
            for (n, h), block in c.blocks[name][s].items():
                for top in block.tops:
                    if top:
                        k = top / 448.0 / 2.0 ** np.floor(np.log2(top / 448.0))  # in [1, 2)
                        assert 1 + 1e-5 < k < 2 - 2e-5, "input at a border"
                word = int(words[c.vectors(s, [16 * n])[0, h] // 16])
                marks = sum(int(m) << i for i, m in enumerate(block.marks))
                assert ((word >> 23) - 127, word & 0x7FFFFF) == (block.e, marks), (name, s, n, h)
                seen += marks != 0
    assert seen == 2  # (rows 2 and 0 of the second and third append lie in the same block)

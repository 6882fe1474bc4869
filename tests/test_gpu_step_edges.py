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

"""tq_norm_rope_grad where sums pass fp32."""
import pytest
import torch

from test_gpu_norm import Call, ctxs  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu


def test_sums_of_weight_gradients_beyond_fp32(ctxs):  # noqa: F811
    """Gradients whose sum passes fp32 give an infinity of its sign."""
    c = Call(ctxs[64], 64, 64, "half", torch.float32, 4000, (2, 1), wtype=torch.float32, seed=5, far=1)
    c.x[0][:, :, 5] = 1.0
    c.g[0][:, :, 5] = 1e36
    c.x[0][:, :, 9] = 1.0
    c.g[0][:, :, 9] = -1e36
    _, dws = c.backward()
    torch.cuda.synchronize()
    assert dws[0][5] == float("inf") and dws[0][9] == -float("inf")
    assert torch.isfinite(dws[1]).all()

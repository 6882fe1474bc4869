"""tq_norm_rope and tq_norm_rope_grad where a value that is not finite lies in a coordinate that is not rotated: it stays
there.  Bounds of finite values as in tests/test_gpu_norm.py."""
import numpy as np
import pytest
import torch

from test_gpu_norm import DT, Call, S, ctxs, f64, pair_sum, rounding  # noqa: F401  (ctxs: the fixture)

pytestmark = pytest.mark.gpu

HEADS = [(128, 96, "half"), (128, 96, "interleaved"), (64, 20, "half"), (256, 64, "half"), (64, 6, "interleaved"),
         (128, 34, "half")]


def partner(i, rotary, layout):
    if i >= rotary:
        return i
    return i ^ 1 if layout == "interleaved" else (i + rotary // 2) % rotary


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d,rotary,layout", HEADS)
def test_infinite_coordinates(ctxs, dtype, d, rotary, layout):  # noqa: F811
    """NaN in an infinite coordinate and the one rotated with it, 0 in the others of its vector, other vectors as before."""
    c = Call(ctxs[d], d, rotary, layout, DT[dtype], 40, (2, 1), wtype=torch.float32, seed=2)
    clean = [o.clone() for o in c.forward()]
    at = sorted({0, 1, rotary // 2, rotary - 1, rotary, rotary + 1, rotary + 7, rotary + 8, d - 9, d - 8, d - 1})
    for n, i in enumerate(at):
        c.x[n % 2][2 * n, 0, i] = float("inf") if n % 3 else -float("inf")
    out = c.forward()
    torch.cuda.synchronize()
    for n, i in enumerate(at):
        hit = torch.zeros(d, dtype=torch.bool, device="cuda")
        hit[[i, partner(i, rotary, layout)]] = True
        row = out[n % 2][2 * n, 0]
        assert torch.isnan(row[hit]).all() and not row[~hit].any(), (i, torch.isnan(row).nonzero().ravel().tolist())
    for k in range(2):
        keep = torch.ones(out[k].shape[:2], dtype=torch.bool, device="cuda")
        keep[[2 * n for n in range(len(at)) if n % 2 == k], 0] = False
        assert torch.equal(out[k][keep], clean[k][keep])


@pytest.mark.parametrize("d,rotary,layout", HEADS)
def test_results_beyond_fp32(ctxs, d, rotary, layout):  # noqa: F811
    """A weight that takes a coordinate beyond fp32 makes an infinity of it and leaves the others."""
    c = Call(ctxs[d], d, rotary, layout, torch.float32, 20, (2, 1), wtype=torch.float32, seed=3)
    for i in (rotary, d - 9, d - 1):
        w = [t.clone() for t in c.w]
        c.w[0][i] = 3e38
        c.x[0][:, :, i] = 4.0
        out = c.forward()
        torch.cuda.synchronize()
        big = torch.isinf(out[0][..., i])
        assert big.any()
        rest = torch.ones(d, dtype=torch.bool, device="cuda")
        rest[i] = False
        y = f64(c.x[0]) / np.sqrt((f64(c.x[0]) ** 2).mean(-1, keepdims=True) + c.eps) * f64(c.w[0])
        y[..., i] = 0.0
        want = S.rope(y, c.pos, c.f, c.m, layout)
        tol = 1.6e-6 * c.m * pair_sum(y, rotary, layout) + rounding(torch.float32, want)
        assert (np.abs(f64(out[0]) - want) <= tol)[..., rest.cpu().numpy()].all()
        c.w = w


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d,rotary,layout", HEADS)
def test_infinite_gradients(ctxs, dtype, d, rotary, layout):  # noqa: F811
    """An infinite gradient of a coordinate that is not rotated makes an infinity of that coordinate of the weight's
    gradient; the others' and other vectors' gradients stay."""
    c = Call(ctxs[d], d, rotary, layout, DT[dtype], 700, (3, 2), wtype=torch.float32, seed=4)
    dx, dws = c.backward()
    torch.cuda.synchronize()
    dx, dws = [t.clone() for t in dx], [t.clone() for t in dws]
    at = sorted({rotary, d - 9, d - 1})
    for n, i in enumerate(at):
        g = [t.clone() for t in c.g]
        keep_g, k = c.g, n % 2
        c.x[k][300, 1, i] = 1.0
        ref_x, ref_w = c.backward()
        torch.cuda.synchronize()
        ref_x, ref_w = [t.clone() for t in ref_x], [t.clone() for t in ref_w]
        g[k][300, 1, i] = float("inf") if n % 2 else -float("inf")
        c.g = g
        got_x, got_w = c.backward()
        torch.cuda.synchronize()
        assert torch.isinf(got_w[k][i]) and (got_w[k][i] > 0) == bool(n % 2), got_w[k][i]
        rest = torch.arange(d, device="cuda") != i
        assert torch.equal(got_w[k][rest], ref_w[k][rest]) and torch.equal(got_w[1 - k], ref_w[1 - k])
        keep = torch.ones(got_x[k].shape[:2], dtype=torch.bool, device="cuda")
        keep[300, 1] = False
        assert torch.equal(got_x[k][keep], ref_x[k][keep]) and torch.equal(got_x[1 - k], ref_x[1 - k])
        # (the vector itself: its sum over g w x' is infinite)
        assert not torch.isfinite(got_x[k][300, 1]).any()
        c.g = keep_g


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

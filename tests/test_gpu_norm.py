"""GPU parity of tq_norm_rope and tq_norm_rope_grad against the fp64 oracle.

Tolerances, fixed before the first run.  All is fp32 until the result is rounded once.
  * forward: r = rsqrtf (2 ulp, 2.4e-7) of a sum of squares of up to 16 + 4 additions of positive terms in a chain (20 2^-24,
    half of that in the root: 6e-7), two products (1.2e-7); the rotation 6e-7 (as tq_rope).  1.6e-6 of m (|y_p| + |y_q|), the
    sizes of a pair before its rotation, plus half a step of the output type;
  * gradient of x: g has the rotation's 6e-7, x' = r x 1e-6, their sum over d as above 1.2e-6: 4e-6 of what the terms of
    the formula add up to in magnitude, plus half a step;
  * gradient of the weight: terms as above (2e-6), a lane adds up at most 8 rows (5000 tokens) in a chain, a CTA 5 + 8 more,
    each 2^-24 of the magnitudes so far; the rest carries what it loses along: 4e-6 of the sum of magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import test_gpu_step as T
from test_gpu_step import DT, ctxs, f64, rounding  # noqa: F401  (ctxs: the fixture)
from kv_cache_quantization_turbo_gb300 import tq
from kv_cache_quantization_turbo_gb300 import workloads as W
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

KW = dict(base=500000.0, factor=8.0, original_ctx=8192.0)


def pair_sum(a, rotary, layout):
    """|a| of a coordinate plus that of its partner; unrotated ones alone."""
    a = np.abs(a)
    out = a.copy()
    r2 = rotary // 2
    p, q = (slice(0, r2), slice(r2, rotary)) if layout == "half" else (slice(0, rotary, 2), slice(1, rotary, 2))
    out[..., p] = out[..., q] = a[..., p] + a[..., q]
    return out


class Call:
    """Inputs of one call, and its checks."""

    def __init__(self, ctx, d, rotary, layout, dtype, tokens, heads, *, wtype=None, scaling="none", eps=1e-6, seed=0,
                 far=100000, size=1.0):
        self.ctx, self.d, self.rotary, self.layout, self.eps = ctx, d, rotary, layout, eps
        self.table = tq.tq_rope_build(d, rotary, layout, scaling, **KW)
        self.f, self.m = S.rope_angles(rotary, scaling, **KW)
        self.pos = np.random.default_rng(seed).integers(0, far, tokens).astype(np.int32)
        self.pos_t = torch.as_tensor(self.pos, device="cuda")
        hq, hk = heads
        both = (size * W.normal_tensor((tokens, hq + hk + 1, d), seed=seed, device="cuda")).to(dtype)
        self.x = [both[:, :hq] if hq else None, both[:, hq:hq + hk] if hk else None]
        self.w = [None, None]
        if wtype is not None:
            w = (1 + 0.3 * W.normal_tensor((2, d), seed=seed + 1, device="cuda")).to(wtype)
            self.w = [w[0], w[1]]
        self.g = [None if x is None else W.normal_tensor(tuple(x.shape), seed=seed + 2 + i, device="cuda").to(dtype)
                  for i, x in enumerate(self.x)]
        self.tokens, self.heads, self.dtype = tokens, heads, dtype

    def empty(self, value=7.0):
        return [None if x is None else torch.full(tuple(x.shape), value, dtype=self.dtype, device="cuda") for x in self.x]

    def forward(self, out=None, stream=None):
        out = out or self.empty()
        a = [t for i in range(2) for t in (self.x[i], out[i], self.w[i])]
        st = tq.tq_norm_rope(self.ctx.h, self.table, *a, self.eps, self.pos_t, stream=stream)
        assert st == tq.TQ_OK, tq.tq_status_string(st)
        return out

    def backward(self, dx=None, dw="both", ws=None, stream=None):
        dx = dx or self.empty()
        dws = [torch.full((self.d,), 5.0, device="cuda") if x is not None and dw == "both" else None for x in self.x]
        n = tq.tq_norm_rope_grad_workspace_bytes(self.ctx.h, self.tokens, sum(self.heads))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) if ws is None else ws
        a = [t for i in range(2) for t in (self.x[i], self.g[i], self.w[i], dx[i], dws[i])]
        st = tq.tq_norm_rope_grad(self.ctx.h, self.table, *a, self.eps, self.pos_t, ws, n, stream=stream)
        assert st == tq.TQ_OK, tq.tq_status_string(st)
        return dx, dws

    def check_forward(self, out):
        torch.cuda.synchronize()
        for x, w, o in zip(self.x, self.w, out):
            if x is None:
                continue
            x, w = f64(x), None if w is None else f64(w)
            want = S.norm_rope(x, w, self.pos, self.f, self.eps, self.m, self.layout)
            y = x / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps) * (1.0 if w is None else w)
            tol = 1.6e-6 * max(self.m, 1.0) * pair_sum(y, self.rotary, self.layout) + rounding(o.dtype, want)
            err = np.abs(f64(o) - want)
            assert (err <= tol).all(), ((err - tol).max(), np.argwhere(~(err <= tol))[:5])

    def check_backward(self, dx, dws):
        torch.cuda.synchronize()
        for x, w, g, o, dw in zip(self.x, self.w, self.g, dx, dws):
            if x is None:
                continue
            x, w, g = f64(x), np.ones(self.d) if w is None else f64(w), f64(g)
            want, want_w = S.norm_rope_grad(x, g, w, self.pos, self.f, self.eps, self.m, self.layout)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
            ga, xr = max(self.m, 1.0) * pair_sum(g, self.rotary, self.layout), np.abs(x * r)
            size = r * (ga * np.abs(w) + xr * (ga * np.abs(w) * xr).sum(-1, keepdims=True) / self.d)
            err = np.abs(f64(o) - want) - rounding(o.dtype, want)
            assert (err <= 4e-6 * size).all(), ((err / size).max(), np.argwhere(~(err <= 4e-6 * size))[:5])
            if dw is not None:
                assert (np.abs(f64(dw) - want_w) <= 4e-6 * (ga * xr).sum((0, 1))).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 128), (128, 64), (256, 256), (256, 40), (64, 20), (128, 126),
                                      (256, 2), (64, 32)])
def test_layouts_types_and_parts(ctxs, dtype, layout, d, rotary):  # noqa: F811
    c = Call(ctxs[d], d, rotary, layout, DT[dtype], 37, (5, 2), wtype=DT[dtype], seed=rotary)
    c.check_forward(c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("tokens,heads", [(1, (1, 1)), (1, (40, 8)), (3, (33, 0)), (700, (0, 9)), (5000, (7, 1)),
                                          (513, (16, 16)), (2048, (1, 1))])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sizes_and_one_side_alone(ctxs, d, tokens, heads):  # noqa: F811
    c = Call(ctxs[d], d, d, "half", torch.bfloat16, tokens, heads, wtype=torch.float32, seed=tokens)
    c.check_forward(c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("wtype", [None, "fp32", "fp16", "bf16"])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_weights_and_factors(ctxs, wtype, scaling):  # noqa: F811
    """Weights of every type and none; a factor on the rotated coordinates; an eps that counts."""
    c = Call(ctxs[128], 128, 96, "half", torch.float32, 50, (3, 2), wtype=None if wtype is None else DT[wtype],
             scaling=scaling, eps=0.5, seed=3)
    c.check_forward(c.forward())
    c.check_backward(*c.backward())
    c.check_backward(*c.backward(dw=None))


@pytest.mark.parametrize("dtype", list(DT))
def test_in_place_strides_and_neighbours(ctxs, dtype):  # noqa: F811
    """Results over the inputs, rows of a wider matrix: what lies between the rows stays."""
    for layout in ("half", "interleaved"):
        c = Call(ctxs[64], 64, 64, layout, DT[dtype], 300, (4, 3), wtype=DT[dtype], seed=5)
        fresh, grads = c.forward(), c.backward()
        buf = torch.cat([c.x[0], c.x[1], torch.full((300, 2, 64), 3.0, device="cuda", dtype=DT[dtype])], 1)
        c.x = [buf[:, :4], buf[:, 4:7]]
        c.forward(out=c.x)
        torch.cuda.synchronize()
        assert torch.equal(buf[:, :4], fresh[0]) and torch.equal(buf[:, 4:7], fresh[1]) and (buf[:, 7:] == 3.0).all()
        c = Call(ctxs[64], 64, 64, layout, DT[dtype], 300, (4, 3), wtype=DT[dtype], seed=5)
        dx, dws = c.backward(dx=c.g)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(dx + dws, grads[0] + grads[1]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_magnitudes_whose_squares_leave_fp32(ctxs, d, dtype):  # noqa: F811
    """Rows of 1e25 and 1e37, next to ordinary ones in the same warp, and rows far below sqrt(eps)."""
    c = Call(ctxs[d], d, d, "half", DT[dtype], 40, (3, 2), wtype=torch.float32, seed=1)
    scale = torch.tensor([1.0, 1e25, 1e-25, 3e37, 1e-3], device="cuda").repeat(8)[:, None, None]
    c.x = [(x.float().clamp(-5, 5) * scale).to(x.dtype) for x in c.x]
    c.check_forward(c.forward())
    dx, dws = c.backward()
    torch.cuda.synchronize()
    for x, w, g, o in zip(c.x, c.w, c.g, dx):
        want, _ = S.norm_rope_grad(f64(x), f64(g), f64(w), c.pos, c.f, c.eps, c.m)
        xs, r = f64(x), 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + c.eps)
        ga, xr, aw = pair_sum(f64(g), d, "half"), np.abs(xs * r), np.abs(f64(w))
        size = r * (ga * aw + xr * (ga * aw * xr).sum(-1, keepdims=True) / d)
        # gradients of 1e-37 are near the end of fp32's normal numbers (1.2e-38): 2^-149 absolute, times a few
        assert (np.abs(f64(o) - want) <= 4e-6 * size + rounding(o.dtype, want) + 8 * 2.0 ** -149).all()
    assert all(torch.isfinite(w).all() for w in dws)


def test_zero_rows_and_rows_that_are_not_finite(ctxs):  # noqa: F811
    c = Call(ctxs[128], 128, 128, "half", torch.float16, 16, (2, 1), wtype=torch.float16, seed=2)
    clean = [o.clone() for o in c.forward()]
    c.x[0][3, 0] = 0.0
    c.x[0][5, 1, 17] = float("nan")
    c.x[1][7, 0, 100] = float("inf")
    out = c.forward()
    torch.cuda.synchronize()
    assert not out[0][3, 0].any()
    assert torch.isnan(out[0][5, 1]).all()
    hit = torch.zeros(128, dtype=torch.bool, device="cuda")
    hit[[36, 100]] = True  # the pair of the infinity; the others are x / infinity
    assert torch.isnan(out[1][7, 0][hit]).all() and not out[1][7, 0][~hit].any()
    for i, (a, b) in enumerate(zip(out, clean)):
        keep = torch.ones(16, c.heads[i], dtype=torch.bool, device="cuda")
        for t, h in ([(3, 0), (5, 1)], [(7, 0)])[i]:
            keep[t, h] = False
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("layout,rotary", [("half", 128), ("interleaved", 128), ("half", 50)])
def test_gradient_is_that_of_differences(ctxs, layout, rotary):  # noqa: F811
    """Central differences of the kernel's own forward pass in fp32, along random directions: <f(x + h v) - f(x - h v), g> /
    2 h.  h = 2^-6: the third-order term is h^2 / 6 of third derivatives of order |v|^3 per element of unit-size rows,
    below h^2 of the magnitudes' sum; the values' fp32 error 1.6e-6 / h of it."""
    c = Call(ctxs[128], 128, rotary, layout, torch.float32, 64, (3, 2), wtype=torch.float32, seed=7, far=5000)
    dx, dws = c.backward()
    h = 2.0 ** -6
    v = [W.normal_tensor(tuple(x.shape), seed=20 + i, device="cuda") for i, x in enumerate(c.x)]
    vw = [W.normal_tensor((128,), seed=30 + i, device="cuda") for i in range(2)]
    base_x, base_w = [x.clone() for x in c.x], [w.clone() for w in c.w]

    def value(s, t):
        c.x = [x + s * a for x, a in zip(base_x, v)]
        c.w = [w + t * a for w, a in zip(base_w, vw)]
        out = c.forward()
        torch.cuda.synchronize()
        return [(o.double() * g.double()).sum((1, 2)) for o, g in zip(out, c.g)]
    for s, t, grads in ((h, 0.0, [(d * a).double().sum((1, 2)) for d, a in zip(dx, v)]), (0.0, h, None)):
        up, down = value(s, t), value(-s, -t)
        for i in range(2):
            size = (c.g[i].abs().double() * (v[i].abs() + 1).double()).sum((1, 2))
            diff = (up[i] - down[i]) / (2 * h)
            if grads is not None:
                assert ((diff - grads[i]).abs() < (h * h + 4e-6 / h) * size).all()
            else:
                total = float((dws[i] * vw[i]).double().sum())
                assert abs(float(diff.sum()) - total) < (4e-6 / h) * float(size.sum())


def test_no_tokens(ctxs):  # noqa: F811
    c = Call(ctxs[64], 64, 64, "half", torch.float32, 0, (2, 1), wtype=torch.float32)
    c.forward()
    _, dws = c.backward()
    torch.cuda.synchronize()
    assert not any(w.any() for w in dws)


def test_repeats_graphs_and_streams(ctxs):  # noqa: F811
    """The same bits on every run, in a replayed graph, and from two streams at once with a workspace each."""
    c = Call(ctxs[128], 128, 128, "half", torch.bfloat16, 1500, (9, 3), wtype=torch.bfloat16, seed=9)
    out, (dx, dws) = c.forward(), c.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in out + dx + dws]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(5):
                o = c.forward(stream=s)
                d, w = c.backward(stream=s)
            got.append(o + d + w)
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    o, d = c.empty(), c.empty()
    dw = [torch.empty(128, device="cuda") for _ in range(2)]
    n = tq.tq_norm_rope_grad_workspace_bytes(c.ctx.h, 1500, 12)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        assert tq.tq_norm_rope(c.ctx.h, c.table, c.x[0], o[0], c.w[0], c.x[1], o[1], c.w[1], c.eps, c.pos_t,
                               stream=torch.cuda.current_stream()) == tq.TQ_OK
        assert tq.tq_norm_rope_grad(c.ctx.h, c.table, c.x[0], c.g[0], c.w[0], d[0], dw[0], c.x[1], c.g[1], c.w[1], d[1],
                                    dw[1], c.eps, c.pos_t, ws, n, stream=torch.cuda.current_stream()) == tq.TQ_OK
    for _ in range(3):
        for t in o + d + dw:
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o + d + dw, want))


def test_refusals(ctxs):  # noqa: F811
    ctx = ctxs[64]
    c = Call(ctx, 64, 64, "half", torch.float32, 4, (2, 1), wtype=torch.float32)
    n = tq.tq_norm_rope_grad_workspace_bytes(ctx.h, 4, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    x, pos, w = torch.zeros((4, 2, 64), device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), c.w[0]
    y, p = torch.zeros_like(x), x.data_ptr()
    rows = dict(x=p, x_token_stride=128, out=y.data_ptr(), out_token_stride=128, weight=w.data_ptr(), n_heads=2)
    grad = dict(x=p, x_token_stride=128, dout=p, dout_token_stride=128, weight=w.data_ptr(), dx=y.data_ptr(),
                dx_token_stride=128, dweight=w.data_ptr(), n_heads=2)
    base = dict(ctx=ctx.h, dtype=0, wtype=0, eps=1e-6, n=4, pos=pos.data_ptr(), ws=ws.data_ptr(), bytes=n)

    def call(change=None, fwd=True, **kw):
        a = {**base, **kw}
        r = {**(rows if fwd else grad), **(change or {})}
        s = ctypes.byref((tq.tq_norm_rows if fwd else tq.tq_norm_grad_rows)(**r))
        head = (a["ctx"], ctypes.byref(c.table), s, None, a["dtype"], a["wtype"], a["eps"], a["n"], a["pos"])
        if fwd:
            return tq._lib.tq_norm_rope(*head, None)
        return tq._lib.tq_norm_rope_grad(*head, a["ws"], a["bytes"], None)
    for fwd in (True, False):
        assert call(fwd=fwd) == tq.TQ_OK
        assert call(fwd=fwd, n=0) == tq.TQ_OK
        for kw in (dict(dtype=3), dict(wtype=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf")), dict(eps=1e-39), dict(n=-1), dict(pos=None), dict(ctx=ctxs[128].h)):
            assert call(fwd=fwd, **kw) == tq.TQ_ERR_INVALID_ARG, kw
        outs = ("out",) if fwd else ("dout", "dx")
        for change in (dict(x=None), dict(x=p + 4), dict(x_token_stride=127), dict(x_token_stride=130), dict(n_heads=0),
                       dict(n_heads=1 << 21), dict(weight=w.data_ptr() + 2), *({k: None} for k in outs),
                       *({k + "_token_stride": 64} for k in outs), {outs[-1]: p, outs[-1] + "_token_stride": 132}):
            assert call(change, fwd=fwd) == tq.TQ_ERR_INVALID_ARG, change
    for kw in (dict(ws=None), dict(bytes=n - 1), dict(ws=ws.data_ptr() + 64)):
        assert call(fwd=False, **kw) == tq.TQ_ERR_WORKSPACE
    assert call(dict(dweight=w.data_ptr() + 2), fwd=False) == tq.TQ_ERR_INVALID_ARG
    assert tq._lib.tq_norm_rope(ctx.h, ctypes.byref(c.table), None, None, 0, 0, 1e-6, 4, pos.data_ptr(), None) == \
        tq.TQ_ERR_INVALID_ARG
    torch.cuda.synchronize()
    for bad in ((None, None, None, None, None, None), (x, None, w, None, None, None), (x, y[:3], w, None, None, None),
                (x, y.half(), w, None, None, None), (x, y, w[:32], None, None, None), (x, y, w.cpu(), None, None, None),
                (x, y, w, x.half(), y.half(), w), (x, y, w, x, y, w.half())):
        with pytest.raises(ValueError):
            tq.tq_norm_rope(ctx.h, c.table, *bad, 1e-6, pos)
    with pytest.raises(ValueError):
        tq.tq_norm_rope_grad(ctx.h, c.table, x, x, w, y, w.half(), None, None, None, None, None, 1e-6, pos, ws, n)
    assert T.status(ctx) == 0

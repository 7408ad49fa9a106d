"""GPU parity of layer norm (forward, gradients) and of the norm-and-gate
gradients against the fp64 oracle, through the C ABI.

Tolerances.  All arithmetic is float32 (u = 2^-24) on rows of up to 16384
channels; statistics are sums of at most ~64 sequential adds joined by a tree,
so each carries under 80 u, and an output element a few of those: 1e-5 of the
row's largest output (168 u) bounds it.  A mean far from zero costs
cancellation in x - mu: 4 u |mu| rstd of one output unit is added.  A bf16
store adds half a step, 2^-8 of the value.  The weights' gradients sum one
term per token with signs: their error is measured against the sum of the
terms' sizes (1e-5, the chains being shorter than 150 adds).  The size of xh
there is |xh| + max|x| rstd / 2: the mean's 80 u max|x| (4.8e-6) moves xh by
that times rstd however small xh itself is.
"""

import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_retention_b200 import ops, workloads as W
from tests._util import BF16_U
from tests.test_gpu_guards import assert_guards, guarded

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def draw(shape, dtype, seed, scale=1.0, shift=0.0):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale + shift).to(W.torch_dtype(dtype))


def check(got, ref, what, shift=0.0):
    """Row by row: within 1e-5 of the row's largest element, plus the store and the shift."""
    stored = got.dtype == torch.bfloat16
    g = W.to_f64(got).reshape(ref.shape)
    assert np.all(np.isfinite(g)), f"{what}: non-finite"
    bound = (1e-5 + 4 * U32 * shift) * np.abs(ref).max(axis=-1, keepdims=True) + 1e-30
    if stored:
        bound = bound + BF16_U * np.abs(ref)
    worst = (np.abs(g - ref) / bound).max(initial=0.0)
    assert worst <= 1.0, f"{what}: an element is {worst:.2f} times its bound off"


def check_sum(got, ref, size, what):
    err = np.abs(W.to_f64(got).reshape(ref.shape) - ref)
    assert np.all(err <= 1e-5 * size + 1e-30), f"{what}: off by {(err / (size + 1e-30)).max():.2e} of the terms"


def xh_size(x, eps=1e-5):
    mu, rstd = x.mean(-1, keepdims=True), 1 / np.sqrt(x.var(-1, keepdims=True) + eps)
    return (np.abs(x - mu) + np.abs(x).max(-1, keepdims=True) / 2) * rstd


LN_SHAPES = [(1, 1), (3, 2), (1, 37), (7, 64), (33, 100), (5, 256), (300, 96), (129, 1001), (64, 1024),
             (3, 2056), (40, 4096), (2, 5000), (700, 512), (9, 8192), (3, 9999), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("n,D", LN_SHAPES)
@pytest.mark.parametrize("x_t,y_t", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm(n, D, x_t, y_t, affine):
    x, dy = draw((n, D), x_t, n + D), draw((n, D), y_t, n + D + 1)
    w, b = (draw((D,), "f32", 3, 0.5, 1.0), draw((D,), "f32", 4)) if affine else (None, None)
    f = lambda t: None if t is None else W.to_f64(t)  # noqa: E731
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    td = W.torch_dtype(y_t)
    y, mean, rstd = ops.layer_norm_fwd(d(x), d(w), d(b), out_dtype=td, return_stats=True)
    assert y.dtype == td and mean.shape == rstd.shape == (n,)
    check(y, oracle.layer_norm(f(x), f(w), f(b)), "y")
    x64 = f(x)
    # the mean against the row's size, 1/sqrt(var + eps) against itself
    assert np.all(np.abs(W.to_f64(mean) - x64.mean(-1)) <= 80 * U32 * np.abs(x64).max(-1))
    rs = 1 / np.sqrt(x64.var(-1) + 1e-5)
    assert np.all(np.abs(W.to_f64(rstd) - rs) <= 1e-5 * rs)
    got = ops.layer_norm_bwd(d(x), d(dy), mean, rstd, d(w), grad_dtype=td)
    dx, dw, db = oracle.layer_norm_backward(x64, f(dy), f(w))
    if D > 2:              # one or two channels: dx is a difference of equal terms
        check(got[0], dx, "dx")
    check_sum(got[1], dw, (np.abs(f(dy)) * xh_size(x64)).sum(0), "d_weight")
    check_sum(got[2], db, np.abs(f(dy)).sum(0), "d_bias")
    only = ops.layer_norm_bwd(d(x), d(dy), mean, rstd, d(w), grad_dtype=td, return_d_affine=False)
    assert torch.equal(only, got[0])
    assert torch.equal(ops.layer_norm_fwd(d(x), d(w), d(b), out_dtype=td), y)


@pytest.mark.parametrize("n,D", [(5, 1), (4, 2)])
def test_layer_norm_of_one_or_two_channels(n, D):
    """With one channel y is the bias and dx zero; with two, dx is what eps leaves: absolute
    bounds (a few u of the terms rstd n, which cancel)."""
    x, dy, w = draw((n, D), "f32", 1), draw((n, D), "f32", 2), draw((D,), "f32", 3)
    y, mean, rstd = ops.layer_norm_fwd(x.cuda(), w.cuda(), None, return_stats=True)
    dx, _, _ = ops.layer_norm_bwd(x.cuda(), dy.cuda(), mean, rstd, w.cuda())
    ref = oracle.layer_norm_backward(W.to_f64(x), W.to_f64(dy), W.to_f64(w))[0]
    size = W.to_f64(rstd)[:, None] * np.abs(W.to_f64(dy) * W.to_f64(w)).max(-1, keepdims=True)
    assert np.all(np.abs(W.to_f64(dx) - ref) <= 64 * U32 * size)
    np.testing.assert_allclose(W.to_f64(y), oracle.layer_norm(W.to_f64(x), W.to_f64(w)), atol=1e-5)


def test_layer_norm_far_from_zero_and_constant_rows():
    x = draw((6, 512), "f32", 1, shift=300.0)
    x[2] = 7.25                                             # no variance: y = bias, rstd = 1/sqrt(eps)
    dy = draw((6, 512), "f32", 2)
    y, mean, rstd = ops.layer_norm_fwd(x.cuda(), return_stats=True)
    ref = oracle.layer_norm(W.to_f64(x))
    rows = [0, 1, 3, 4, 5]
    check(y[rows], ref[rows], "y", shift=300.0)
    assert torch.equal(y[2].cpu(), torch.zeros(512)) and abs(float(rstd[2]) - 1e-5 ** -0.5) < 1e-2
    dx, dw, db = ops.layer_norm_bwd(x.cuda(), dy.cuda(), mean, rstd)
    rdx, rdw, rdb = oracle.layer_norm_backward(W.to_f64(x), W.to_f64(dy))
    check(dx, rdx, "dx", shift=300.0)
    check_sum(dw, rdw, (np.abs(W.to_f64(dy)) * xh_size(W.to_f64(x))).sum(0), "dw")


def test_layer_norm_rows_are_independent():
    """NaN and infinity stay in their row (and in the weights' gradients)."""
    x, dy = draw((9, 300), "f32", 1), draw((9, 300), "f32", 2)
    y0, m0, r0 = ops.layer_norm_fwd(x.cuda(), return_stats=True)
    d0 = ops.layer_norm_bwd(x.cuda(), dy.cuda(), m0, r0)
    x[4, 7], x[6, 0] = float("nan"), float("inf")
    y, m, r = ops.layer_norm_fwd(x.cuda(), return_stats=True)
    g = ops.layer_norm_bwd(x.cuda(), dy.cuda(), m, r)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(g[0][keep], d0[0][keep])
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).all() and torch.equal(g[2], d0[2])


def test_no_tokens():
    x = torch.empty(0, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    y, m, r = ops.layer_norm_fwd(x, w, return_stats=True)
    assert y.shape == (0, 40) and m.shape == (0,)
    dx, dw, db = ops.layer_norm_bwd(x, x, m, r, w)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()
    o = torch.empty(0, 2, 20, device="cuda")
    d_o, d_g, dw, db = ops.norm_gate_bwd(o, o, o)
    assert d_o.shape == (0, 2, 20) and not dw.any() and not db.any() and dw.shape == (40,)


def test_layer_norm_leading_dimensions():
    x = draw((2, 3, 5, 48), "f32", 1).cuda()
    y, m, r = ops.layer_norm_fwd(x, return_stats=True)
    assert y.shape == x.shape and m.shape == (2, 3, 5)
    assert torch.equal(y.view(30, 48), ops.layer_norm_fwd(x.view(30, 48)))
    one = ops.layer_norm_fwd(x[0, 0, 0].contiguous())
    assert one.shape == (48,) and torch.equal(one, y[0, 0, 0])


NG_SHAPES = [(1, 1, 1), (2, 3, 2), (1, 1, 33), (5, 2, 64), (40, 3, 100), (3, 5, 128), (300, 2, 96),
             (7, 16, 256), (70, 4, 512), (2, 1, 1024), (11, 3, 1000), (5, 2, 777), (600, 1, 24), (4, 70, 40)]


@pytest.mark.parametrize("n,H,dv", NG_SHAPES)
@pytest.mark.parametrize("o_t,g_t,grad_t", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                             ("f32", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                             ("bf16", "bf16", "f32"), ("f32", "f32", "bf16")])
@pytest.mark.parametrize("affine", [False, True])
def test_norm_gate_gradients(n, H, dv, o_t, g_t, grad_t, affine):
    o, g, dy = draw((n, H, dv), o_t, n + dv, 0.5), draw((n, H * dv), g_t, dv), draw((n, H, dv), g_t, 7)
    w, b = (draw((H * dv,), "f32", 3, 0.5, 1.0), draw((H * dv,), "f32", 4)) if affine else (None, None)
    f = lambda t: None if t is None else W.to_f64(t)  # noqa: E731
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    td = W.torch_dtype(grad_t)
    got = ops.norm_gate_bwd(d(o), d(g), d(dy), d(w), d(b), grad_dtype=td)
    w2, b2 = [None if t is None else f(t).reshape(H, dv) for t in (w, b)]
    ref = oracle.norm_gate_backward(f(o), f(g), f(dy), weight=w2, bias=b2)
    assert got[0].dtype == got[1].dtype == td and got[0].shape == o.shape and got[1].shape == g.shape
    if dv > 2:
        check(got[0], ref[0], "d_o")
    check(got[1], ref[1], "d_g")
    dt = f(dy) * oracle.swish(f(g)).reshape(n, H, dv)
    check_sum(got[2], ref[2], (np.abs(dt) * xh_size(f(o))).sum(0), "d_weight")
    check_sum(got[3], ref[3], np.abs(dt).sum(0), "d_bias")
    only = ops.norm_gate_bwd(d(o), d(g), d(dy), d(w), d(b), grad_dtype=td, return_d_affine=False)
    assert all(torch.equal(p, q) for p, q in zip(only, got))


def test_norm_gate_gradients_match_differences():
    """Central differences of msr_norm_gate itself (float32, step 2^-5: truncation step^2/6 of
    third derivatives of order one, 2e-4; rounding 1e-6 / step = 3e-5), to 1e-3 of the scale."""
    n, H, dv = 3, 2, 40
    o, g, dy = (draw((n, H, dv), "f32", s).cuda() for s in (1, 2, 3))
    w, b = draw((H * dv,), "f32", 4, 0.3, 1.0).cuda(), draw((H * dv,), "f32", 5).cuda()
    grads = ops.norm_gate_bwd(o, g, dy, w, b)
    base = dict(o=o, g=g, weight=w, bias=b)
    step = 2.0 ** -5
    scale = max(float(t.abs().max()) for t in grads)
    for (name, t), grad in zip(base.items(), grads):
        for k in (0, 17, t.numel() - 1):
            v = []
            for sign in (1, -1):
                m = t.reshape(-1).clone()
                m[k] += sign * step
                v.append(float((ops.norm_gate(**dict(base, **{name: m.view(t.shape)})).double() * dy.double()).sum()))
            fd = (v[0] - v[1]) / (2 * step)
            assert abs(fd - float(grad.reshape(-1)[k])) <= 1e-3 * scale, (name, k)


def test_norm_gate_extreme_gates():
    """Gates far out: swish and its slope saturate without NaN; infinite gates as the formula."""
    n, H, dv = 4, 1, 64
    o, dy = draw((n, H, dv), "f32", 1), draw((n, H, dv), "f32", 2)
    g = draw((n, H, dv), "f32", 3)
    g[0, 0, 0], g[1, 0, 1], g[2, 0, 2], g[3, 0, 3] = -100.0, 100.0, -1e30, 1e30
    d_o, d_g, dw, db = ops.norm_gate_bwd(o.cuda(), g.cuda(), dy.cuda())
    for t in (d_o, d_g, dw, db):
        assert torch.isfinite(t).all()
    ref = oracle.norm_gate_backward(*[W.to_f64(t) for t in (o, g, dy)])
    check(d_o, ref[0], "d_o")
    check(d_g, ref[1], "d_g")


@pytest.mark.parametrize("n,D", [(37, 300), (130, 1024)])
def test_write_only_their_outputs(n, D):
    x, dy = draw((n, D), "bf16", 1).cuda(), draw((n, D), "bf16", 2).cuda()
    y, yb = guarded((n, D), torch.bfloat16)
    _, mean, rstd = ops.layer_norm_fwd(x, out=y, return_stats=True)
    assert_guards(yb, "y")
    ws, wb = guarded((max(256, ops.layer_norm_bwd_workspace_size(n, D)),), torch.uint8)
    ops.layer_norm_bwd(x, dy, mean, rstd, workspace=ws)
    assert_guards(wb, "workspace")
    # the C call, with every output guarded
    for tail in (True, False):
        outs = [guarded((n, D), torch.float32)] + [guarded((D,), torch.float32) for _ in range(2)]
        if tail:
            st = ops.lib().retention_layer_norm_bwd(
                ops._ptr(x), 1, ops._ptr(dy), 1, ops._ptr(mean), ops._ptr(rstd), None,
                ops._ptr(outs[0][0]), 0, ops._ptr(outs[1][0]), ops._ptr(outs[2][0]), ops._ptr(ws),
                ws.numel(), n, D, ops._stream(None))
        else:
            outs.append(guarded((n, D), torch.float32))
            ng = ops.NormGate(dy.data_ptr(), 1, None, None, 1e-5)
            H = 2
            ws, wb = guarded((max(256, ops.norm_gate_bwd_workspace_size(n, H, D // H)),), torch.uint8)
            st = ops.lib().msr_norm_gate_bwd(
                ops._ptr(x), 1, ops.ctypes.byref(ng), ops._ptr(dy), ops._ptr(outs[0][0]),
                ops._ptr(outs[3][0]), 0, ops._ptr(outs[1][0]), ops._ptr(outs[2][0]), ops._ptr(ws),
                ws.numel(), n, H, D // H, ops._stream(None))
        assert st == ops.RET_OK
        torch.cuda.synchronize()
        for _, buf in outs:
            assert_guards(buf, "output")
        assert_guards(wb, "workspace")


def test_streams_graphs_and_repeats():
    """The same bits on two streams at once, captured and replayed, and in every run."""
    x, dy = draw((999, 520), "bf16", 1).cuda(), draw((999, 520), "bf16", 2).cuda()
    o, g = x.view(999, 2, 260), draw((999, 2, 260), "bf16", 3).cuda()
    w = draw((520,), "f32", 4).cuda()

    def once(stream=None):
        y, m, r = ops.layer_norm_fwd(x, w, return_stats=True, stream=stream)
        return ((y,) + tuple(ops.layer_norm_bwd(x, dy, m, r, w, stream=stream))
                + tuple(ops.norm_gate_bwd(o, g, dy.view(o.shape), w, stream=stream)))
    want = once()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [once(s) for s in streams]
        junk = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        for q in got:
            assert all(torch.equal(a, b) for a, b in zip(q, want))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = once()
        graphs.append((gr, out))
    for gr, out in graphs:
        for t in out:
            t.zero_()
    for gr, _ in graphs:
        gr.replay()
    eager = once()
    torch.cuda.synchronize()
    for out in [o for _, o in graphs] + [eager]:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows equal a short call's."""
    n, D = 132000, 16384                                   # 2.16e9 elements
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    x, dy = (torch.randn(n, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y, m, r = ops.layer_norm_fwd(x, return_stats=True)
    k = n - 5
    y2, m2, r2 = ops.layer_norm_fwd(x[k:].clone(), return_stats=True)
    torch.testing.assert_close(y[k:].float(), y2.float(), rtol=2.0 ** -7, atol=1e-6)
    torch.testing.assert_close(r[k:], r2, rtol=1e-6, atol=0)
    dx, dw, db = ops.layer_norm_bwd(x, dy, m, r)
    dx2 = ops.layer_norm_bwd(x[k:].clone(), dy[k:].clone(), m2, r2)[0]
    torch.testing.assert_close(dx[k:].float(), dx2.float(), rtol=2.0 ** -7, atol=1e-6)
    assert torch.isfinite(dw).all()
    del dx, dx2, y, y2
    o, dyo = x.view(n, 16, 1024), dy.view(n, 16, 1024)
    d_o, d_g, dw, db = ops.norm_gate_bwd(o, dyo, dyo)
    e = ops.norm_gate_bwd(o[k:].clone(), dyo[k:].clone(), dyo[k:].clone())
    torch.testing.assert_close(d_o[k:].float(), e[0].float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(d_g[k:].float(), e[1].float(), rtol=2.0 ** -7, atol=1e-5)


def test_binding_refusals():
    x = torch.zeros(4, 16, device="cuda")
    m = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ops.layer_norm_fwd(x.t())
    with pytest.raises(ValueError, match="weight must be"):
        ops.layer_norm_fwd(x, m)
    with pytest.raises(ValueError, match="bias must be"):
        ops.layer_norm_fwd(x, None, torch.zeros(16, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out must be"):
        ops.layer_norm_fwd(x, out=x[:2].clone())
    with pytest.raises(TypeError, match="unsupported dtype"):
        ops.layer_norm_fwd(x.half())
    with pytest.raises(ops.RetentionError):
        ops.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(ops.RetentionError, match="UNSUPPORTED"):
        ops.layer_norm_fwd(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(ValueError, match="mean must be"):
        ops.layer_norm_bwd(x, x, m[:2].clone(), m)
    with pytest.raises(ValueError, match="d_y must be"):
        ops.layer_norm_bwd(x, x[:2].clone(), m, m)
    o = x.view(4, 2, 8)
    with pytest.raises(ValueError, match="g must have"):
        ops.norm_gate_bwd(o, o.bfloat16(), o)
    with pytest.raises(ValueError, match="weight must be"):
        ops.norm_gate_bwd(o, o, o, weight=m)
    with pytest.raises(ValueError, match="d_y must be"):
        ops.norm_gate_bwd(o, o, o[:2].clone())
    with pytest.raises(ops.RetentionError, match="UNSUPPORTED"):
        big = torch.zeros(1, 1, 1028, device="cuda")
        ops.norm_gate_bwd(big, big, big)

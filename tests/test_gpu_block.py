"""The new operators together, as a training step and a serving loop use them.

A retention block in float32: layer norm, the projections (plain matrix
products), the chunkwise retention, GroupNorm + gate, and back through every
one of them to the block's input and weights, against the same chain of
fp64 oracle functions.  Each float32 operator is within rel-L2 1e-5 of its
oracle on its own inputs; the chain passes through at most six of them (forward
and backward), so 6e-5 bounds an output.  In bfloat16 every operator's result
is rounded (2^-8 of a value at most, 2^-9 rms) at up to ten places of the chain:
rel-L2 10 * 2^-8 = 4e-2.
"""

import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_retention_b200 import ops, workloads as W
from tests._util import rel_l2

pytestmark = pytest.mark.gpu

F32_CHAIN, BF16_CHAIN = 6e-5, 4e-2


def close(got, ref, tol, what):
    e = rel_l2(W.to_f64(got), ref)
    assert e <= tol, f"{what}: rel-L2 {e:.2e} > {tol}"


def weights(seed, *shapes):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal(s) / np.sqrt(s[0])).float() for s in shapes]


@pytest.mark.parametrize("dtype,T,H,dk,dv,chunk", [("f32", 77, 2, 16, 32, 16), ("bf16", 300, 2, 64, 128, 128)])
def test_training_step_of_a_retention_block(dtype, T, H, dk, dv, chunk):
    B, Dm = 2, 96
    td, tol = W.torch_dtype(dtype), F32_CHAIN if dtype == "f32" else BF16_CHAIN
    gen = torch.Generator()
    gen.manual_seed(3)
    x = torch.randn(B * T, Dm, generator=gen).to(td)
    dy = torch.randn(B, T, H, dv, generator=gen).to(td)
    wn, bn = 1 + 0.1 * torch.randn(Dm, generator=gen), 0.1 * torch.randn(Dm, generator=gen)
    wg, bg = 1 + 0.1 * torch.randn(H * dv, generator=gen), 0.1 * torch.randn(H * dv, generator=gen)
    proj = [w.to(td) for w in weights(0, (Dm, H * dk), (Dm, H * dk), (Dm, H * dv), (Dm, H * dv))]
    gam = W.head_gammas(H)
    shapes = [(B, T, H, dk), (B, T, H, dk), (B, T, H, dv), (B, T, H * dv)]

    # on the GPU, every intermediate in `dtype`
    c = [t.cuda() for t in (x, dy, wn, bn, wg, bg)]
    pw = [p.cuda() for p in proj]
    xd, dyd, wnd, bnd, wgd, bgd = c
    xn, mean, rstd = ops.layer_norm_fwd(xd, wnd, bnd, return_stats=True)
    q, k, v, g = [(xn @ p).view(s) for p, s in zip(pw, shapes)]
    o = ops.chunkwise_fwd(q, k, v, gam, chunk)
    y = ops.norm_gate(o, g, wgd, bgd)
    d_o, d_g, d_wg, d_bg = ops.norm_gate_bwd(o, g, dyd, wgd, bgd)
    dq, dk_, dv_ = ops.chunkwise_bwd(q, k, v, d_o, gam, chunk)
    dp = [t.reshape(B * T, -1).to(td) for t in (dq, dk_, dv_, d_g)]
    d_xn = sum(t.float() @ p.float().t() for t, p in zip(dp, pw)).to(td)
    d_proj = [xn.float().t() @ t.float() for t in dp]
    dx, d_wn, d_bn = ops.layer_norm_bwd(xd, d_xn, mean, rstd, wnd)
    ops.check_device_error()

    # the same chain in float64
    f = W.to_f64
    X, DY = f(x), f(dy)
    P = [f(p) for p in proj]
    XN = oracle.layer_norm(X, f(wn), f(bn))
    Q, K, V, G = [(XN @ p).reshape(s) for p, s in zip(P, shapes)]
    O, _ = oracle.msr_chunkwise(Q, K, V, gam, chunk)
    Y = oracle.norm_gate(O, G, weight=f(wg).reshape(H, dv), bias=f(bg).reshape(H, dv))
    DO, DG, DWG, DBG = oracle.norm_gate_backward(O, G, DY, weight=f(wg).reshape(H, dv),
                                                 bias=f(bg).reshape(H, dv))
    DQ, DK, DV, _ = oracle.msr_backward(Q, K, V, gam, DO)
    DP = [t.reshape(B * T, -1) for t in (DQ, DK, DV, DG)]
    DXN = sum(t @ p.T for t, p in zip(DP, P))
    DX, DWN, DBN = oracle.layer_norm_backward(X, DXN, f(wn))
    for name, a, b in [("y", y, Y), ("d_gn_weight", d_wg, DWG.ravel()), ("d_gn_bias", d_bg, DBG.ravel()),
                       ("dx", dx, DX), ("d_norm_weight", d_wn, DWN), ("d_norm_bias", d_bn, DBN)] + [
            (f"d_proj{n}", a, XN.T @ b) for n, (a, b) in enumerate(zip(d_proj, DP))]:
        close(a, b, tol, name)

    # the chain's gradient against a difference along a random direction (float64)
    def loss(X):
        XN = oracle.layer_norm(X, f(wn), f(bn))
        q, k, v, g = [(XN @ p).reshape(s) for p, s in zip(P, shapes)]
        o, _ = oracle.msr_chunkwise(q, k, v, gam, chunk)
        return float(np.sum(DY * oracle.norm_gate(o, g, weight=f(wg).reshape(H, dv), bias=f(bg).reshape(H, dv))))
    step = np.random.default_rng(1).standard_normal(X.shape) * 1e-5
    assert abs(loss(X + step) - loss(X - step) - 2 * np.sum(DX * step)) <= 1e-5 * np.linalg.norm(DX) * np.linalg.norm(step)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_of_a_recurrent_block(dtype):
    """Layer norm, projections, the gated linear recurrence and back."""
    B, T, Dm, D = 2, 150, 64, 96
    td, tol = W.torch_dtype(dtype), F32_CHAIN if dtype == "f32" else BF16_CHAIN
    gen = torch.Generator()
    gen.manual_seed(5)
    x, dh = torch.randn(B * T, Dm, generator=gen).to(td), torch.randn(B, T, D, generator=gen).to(td)
    wn, bn = 1 + 0.1 * torch.randn(Dm, generator=gen), 0.1 * torch.randn(Dm, generator=gen)
    lam = torch.randn(D, generator=gen) - 4.0
    proj = [w.to(td) for w in weights(1, (Dm, D), (Dm, D), (Dm, D))]
    xd, dhd, wnd, bnd, ld = [t.cuda() for t in (x, dh, wn, bn, lam)]
    pw = [p.cuda() for p in proj]
    xn, mean, rstd = ops.layer_norm_fwd(xd, wnd, bnd, return_stats=True)
    u, r, i = [(xn @ p).view(B, T, D) for p in pw]
    h, S, chunks = ops.glr_fwd(u, r, i, ld, return_state=True, return_chunks=True)
    du, dr, di, d_lam = ops.glr_bwd(u, r, i, ld, chunks, dhd)
    d_xn = sum(t.view(B * T, D).float() @ p.float().t() for t, p in zip((du, dr, di), pw)).to(td)
    dx, d_wn, d_bn = ops.layer_norm_bwd(xd, d_xn, mean, rstd, wnd)

    f = W.to_f64
    P = [f(p) for p in proj]
    XN = oracle.layer_norm(f(x), f(wn), f(bn))
    U, R, I = [(XN @ p).reshape(B, T, D) for p in P]
    Href, Sref = oracle.glr(U, R, I, f(lam))
    DU, DR, DI, DL, _ = oracle.glr_backward(U, R, I, f(lam), f(dh))
    DXN = sum(t.reshape(B * T, D) @ p.T for t, p in zip((DU, DR, DI), P))
    DX, DWN, DBN = oracle.layer_norm_backward(f(x), DXN, f(wn))
    for name, a, b in [("h", h, Href), ("state", S, Sref), ("du", du, DU), ("dr", dr, DR), ("di", di, DI),
                       ("d_lam", d_lam, DL), ("dx", dx, DX), ("d_norm_weight", d_wn, DWN), ("d_norm_bias", d_bn, DBN)]:
        close(a, b, tol, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_then_steps_equal_one_forward(dtype):
    """Serving: a packed prefill of prompts of different lengths, then one token at a time for
    all of them, against the recurrence over the whole sequences (float32 outputs: the class
    bound 1e-5)."""
    lens, extra, D = [1, 130, 64, 0, 7], 5, 200
    td = W.torch_dtype(dtype)
    gen = torch.Generator()
    gen.manual_seed(8)
    lam = torch.randn(D, generator=gen) - 4.0
    full = [[torch.randn(n + extra, D, generator=gen).to(td) for _ in range(3)] for n in lens]
    cu = torch.from_numpy(W.cu_seqlens_of(lens)).cuda()
    prompt = [torch.cat([s[a][:n] for s, n in zip(full, lens)])[None].cuda() for a in range(3)]
    h, S = ops.glr_fwd(*prompt, lam.cuda(), cu_seqlens=cu, return_state=True, out_dtype=torch.float32)
    steps = []
    for t in range(extra):
        tok = [torch.stack([s[a][n + t] for s, n in zip(full, lens)]).cuda() for a in range(3)]
        steps.append(ops.glr_step(*tok, lam.cuda(), S))
    first = 0
    for n, seq in enumerate(full):
        ref, Sref = oracle.glr(*[W.to_f64(t)[None] for t in seq], W.to_f64(lam))
        L = lens[n]
        if L:
            close(h[:, first:first + L], ref[:, :L], 1e-5, f"prompt {n}")
        first += L
        for t in range(extra):
            close(steps[t][n], ref[0, L + t], 1e-5, f"sequence {n} token {t}")
        close(S[n], Sref[0], 1e-5, f"state {n}")

"""Pins for the oracle's gated linear recurrence, layer norm and norm gradients.

The forwards are pinned by closed forms that share nothing with them (a product
form of the recurrence, constant gates, torch's float64 layer norm), every
gradient by central differences of its forward, and packed sequences by the
separate calls.
"""

import numpy as np
import pytest
import torch

import oracle


def _glr_inputs(rng, B, T, D, nstate=None):
    n = nstate or B
    return dict(x=rng.standard_normal((B, T, D)), r=rng.standard_normal((B, T, D)),
                i=rng.standard_normal((B, T, D)), lam=rng.standard_normal(D) - 2.0,
                state=rng.standard_normal((n, D)))


def test_glr_product_form():
    """h_t = (prod a) S0 + sum_m (prod_{j>m} a_j) v_m, the recurrence unrolled."""
    rng = np.random.default_rng(0)
    p = _glr_inputs(rng, 1, 7, 3)
    h, S = oracle.glr(**p)
    a = np.exp(-8.0 * np.log1p(np.exp(p["lam"])) / (1 + np.exp(-p["r"][0])))
    v = np.sqrt(1 - a ** 2) / (1 + np.exp(-p["i"][0])) * p["x"][0]
    for t in range(7):
        ref = np.prod(a[:t + 1], axis=0) * p["state"][0]
        for m in range(t + 1):
            ref = ref + np.prod(a[m + 1:t + 1], axis=0) * v[m]
        np.testing.assert_allclose(h[0, t], ref, rtol=1e-12, atol=1e-14)
    np.testing.assert_array_equal(S[0], h[0, -1])


def test_glr_keeps_unit_variance_and_extreme_gates():
    """Open input gate, constant decay: h = a^t S0 + ...; closed gates pass the state through."""
    rng = np.random.default_rng(1)
    p = _glr_inputs(rng, 1, 4, 2)
    p["r"][:] = -800.0                       # a = 1: nothing decays, nothing enters
    h, _ = oracle.glr(**p)
    np.testing.assert_allclose(h[0], np.broadcast_to(p["state"][0], (4, 2)), rtol=1e-15)
    p["r"][:] = 800.0
    p["lam"][:] = 800.0                      # a = 0: only the token's own input is left
    h, _ = oracle.glr(**p)
    np.testing.assert_allclose(h[0], p["x"][0] / (1 + np.exp(-p["i"][0])), rtol=1e-14)
    grads = oracle.glr_backward(d_h=np.ones((1, 4, 2)), **p)
    assert all(np.all(np.isfinite(g)) for g in grads)


def test_glr_packed_equals_separate_calls():
    rng = np.random.default_rng(2)
    lens = [3, 0, 1, 5]
    cu = np.concatenate([[0], np.cumsum(lens)])
    p = _glr_inputs(rng, 1, 9, 2, nstate=4)
    dh, dS = rng.standard_normal((1, 9, 2)), rng.standard_normal((4, 2))
    h, S = oracle.glr(**p, cu_seqlens=cu)
    got = oracle.glr_backward(**p, d_h=dh, d_state=dS, cu_seqlens=cu)
    dlam = np.zeros(2)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        one = dict(x=p["x"][:, a:b], r=p["r"][:, a:b], i=p["i"][:, a:b], lam=p["lam"],
                   state=p["state"][s:s + 1])
        hs, Ss = oracle.glr(**one)
        np.testing.assert_array_equal(h[:, a:b], hs)
        np.testing.assert_array_equal(S[s], Ss[0])
        g = oracle.glr_backward(**one, d_h=dh[:, a:b], d_state=dS[s:s + 1])
        for full, part in zip(got[:3], g[:3]):
            np.testing.assert_array_equal(full[:, a:b], part)
        dlam += g[3]
        np.testing.assert_array_equal(got[4][s], g[4][0])
    np.testing.assert_allclose(got[3], dlam, rtol=1e-13)
    chunks = oracle.glr_chunk_states(h, p["state"], 2, cu)
    assert set(chunks) == {(0, 0), (0, 1), (2, 0), (3, 0), (3, 1), (3, 2)}
    np.testing.assert_array_equal(chunks[3, 1], h[0, cu[3] + 1])


def _differences(f, args, grads, step=1e-5, rtol=2e-8):
    """Central differences of the scalar f: truncation ~step^2, rounding ~1e-16/step, both
    ~1e-10 of the gradients' scale; rtol leaves two orders."""
    scale = max(1.0, max(float(np.abs(g).max()) for g in grads.values()))
    for name, g in grads.items():
        for idx in np.ndindex(args[name].shape):
            up, dn = args[name].copy(), args[name].copy()
            up[idx] += step
            dn[idx] -= step
            fd = (f(**dict(args, **{name: up})) - f(**dict(args, **{name: dn}))) / (2 * step)
            assert abs(fd - g[idx]) <= rtol * scale, (name, idx, fd, g[idx])


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 6]])
def test_glr_gradients_match_differences(cu):
    rng = np.random.default_rng(3)
    p = _glr_inputs(rng, 1, 6, 2, nstate=None if cu is None else 3)
    dh, dS = rng.standard_normal((1, 6, 2)), rng.standard_normal(p["state"].shape)

    def loss(**a):
        h, S = oracle.glr(**a, cu_seqlens=cu)
        return float(np.sum(dh * h) + np.sum(dS * S))
    g = oracle.glr_backward(**p, d_h=dh, d_state=dS, cu_seqlens=cu)
    _differences(loss, p, dict(zip(("x", "r", "i", "lam", "state"), g)))


def test_a_wrong_glr_gradient_is_caught():
    """The differences catch a backward that reads h_t in place of h_(t-1)."""
    rng = np.random.default_rng(4)
    p = _glr_inputs(rng, 1, 5, 2)
    dh = rng.standard_normal((1, 5, 2))
    h, _ = oracle.glr(**p)
    good = oracle.glr_backward(**p, d_h=dh)
    shifted = oracle.glr_backward(**dict(p, state=h[:, 0]), d_h=dh)
    with pytest.raises(AssertionError):
        _differences(lambda **a: float(np.sum(dh * oracle.glr(**a)[0])), p, {"r": shifted[1]})
    _differences(lambda **a: float(np.sum(dh * oracle.glr(**a)[0])), p, {"r": good[1]})


def test_layer_norm_matches_torch_float64():
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((4, 3, 7)) + 2.0, rng.standard_normal((4, 3, 7))
    w, b = rng.standard_normal(7), rng.standard_normal(7)
    tx, tw, tb = (torch.from_numpy(a).requires_grad_() for a in (x, w, b))
    y = torch.nn.functional.layer_norm(tx, (7,), tw, tb, 1e-3)
    np.testing.assert_allclose(oracle.layer_norm(x, w, b, 1e-3), y.detach().numpy(), rtol=1e-12,
                               atol=1e-13)
    ref = torch.autograd.grad(y, (tx, tw, tb), torch.from_numpy(dy))
    for got, want in zip(oracle.layer_norm_backward(x, dy, w, 1e-3), ref):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("affine", [False, True])
def test_norm_gate_gradients_match_differences(affine):
    rng = np.random.default_rng(6)
    a = dict(o=rng.standard_normal((2, 2, 3)), g=rng.standard_normal((2, 2, 3)))
    if affine:
        a |= dict(weight=rng.standard_normal((2, 3)), bias=rng.standard_normal((2, 3)))
    dy = rng.standard_normal((2, 2, 3))
    g = oracle.norm_gate_backward(d_y=dy, eps=1e-2, **a)
    names = ("o", "g", "weight", "bias") if affine else ("o", "g")
    _differences(lambda **k: float(np.sum(dy * oracle.norm_gate(eps=1e-2, **k))), a,
                 dict(zip(names, g)))
    if not affine:                            # weight and bias gradients at weight 1, bias 0
        one = dict(a, weight=np.ones((2, 3)), bias=np.zeros((2, 3)))
        _differences(lambda **k: float(np.sum(dy * oracle.norm_gate(eps=1e-2, **k))), one,
                     dict(weight=g[2], bias=g[3]))

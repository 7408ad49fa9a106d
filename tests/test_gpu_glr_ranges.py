"""The gated linear recurrence at the ends of its parameters' ranges, against the fp64
oracle (tolerances of test_gpu_glr.py)."""

import numpy as np
import pytest
import torch

from linear_recurrent_sequence_retention_b200 import ops, workloads as W
from tests.test_gpu_glr import C, Reference, cuda, make

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 31, 33, 64, 100, 1100])
@pytest.mark.parametrize("D", [40, 65])
def test_gate_scale_beyond_the_largest_float(dtype, T, D):
    """c softplus(lam) overflows: the decay is zero, so every token starts anew.  The padding of
    the last tile must not turn that into NaN.  The oracle's limit of an infinite lam is the
    finite 1e38's (both decays are below any float64)."""
    x, r, i, lam, dh, S0, dS = make(2, T, D, dtype, seed=T)
    big = [4.3e37, 1e38, 3.4e38, INF]
    lam[:4] = torch.tensor(big)
    r[:, :, 1:4] = r[:, :, 1:4].abs()
    r[:, 0, 0], r[:, -1, 0] = 17.0, 100.0                    # the sigmoid saturates at one
    ref = Reference(x, r, i, lam.clamp(max=3.4e38), dh, S0, dS)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, return_state=True,
                               return_chunks=True, out_dtype=torch.float32)
    ref.check_forward(h, S, T, chunks)
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, d_state_out=dSd, return_d_state=True,
                      grad_dtype=torch.float32)
    ref.check_gradients(got, T)
    # the step, from the same states
    tok = [t[:, 0].contiguous() for t in (xd, rd, id_)]
    h1 = ops.glr_step(*tok, ld, S0d.clone())
    torch.testing.assert_close(h1, h[:, 0], rtol=1e-5, atol=1e-6)
    assert torch.equal(h1[:, :4], h[:, 0, :4])
    ops.check_device_error()


def test_large_gate_constant():
    """The same overflow from c: every channel decays at once, the padding changes nothing."""
    x, r, i, lam, dh, S0, dS = make(1, 70, 33, seed=3)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, torch.full_like(lam, 2.0), dh, S0, dS)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, c=3e38, state_in=S0d, return_state=True,
                               return_chunks=True)
    want = W.to_f64(x) / (1 + np.exp(-W.to_f64(i)))
    np.testing.assert_allclose(W.to_f64(h), want, rtol=1e-5, atol=1e-7)
    assert torch.equal(S, h[:, -1])
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, c=3e38, d_state_out=dSd, return_d_state=True)
    assert all(torch.isfinite(g).all() for g in got)
    assert not got[1].any() and not got[3].any() and not got[4].any()


def test_gate_of_nan_stays_nan():
    x, r, i, lam, dh, S0, dS = cuda(*make(1, 70, 33, seed=4))
    clean = ops.glr_fwd(x, r, i, lam)
    lam[5] = float("nan")
    h, S, chunks = ops.glr_fwd(x, r, i, lam, state_in=None, return_state=True, return_chunks=True)
    assert torch.isnan(h[:, :, 5]).all() and torch.isnan(S[:, 5]).all()
    keep = torch.arange(33, device="cuda") != 5
    assert torch.equal(h[:, :, keep], clean[:, :, keep])
    got = ops.glr_bwd(x, r, i, lam, chunks, dh)
    assert all(torch.isnan(g[..., 5]).all() for g in got)
    assert all(torch.isfinite(g[..., keep]).all() for g in got)


@pytest.mark.parametrize("T", [9, 40])
def test_lam_whose_exponential_is_subnormal(T):
    """sigmoid(lam) / softplus(lam) tends to one from below zero on, also where exp(-lam) is
    infinite in float32 (lam < -88.7).  A large c makes such channels count.  softplus(lam) is
    then subnormal: at lam >= -89.5 it is off by at most two of 2^-149, 2.1e-6 of itself, which
    every bound below leaves room for."""
    c = 1e38
    x, r, i, lam, dh, S0, dS = make(2, T, 24, seed=T)
    lam[:] = torch.linspace(-89.5, -85.0, 24)
    # the oracle at its default c and the lam that gives the same decays; d_lam / d(c softplus)
    # differs by the factors, the one here being one to 1e-37
    scale = c * np.exp(W.to_f64(lam))
    same = np.log(np.expm1(scale / C))
    ref = Reference(x, r, i, torch.from_numpy(same), dh, S0, dS)
    factor = (1 + np.exp(-same)) * scale / C
    ref.dlam, ref.dlam_size = ref.dlam * factor, ref.dlam_size * factor
    args = cuda(x, r, i, lam, dh, S0, dS)
    h, S, chunks = ops.glr_fwd(*args[:4], c=c, state_in=args[5], return_state=True, return_chunks=True)
    ref.check_forward(h, S, T, chunks)
    ref.check_gradients(ops.glr_bwd(*args[:4], chunks, args[4], c=c, d_state_out=args[6],
                                    return_d_state=True), T)


def test_d_lam_is_the_sum_of_dr_for_any_negative_lam():
    """Below lam = -20 the factor is one, and d_lam = sum u = sum dr / (1 - s): float32 sums of 80
    terms (1e-5 of the terms' sizes), whatever softplus(lam) has been rounded to."""
    x, r, i, lam, dh, S0, dS = make(2, 40, 64, seed=1)
    lam[:] = torch.linspace(-103.0, -20.0, 64)
    args = cuda(x, r, i, lam, dh, S0, dS)
    for c in (8.0, 1e20, 1e38):
        h, chunks = ops.glr_fwd(*args[:4], c=c, state_in=args[5], return_chunks=True)
        _, dr, _, d_lam = ops.glr_bwd(*args[:4], chunks, args[4], c=c)
        u = W.to_f64(dr) * (1 + np.exp(W.to_f64(r)))
        err = np.abs(W.to_f64(d_lam) - u.sum(axis=(0, 1)))
        size = np.abs(u).sum(axis=(0, 1))
        assert np.all(err <= 1e-5 * size + 1e-36), (c, (err / (size + 1e-36)).max())
        assert c < 1e38 or np.all(size[W.to_f64(lam) < -88.7] > 1e-5)

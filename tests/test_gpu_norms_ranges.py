"""The norms' gradients at the most tokens a call takes."""

import pytest
import torch

from linear_recurrent_sequence_retention_b200 import ops

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _pattern(n, *shape):
    """n rows of bf16, the same 4099 over and over."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rows = torch.randn(4099, *shape, generator=gen, device="cuda").bfloat16()
    out = torch.empty(n, *shape, dtype=torch.bfloat16, device="cuda")
    whole = n // 4099 * 4099
    out[:whole].view(-1, 4099, *shape).copy_(rows)
    out[whole:].copy_(rows[:n - whole])
    return out, rows


def test_layer_norm_gradients_of_the_most_tokens():
    """2^31 - 1 rows of three channels: every row's dx has the bits of a short call's."""
    x, rows = _pattern(MOST, 3)
    dy = torch.ones_like(x)
    y, mean, rstd = ops.layer_norm_fwd(rows, return_stats=True)
    want = ops.layer_norm_bwd(rows, torch.ones_like(rows), mean, rstd, return_d_affine=False)
    whole = MOST // 4099 * 4099
    mean, rstd = (torch.cat([t.repeat(whole // 4099), t[:MOST - whole]]) for t in (mean, rstd))
    dx, _, db = ops.layer_norm_bwd(x, dy, mean, rstd)
    assert (db / MOST - 1).abs().max() <= 1e-5
    for first in (0, 4099 * 1000, whole - 4099):
        assert torch.equal(dx[first:first + 4099], want)
    assert torch.equal(dx[whole:], want[:MOST - whole])
    only = ops.layer_norm_bwd(x, dy, mean, rstd, return_d_affine=False)
    assert torch.equal(only[whole - 4099:whole], want) and torch.equal(only[whole:], want[:MOST - whole])


def test_norm_gate_gradients_of_the_most_tokens():
    """2^31 - 1 rows of eight channels (34 GB a tensor; o, g and d_y are one)."""
    o, rows = _pattern(MOST, 1, 8)
    want = ops.norm_gate_bwd(rows, rows, rows, return_d_affine=False)
    got = ops.norm_gate_bwd(o, o, o, return_d_affine=False)
    whole = MOST // 4099 * 4099
    for g, w in zip(got, want):
        for first in (0, 4099 * 1000, whole - 4099):
            assert torch.equal(g[first:first + 4099], w)
        assert torch.equal(g[whole:], w[:MOST - whole])

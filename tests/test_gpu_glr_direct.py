"""The gated recurrence where a thread walks a sequence alone: up to 32 tokens per sequence (packed:
16 on average), in batches of 8 tokens, with a stored state every 64.  Lengths around the batches, and
packed lists whose average is short while one sequence crosses batches and stored states.  Against
the fp64 oracle, with the tolerances of test_gpu_glr.py."""

import numpy as np
import pytest
import torch

from linear_recurrent_sequence_retention_b200 import ops, workloads as W
from tests.test_gpu_glr import Reference, cuda, make

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")]


def _run(x, r, i, lam, dh, S0, dS, T, out, cu=None):
    ref = Reference(x, r, i, lam, dh, S0, dS, cu)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    cud = None if cu is None else torch.from_numpy(cu).cuda()
    td = W.torch_dtype(out)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, cu_seqlens=cud, state_in=S0d, return_state=True,
                               return_chunks=True, out_dtype=td)
    ref.check_forward(h, S, T, chunks, cu)
    ref.check_gradients(ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, cu_seqlens=cud, d_state_out=dSd,
                                    return_d_state=True, grad_dtype=td), T)
    ops.check_device_error()


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("T", [7, 8, 9, 15, 16, 17, 24, 25, 31, 32])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 34), (2, 257), (2, 600)])
def test_lengths_around_the_batches(dtype, out, T, B, D):
    x, r, i, lam, dh, S0, dS = make(B, T, D, dtype, seed=T + D)
    if T % 2:
        S0 = dS = None
    _run(x, r, i, lam, dh, S0, dS, T, out)


SKEWED = [[200] + [0] * 20, [0] * 10 + [129] + [1] * 10, [1] * 12 + [64] + [1] * 3, [65] + [2, 0] * 4,
          [9, 8, 7, 17, 16, 0, 33, 1], [5] * 3 + [136, 72] + [1] * 10 + [0] * 3]


@pytest.mark.parametrize("lens", SKEWED, ids=lambda l: f"{len(l)}seq{max(l)}")
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("D", [33, 70])
def test_one_long_sequence_among_short_ones(lens, dtype, out, D):
    assert sum(lens) <= 16 * len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x, r, i, lam, dh, S0, dS = make(1, T, D, dtype, nstate=len(lens), seed=len(lens) + D)
    _run(x, r, i, lam, dh, S0, dS, T, out, cu)

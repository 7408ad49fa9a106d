"""Calls from several host threads at once, each on its own stream."""

import threading

import pytest
import torch

from linear_recurrent_sequence_retention_b200 import ops

pytestmark = pytest.mark.gpu


def in_threads(jobs):
    """Runs the jobs at the same time, each in a thread of its own with a stream of its own."""
    start, errors = threading.Barrier(len(jobs)), []

    def work(job):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            job(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))
    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recurrence_of_two_cluster_sizes(dtype):
    """One kernel at two cluster sizes, whose shared memory differs: 64 tokens (one CTA) and 2048
    (a cluster).  The threads call the library itself, which holds no lock, as often as they can."""
    D = 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    lam = torch.full((D,), -4.0, device="cuda")
    L, p = ops.lib(), lambda t: t.data_ptr()
    code = ops._dt(torch.empty(0, dtype=dtype))
    jobs, checks = [], []
    for T in (64, 2048):
        x, r, i, dh = (torch.randn(1, T, D, generator=gen, device="cuda").to(dtype) for _ in range(4))
        want_h, chunks = ops.glr_fwd(x, r, i, lam, return_chunks=True)
        want = (want_h,) + ops.glr_bwd(x, r, i, lam, chunks, dh)
        out = [torch.empty_like(t) for t in want]
        ws = torch.empty(ops.glr_bwd_workspace_size(1, T, D), dtype=torch.uint8, device="cuda")

        def job(stream, x=x, r=r, i=i, dh=dh, chunks=chunks, out=out, ws=ws, T=T):
            fwd = (p(x), p(r), p(i), code, p(lam), 8.0, None, 0, None, None, p(out[0]), code, None,
                   1, T, D, stream.cuda_stream)
            bwd = (p(x), p(r), p(i), code, p(lam), 8.0, None, 0, p(chunks), p(dh), code, None,
                   p(out[1]), p(out[2]), p(out[3]), code, p(out[4]), None, p(ws), ws.numel(),
                   1, T, D, stream.cuda_stream)
            for n in range(4000):
                st = L.retention_glr_fwd(*fwd) or L.retention_glr_bwd(*bwd)
                assert st == ops.RET_OK, f"{T} tokens, call {n}: {ops.status_string(st)}"
        jobs.append(job)
        checks.append((out, want))
    torch.cuda.synchronize()
    in_threads(jobs)
    for out, want in checks:
        assert all(torch.equal(a, b) for a, b in zip(out, want))

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


def _retention_jobs(kind, small):
    """A job that repeats a call of one kernel at small or large head dimensions, and a check of its
    last results."""
    L, p = ops.lib(), lambda t: t.data_ptr()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    dt = torch.bfloat16 if kind == "steps_tc" else torch.float32
    code = ops._dt(torch.empty(0, dtype=dt))
    H, gam = 1, ops._gammas([0.9], 1)

    def rand(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)
    if kind in ("chunkwise", "parallel", "backward"):
        d, B, T = (16 if small else 256), 1, 32
        q, k, v = (rand(B, T, H, d) for _ in range(3))
        if kind == "parallel":
            want = (ops.parallel_fwd(q, k, v, [0.9]),)
            out = [torch.empty_like(t) for t in want]
            args = (p(q), p(k), p(v), code, gam, p(out[0]), code, None, 0, B, T, H, d, d)
            call = L.retention_parallel_fwd
        elif kind == "chunkwise":
            want = (ops.chunkwise_fwd(q, k, v, [0.9], 16),)
            out = [torch.empty_like(t) for t in want]
            ws = torch.empty(ops.chunkwise_workspace_size(dt, 16, B, T, H, d, d), dtype=torch.uint8, device="cuda")
            args = (p(q), p(k), p(v), code, gam, 16, None, 0, None, None, p(out[0]), code, None, p(ws), ws.numel(),
                    B, T, H, d, d)
            call = L.retention_chunkwise_fwd
        else:
            do = rand(B, T, H, d)
            want = ops.chunkwise_bwd(q, k, v, do, [0.9], 16)
            out = [torch.empty_like(t) for t in want]
            ws = torch.empty(ops.chunkwise_bwd_workspace_size(dt, 16, B, T, H, d, d), dtype=torch.uint8,
                             device="cuda")
            args = (p(q), p(k), p(v), p(do), code, gam, 16, None, 0, None, None, *[p(t) for t in out], None, p(ws),
                    ws.numel(), B, T, H, d, d)
            call = L.retention_chunkwise_bwd
    else:
        N, Tn = 1, 16
        dk = (128 if small else 256) if kind == "steps_tc" else (16 if small else 512)
        dv = 128
        q, k, v = (rand(N, Tn, H, n) for n in (dk, dk, dv))
        # gamma and the state zero: every call of a run gives the same
        gam = ops._gammas([0.0], 1)
        S = torch.zeros(N, H, dk, dv, device="cuda")
        if kind == "step":
            q, k, v = (t[:, 0].contiguous() for t in (q, k, v))
            want = (ops.recurrent_step(q, k, v, [0.0], S.clone(), out_dtype=dt),)
            out = [torch.empty_like(t) for t in want]
            args = (p(q), p(k), p(v), code, gam, p(S), p(out[0]), code, N, H, dk, dv)
            call = L.retention_recurrent_step
        else:
            want = (ops.recurrent_steps(q, k, v, [0.0], S.clone(), out_dtype=dt),)
            out = [torch.empty_like(t) for t in want]
            args = (p(q), p(k), p(v), code, gam, p(S), p(out[0]), code, N, Tn, H, dk, dv)
            call = L.retention_recurrent_steps
    held = [t for t in locals().values() if isinstance(t, torch.Tensor)]

    def job(stream, held=held):
        for n in range(4000):
            st = call(*args, stream.cuda_stream)
            assert st == ops.RET_OK, f"{kind}, {'small' if small else 'large'}, call {n}: {ops.status_string(st)}"
    return job, out, want


@pytest.mark.parametrize("kind", ["parallel", "chunkwise", "backward", "step", "steps", "steps_tc"])
def test_retention_of_two_head_sizes(kind):
    """One kernel with the shared memory of its small and of its large heads."""
    runs = [_retention_jobs(kind, small) for small in (True, False)]
    torch.cuda.synchronize()
    in_threads([job for job, _, _ in runs])
    for _, out, want in runs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))

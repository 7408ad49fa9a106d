"""Host-only checks of the gated linear recurrence, layer norm and norm-gradient
entry points: size queries, and bad arguments refused before the GPU is touched."""

import ctypes

import pytest
import torch

from tests.test_abi_host import FAKE, FAKE_WS, MISALIGNED, _lib

INF, NAN = float("inf"), float("nan")


def test_glr_sizes():
    ops, L = _lib()
    assert ops.GLR_CHUNK == 64
    # one row per 64 flat tokens, and one more per sequence
    assert ops.glr_chunk_slots(2, 100) == 200 // 64 + 2
    assert ops.glr_chunk_slots(1, 1000, nseq=7) == 1000 // 64 + 7
    assert ops.glr_chunk_slots(1, 0, nseq=3) == 3
    assert ops.glr_chunk_slots(0, 10) == 0 and ops.glr_chunk_slots(2, 10, nseq=3) == 0
    assert ops.glr_chunk_slots(1 << 16, 1 << 15) == 0            # 2^31 tokens
    assert ops.glr_chunk_slots(1, (1 << 31) - 2048) == 0          # indexes past the last round
    assert ops.glr_chunk_slots(1, (1 << 31) - 2049) > 0
    need = ops.glr_bwd_workspace_size(2, 8192, 4096)
    assert need > 0 and need % 256 == 0
    assert ops.glr_bwd_workspace_size(2, 8192, 0) == 0
    assert ops.glr_bwd_workspace_size(2, 8192, (1 << 20) + 1) == 0


def test_chunk_rows_of_packed_sequences_do_not_overlap():
    """Rows floor(start/64) + s and on: disjoint, and inside the slots of the size query."""
    import random
    ops, _ = _lib()
    rng = random.Random(0)
    for _ in range(300):
        lens = [rng.choice([0, 1, 63, 64, 65, rng.randrange(400)]) for _ in range(rng.randint(1, 12))]
        start, end, total = 0, 0, sum(lens)
        for s, n in enumerate(lens):
            row = start // 64 + s
            assert row >= end
            end = row + (n + 63) // 64
            start += n
        assert end <= ops.glr_chunk_slots(1, total, nseq=len(lens))


def test_glr_fwd_rejects_bad_arguments():
    ops, L = _lib()

    def call(x=FAKE, r=FAKE, lam=FAKE, c=8.0, cu=None, nseq=0, h=FAKE, h_t=0, t=1, B=1, T=8, D=16,
             S0=None, chunks=None):
        return L.retention_glr_fwd(x, r, FAKE, t, lam, c, cu, nseq, S0, None, h, h_t, chunks, B, T,
                                   D, None)
    bad = ops.RET_ERR_INVALID_ARG
    assert call(x=None) == bad and call(lam=None) == bad and call(h=None) == bad
    assert call(r=MISALIGNED) == bad and call(S0=MISALIGNED) == bad and call(chunks=MISALIGNED) == bad
    for c in (0.0, -1.0, INF, NAN, 1e300):
        assert call(c=c) == bad
    assert call(t=2) == bad and call(h_t=-1) == bad
    assert call(B=0) == bad and call(T=0) == bad and call(D=0) == bad
    assert call(cu=FAKE) == bad and call(nseq=3) == bad and call(cu=FAKE, nseq=3, B=2) == bad
    assert call(B=1 << 16, T=1 << 15) == bad
    assert call(D=(1 << 20) + 1) == ops.RET_ERR_UNSUPPORTED


def test_glr_bwd_rejects_bad_arguments():
    ops, L = _lib()
    need = ops.glr_bwd_workspace_size(1, 8, 16)

    def call(x=FAKE, chunks=FAKE, dh=FAKE, dx=FAKE, dlam=FAKE, g_t=0, c=8.0, ws=FAKE_WS, nb=need,
             T=8, D=16, cu=None, nseq=0):
        return L.retention_glr_bwd(x, FAKE, FAKE, 1, FAKE, c, cu, nseq, chunks, dh, 0, None, dx,
                                   FAKE, FAKE, g_t, dlam, None, ws, nb, 1, T, D, None)
    bad = ops.RET_ERR_INVALID_ARG
    assert call(x=None) == bad and call(chunks=None) == bad and call(dh=None) == bad
    assert call(dx=None) == bad and call(dlam=None) == bad and call(dx=MISALIGNED) == bad
    assert call(g_t=5) == bad and call(c=0.0) == bad and call(T=0) == bad and call(nseq=1) == bad
    assert call(D=(1 << 20) + 1) == ops.RET_ERR_UNSUPPORTED
    assert call(ws=None) == ops.RET_ERR_WORKSPACE and call(nb=need - 1) == ops.RET_ERR_WORKSPACE
    assert call(ws=FAKE_WS + 16) == ops.RET_ERR_WORKSPACE


def test_glr_step_rejects_bad_arguments():
    ops, L = _lib()

    def call(x=FAKE, state=FAKE, out=FAKE, h=FAKE, c=8.0, N=4, D=16):
        return L.retention_glr_step(x, FAKE, FAKE, 1, FAKE, c, state, out, h, 0, N, D, None)
    bad = ops.RET_ERR_INVALID_ARG
    assert call(x=None) == bad and call(state=None) == bad and call(out=None) == bad
    assert call(h=MISALIGNED) == bad and call(N=0) == bad and call(D=0) == bad and call(c=NAN) == bad
    assert call(D=(1 << 20) + 1) == ops.RET_ERR_UNSUPPORTED


def test_layer_norm_rejects_bad_arguments():
    ops, L = _lib()

    def fwd(x=FAKE, w=None, y=FAKE, eps=1e-5, n=4, D=16, t=0, mean=None):
        return L.retention_layer_norm_fwd(x, t, w, None, eps, y, 0, mean, None, n, D, None)
    bad = ops.RET_ERR_INVALID_ARG
    assert fwd(x=None) == bad and fwd(y=None) == bad and fwd(w=MISALIGNED) == bad
    assert fwd(eps=-1.0) == bad and fwd(eps=NAN) == bad and fwd(eps=INF) == bad
    assert fwd(n=-1) == bad and fwd(D=0) == bad and fwd(t=3) == bad and fwd(mean=MISALIGNED) == bad
    assert fwd(D=16385) == ops.RET_ERR_UNSUPPORTED
    assert fwd(n=0, x=None, y=None) == ops.RET_OK          # nothing to do

    need = ops.layer_norm_bwd_workspace_size(4096, 1024)
    assert ops.layer_norm_bwd_workspace_size(-1, 16) == 0
    assert ops.layer_norm_bwd_workspace_size(4, 16385) == 0

    def bwd(x=FAKE, dy=FAKE, mean=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE_WS, nb=need, n=4096,
            D=1024):
        return L.retention_layer_norm_bwd(x, 0, dy, 0, mean, FAKE, None, dx, 0, dw, db, ws, nb, n,
                                          D, None)
    assert bwd(x=None) == bad and bwd(dy=None) == bad and bwd(mean=None) == bad
    assert bwd(dx=MISALIGNED) == bad and bwd(dw=None) == bad and bwd(db=None) == bad
    assert bwd(D=16385) == ops.RET_ERR_UNSUPPORTED
    if need:
        assert bwd(ws=None) == ops.RET_ERR_WORKSPACE
        assert bwd(nb=need - 1) == ops.RET_ERR_WORKSPACE
        assert bwd(ws=FAKE_WS + 16) == ops.RET_ERR_WORKSPACE


def test_norm_gate_bwd_rejects_bad_arguments():
    ops, L = _lib()
    need = ops.norm_gate_bwd_workspace_size(2048, 2, 256)
    assert ops.norm_gate_bwd_workspace_size(4, 2, 1025) == 0
    assert ops.norm_gate_bwd_workspace_size(4, 2048, 1024) == 0

    def call(o=FAKE, g=0x10000, g_t=1, w=None, eps=1e-5, dy=FAKE, d_o=FAKE, dw=FAKE, db=FAKE,
             ws=FAKE_WS, nb=need, n=2048, H=2, dv=256, t=1):
        ng = ops.NormGate(g, g_t, w, None, eps)
        return L.msr_norm_gate_bwd(o, t, ctypes.byref(ng), dy, d_o, FAKE, 1, dw, db, ws, nb, n, H,
                                   dv, None)
    bad = ops.RET_ERR_INVALID_ARG
    assert call(o=None) == bad and call(g=None) == bad and call(dy=None) == bad
    assert call(d_o=None) == bad and call(d_o=MISALIGNED) == bad and call(w=0x10004) == bad
    assert call(g_t=4) == bad and call(t=4) == bad and call(eps=-1.0) == bad and call(eps=NAN) == bad
    assert call(dw=None) == bad and call(db=None) == bad and call(n=-1) == bad and call(H=0) == bad
    assert call(dv=1025) == ops.RET_ERR_UNSUPPORTED
    assert call(H=2048, dv=1024) == ops.RET_ERR_UNSUPPORTED
    assert L.msr_norm_gate_bwd(FAKE, 1, None, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE_WS, need, 4, 2,
                               256, None) == bad
    if need:
        assert call(ws=None) == ops.RET_ERR_WORKSPACE
        assert call(nb=need - 1) == ops.RET_ERR_WORKSPACE
        assert call(ws=FAKE_WS + 16) == ops.RET_ERR_WORKSPACE


def test_binding_refuses_host_tensors():
    ops, _ = _lib()
    x = torch.zeros(1, 4, 8)
    lam = torch.zeros(8)
    for f in (lambda: ops.glr_fwd(x, x, x, lam), lambda: ops.glr_step(x[0], x[0], x[0], lam, x[0]),
              lambda: ops.glr_bwd(x, x, x, lam, x[0], x), lambda: ops.layer_norm_fwd(x),
              lambda: ops.layer_norm_bwd(x, x, x[..., 0], x[..., 0]),
              lambda: ops.norm_gate_bwd(x, x, x)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        ops.layer_norm_fwd([1.0])


class _Elsewhere(torch.Tensor):
    """Stands in for a tensor on a device that is not the current one."""

    device = torch.device("cuda:7")

    def get_device(self):
        return 7


class _Here(_Elsewhere):
    def get_device(self):
        return 0


def test_binding_refuses_another_device(monkeypatch):
    ops, _ = _lib()
    monkeypatch.setattr(ops, "_dev", lambda t, name: t)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="x is on cuda:7, the current device is cuda:0"):
        ops._ready(None, x=_Elsewhere())
    with pytest.raises(ValueError, match="y is on cuda:7, the current device is cuda:0"):
        ops._ready(None, x=_Here(), y=_Elsewhere())
    with pytest.raises(ValueError, match="stream is on cuda:7"):
        ops._ready(_Elsewhere(), x=_Here())

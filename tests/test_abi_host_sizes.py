"""Host-only checks of sizes at the ends of their ranges: the library's queries, and what the binding
lets through to them."""

import pytest
import torch

from tests.test_abi_host import _lib

MOST = (1 << 31) - 1


@pytest.mark.parametrize("D", [1, 2, 37, 96, 256, 257, 1001, 1024, 4096, 8192, 16384])
def test_layer_norm_gradients_of_the_most_tokens(D):
    """A partial row per block and weight: as many at any number of tokens that fills the GPU."""
    ops, _ = _lib()
    want = ops.layer_norm_bwd_workspace_size(1 << 24, D)
    assert 0 < want <= 2 * 148 * 4 * D * 4 + 256
    for n in (MOST, MOST - 1, MOST - 6, MOST - 7, MOST - 8, 1 << 30):
        assert ops.layer_norm_bwd_workspace_size(n, D) == want, n


WIDE = (1 << 32) + 4                    # its low 32 bits are 4


def test_size_queries_refuse_what_a_c_int_does_not_hold():
    ops, _ = _lib()
    assert ops.layer_norm_bwd_workspace_size(4, 8) > 0 and ops.norm_gate_bwd_workspace_size(4, 4, 8) > 0
    assert ops.glr_chunk_slots(4, 4) > 0 and ops.glr_bwd_workspace_size(4, 4, 4) > 0
    for n in (WIDE, -WIDE, 1 << 31, (1 << 31) + 8, 1 << 64):
        assert ops.layer_norm_bwd_workspace_size(n, 8) == 0 == ops.layer_norm_bwd_workspace_size(4, n)
        assert ops.glr_chunk_slots(n, 4) == 0 == ops.glr_chunk_slots(1, n) == ops.glr_chunk_slots(1, 4, n)
        for k in range(4):
            assert ops.glr_bwd_workspace_size(*[n if j == k else (0 if j == 3 else 4) for j in range(4)]) == 0
        for k in range(3):
            assert ops.norm_gate_bwd_workspace_size(*[n if j == k else 4 for j in range(3)]) == 0


class _Recorder:
    """Stands in for the library: every call succeeds and is written down."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _check_call(monkeypatch, call, small):
    """The call with WIDE rows is refused before the library is asked to compute; with few it passes."""
    ops, _ = _lib()
    fake = _Recorder()
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "status_string", lambda status: str(status))
    monkeypatch.setattr(ops, "_ready", lambda stream, **tensors: 0)
    with pytest.raises(ops.RetentionError) as info:
        call(ops, WIDE)
    assert info.value.status == ops.RET_ERR_INVALID_ARG
    assert not [c for c in fake.calls if not c.endswith(("size", "slots"))]
    call(ops, small)
    assert [c for c in fake.calls if not c.endswith(("size", "slots"))]


def _glr(n, packed=False):
    x = _meta(1, n, 2) if packed else _meta(n, 1, 2)
    return x, x, x, _meta(2, dtype=torch.float32)


NEW_CALLS = {
    "glr_fwd_batch": lambda ops, n: ops.glr_fwd(*_glr(n)),
    "glr_fwd_tokens": lambda ops, n: ops.glr_fwd(*_glr(n, True)),
    "glr_fwd_sequences": lambda ops, n: ops.glr_fwd(*_glr(4, True), cu_seqlens=_meta(n + 1, dtype=torch.int32)),
    "glr_bwd": lambda ops, n: ops.glr_bwd(*_glr(n), _meta(0, 2, dtype=torch.float32), _meta(n, 1, 2)),
    "glr_step": lambda ops, n: ops.glr_step(*[_meta(n, 2)] * 3, _meta(2, dtype=torch.float32),
                                            _meta(n, 2, dtype=torch.float32)),
    "layer_norm_fwd": lambda ops, n: ops.layer_norm_fwd(_meta(n // 2, 2, 2)),
    "layer_norm_bwd": lambda ops, n: ops.layer_norm_bwd(_meta(n, 2), _meta(n, 2), _meta(n, dtype=torch.float32),
                                                        _meta(n, dtype=torch.float32)),
    "norm_gate_bwd": lambda ops, n: ops.norm_gate_bwd(_meta(n, 1, 2), _meta(n, 2), _meta(n, 1, 2)),
}


@pytest.mark.parametrize("name", NEW_CALLS)
def test_calls_refuse_more_rows_than_a_c_int_holds(monkeypatch, name):
    _check_call(monkeypatch, NEW_CALLS[name], 4)

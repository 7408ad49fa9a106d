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
        return lambda *args: self.calls.append(name) or (256 if name.endswith("size") else 0)


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


def _gam(h):
    return [0.5] * h


def _qkv(n, axis, dtype=torch.bfloat16):
    shape = [n if axis == k else 1 for k in range(3)] + [2]
    return [_meta(*shape, dtype=dtype) for _ in range(3)]


OLDER_CALLS = {
    "parallel_fwd": lambda ops, n: ops.parallel_fwd(*_qkv(n, 1), _gam(1)),
    "chunkwise_fwd": lambda ops, n: ops.chunkwise_fwd(*_qkv(n, 0), _gam(1), 128),
    "chunkwise_fwd_chunk": lambda ops, n: ops.chunkwise_fwd(*_qkv(4, 1), _gam(1), n),
    "chunkwise_states": lambda ops, n: ops.chunkwise_states(*_qkv(n, 1)[:2], _gam(1), 128),
    "chunkwise_outputs": lambda ops, n: ops.chunkwise_outputs(*_qkv(n, 1), _gam(1), 128, _meta(256)),
    "chunkwise_fwd_static_ws": lambda ops, n: ops.chunkwise_fwd_static_ws(*_qkv(n, 1), _gam(1), 128),
    "chunkwise_bwd": lambda ops, n: ops.chunkwise_bwd(*_qkv(n, 1), _qkv(n, 1)[0], _gam(1), 128),
    "rope": lambda ops, n: ops.rope(*_qkv(n, 1)[:2]),
    "rla_fwd": lambda ops, n: ops.rla_fwd(*_qkv(n, 1), 8),
    "recurrent_step": lambda ops, n: ops.recurrent_step(
        *[_meta(n, 1, 2)] * 3, _gam(1), _meta(n, 1, 2, 2, dtype=torch.float32)),
    "recurrent_steps": lambda ops, n: ops.recurrent_steps(
        *[_meta(n, 1, 1, 2)] * 3, _gam(1), _meta(n, 1, 2, 2, dtype=torch.float32)),
    "norm_gate": lambda ops, n: ops.norm_gate(_meta(n, 1, 2), _meta(n, 2)),
}


@pytest.mark.parametrize("name", OLDER_CALLS)
def test_retention_calls_refuse_more_rows_than_a_c_int_holds(monkeypatch, name):
    ops, _ = _lib()
    monkeypatch.setattr(ops, "_dev", lambda t, name: t)
    monkeypatch.setattr(ops, "_stream", lambda stream: None)
    _check_call(monkeypatch, OLDER_CALLS[name], 4)


def test_retention_size_queries_refuse_what_a_c_int_does_not_hold():
    ops, _ = _lib()
    bf = torch.bfloat16
    sizes = [4, 128, 2, 128, 128]
    assert ops.parallel_workspace_size(bf, *sizes) > 0
    for query in (ops.chunkwise_workspace_size, ops.chunkwise_bwd_workspace_size):
        assert query(bf, 128, *sizes) > 0
    assert ops.chunkwise_fwd_rope_workspace_size(128, *sizes) > 0
    assert ops.chunkwise_executed_chunk(bf, 128, 128, 128) > 0
    low = 1 << 32
    for k in range(5):
        wide = [v + low if j == k else v for j, v in enumerate(sizes)]
        assert ops.parallel_workspace_size(bf, *wide) == 0
        assert ops.chunkwise_workspace_size(bf, 128, *wide) == 0
        assert ops.chunkwise_bwd_workspace_size(bf, 128, *wide) == 0
        assert ops.chunkwise_fwd_rope_workspace_size(128, *wide) == 0
    assert ops.chunkwise_workspace_size(bf, 128 + low, *sizes) == 0
    assert ops.chunkwise_executed_chunk(bf, 128 + low, 128, 128) == 0

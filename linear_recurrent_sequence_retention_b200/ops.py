"""Thin ctypes binding of libretention.so (C ABI in include/retention.h).

Argument marshalling only: every function checks the torch tensors it is
given, passes their device pointers, sizes and the current CUDA stream to the
C entry point of the same name, and raises :class:`RetentionError` on a
non-OK status.  All arithmetic happens in the library's CUDA kernels; there
is no CPU or PyTorch fallback, and calling any function without the built
library raises immediately.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libretention.so")
_IN_TREE_LIBRARY = LIBRARY_PATH

RET_OK = 0
RET_ERR_INVALID_ARG = 1
RET_ERR_UNSUPPORTED = 2
RET_ERR_CUDA = 3
RET_ERR_TIMEOUT = 4
RET_ERR_WORKSPACE = 5
RET_ERR_DEVICE_DATA = 6
RET_ERR_RANGE = 7

RET_F32 = 0
RET_BF16 = 1

# Capacity of the library's built-in scratch (RETENTION_STATIC_WORKSPACE_BYTES).
STATIC_WORKSPACE_BYTES = 32 << 20

# Tokens between two stored states of the gated linear recurrence (RETENTION_GLR_CHUNK).
GLR_CHUNK = 64

EXPORTED = (
    "retention_abi_version",
    "retention_source_sha",
    "retention_status_string",
    "retention_parallel_workspace_size",
    "retention_parallel_fwd",
    "retention_chunkwise_workspace_size",
    "retention_chunkwise_executed_chunk",
    "retention_chunkwise_fwd",
    "retention_chunkwise_states",
    "retention_chunkwise_outputs",
    "retention_chunkwise_fwd_static_ws",
    "retention_chunkwise_fwd_rope_workspace_size",
    "retention_chunkwise_fwd_rope",
    "retention_chunkwise_bwd_workspace_size",
    "retention_chunkwise_bwd",
    "retention_rope",
    "retention_rla_workspace_size",
    "retention_rla_fwd",
    "retention_recurrent_step",
    "retention_recurrent_steps",
    "msr_norm_gate",
    "retention_glr_chunk_slots",
    "retention_glr_fwd",
    "retention_glr_bwd_workspace_size",
    "retention_glr_bwd",
    "retention_glr_step",
    "retention_layer_norm_fwd",
    "retention_layer_norm_bwd_workspace_size",
    "retention_layer_norm_bwd",
    "msr_norm_gate_bwd_workspace_size",
    "msr_norm_gate_bwd",
    "retention_check_device_error",
    "retention_selftest_wait_timeout",
)


class RetentionError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class NormGate(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("g_dtype", ctypes.c_int),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


_lib = None


def _check_sources(L):
    """Refuse the in-tree library if it was built from sources other than the tree's."""
    if (os.path.abspath(LIBRARY_PATH) != _IN_TREE_LIBRARY
            or not os.path.isdir(os.path.join(_HERE, "csrc"))):
        return
    from . import build
    want, got = build.source_sha(), L.retention_source_sha().decode()
    if got != want:
        raise RuntimeError(
            f"{LIBRARY_PATH} was built from other sources (library {got[:12]}, tree "
            f"{want[:12]}): rebuild it with `python -m linear_recurrent_sequence_retention_b200.build`")


def lib():
    """The loaded library (loads it on first use; raises if it is not built or is stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise RuntimeError(
            f"{LIBRARY_PATH} is missing: build it with "
            "`python -m linear_recurrent_sequence_retention_b200.build` (needs nvcc)")
    L = ctypes.CDLL(LIBRARY_PATH)
    vp, ci, cd = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_double)
    L.retention_abi_version.restype = ci
    L.retention_abi_version.argtypes = []
    L.retention_source_sha.restype = ctypes.c_char_p
    L.retention_source_sha.argtypes = []
    _check_sources(L)
    L.retention_status_string.restype = ctypes.c_char_p
    L.retention_status_string.argtypes = [ci]
    L.retention_parallel_workspace_size.restype = ctypes.c_size_t
    L.retention_parallel_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci]
    L.retention_parallel_fwd.restype = ci
    L.retention_parallel_fwd.argtypes = [vp, vp, vp, ci, cd, vp, ci, vp, ctypes.c_size_t,
                                         ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_workspace_size.restype = ctypes.c_size_t
    L.retention_chunkwise_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci, ci]
    L.retention_chunkwise_executed_chunk.restype = ci
    L.retention_chunkwise_executed_chunk.argtypes = [ci, ci, ci, ci]
    L.retention_chunkwise_fwd.restype = ci
    L.retention_chunkwise_fwd.argtypes = [vp, vp, vp, ci, cd, ci, vp, ci, vp, vp, vp, ci,
                                          ctypes.POINTER(NormGate), vp, ctypes.c_size_t,
                                          ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_states.restype = ci
    L.retention_chunkwise_states.argtypes = [vp, vp, ci, cd, ci, vp, ci, vp, vp, vp,
                                             ctypes.c_size_t, ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_outputs.restype = ci
    L.retention_chunkwise_outputs.argtypes = [vp, vp, vp, ci, cd, ci, vp, ci, ci, vp, ci,
                                              ctypes.POINTER(NormGate), vp, ctypes.c_size_t,
                                              ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_fwd_static_ws.restype = ci
    L.retention_chunkwise_fwd_static_ws.argtypes = [vp, vp, vp, ci, cd, ci, vp, ci, vp, vp, vp,
                                                    ci, ctypes.POINTER(NormGate),
                                                    ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_fwd_rope_workspace_size.restype = ctypes.c_size_t
    L.retention_chunkwise_fwd_rope_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci]
    L.retention_chunkwise_fwd_rope.restype = ci
    L.retention_chunkwise_fwd_rope.argtypes = [vp, vp, vp, ci, cd, ci, vp, ci, vp, vp, vp, ci,
                                               ctypes.POINTER(NormGate), ctypes.c_double, vp,
                                               ctypes.c_size_t, ci, ci, ci, ci, ci, vp]
    L.retention_chunkwise_bwd_workspace_size.restype = ctypes.c_size_t
    L.retention_chunkwise_bwd_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci, ci]
    L.retention_chunkwise_bwd.restype = ci
    L.retention_chunkwise_bwd.argtypes = [vp, vp, vp, vp, ci, cd, ci, vp, ci, vp, vp,
                                          vp, vp, vp, vp, vp, ctypes.c_size_t,
                                          ci, ci, ci, ci, ci, vp]
    L.retention_rope.restype = ci
    L.retention_rope.argtypes = [vp, vp, ci, vp, vp, ctypes.c_double, vp, ci, ci, ci, ci, ci, vp]
    L.retention_rla_workspace_size.restype = ctypes.c_size_t
    L.retention_rla_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci]
    L.retention_rla_fwd.restype = ci
    L.retention_rla_fwd.argtypes = [vp, vp, vp, ci, ci, vp, ci, vp, ci, vp, ctypes.c_size_t,
                                    ci, ci, ci, ci, ci, vp]
    L.retention_recurrent_step.restype = ci
    L.retention_recurrent_step.argtypes = [vp, vp, vp, ci, cd, vp, vp, ci, ci, ci, ci, ci, vp]
    L.retention_recurrent_steps.restype = ci
    L.retention_recurrent_steps.argtypes = [vp, vp, vp, ci, cd, vp, vp, ci, ci, ci, ci, ci, ci, vp]
    L.msr_norm_gate.restype = ci
    L.msr_norm_gate.argtypes = [vp, ci, ctypes.POINTER(NormGate), vp, ci, ci, ci, ci, vp]
    cf, cs = ctypes.c_double, ctypes.c_size_t
    L.retention_glr_chunk_slots.restype = cs
    L.retention_glr_chunk_slots.argtypes = [ci, ci, ci]
    L.retention_glr_fwd.restype = ci
    L.retention_glr_fwd.argtypes = [vp, vp, vp, ci, vp, cf, vp, ci, vp, vp, vp, ci, vp,
                                    ci, ci, ci, vp]
    L.retention_glr_bwd_workspace_size.restype = cs
    L.retention_glr_bwd_workspace_size.argtypes = [ci, ci, ci, ci]
    L.retention_glr_bwd.restype = ci
    L.retention_glr_bwd.argtypes = [vp, vp, vp, ci, vp, cf, vp, ci, vp, vp, ci, vp, vp, vp, vp, ci,
                                    vp, vp, vp, cs, ci, ci, ci, vp]
    L.retention_glr_step.restype = ci
    L.retention_glr_step.argtypes = [vp, vp, vp, ci, vp, cf, vp, vp, vp, ci, ci, ci, vp]
    L.retention_layer_norm_fwd.restype = ci
    L.retention_layer_norm_fwd.argtypes = [vp, ci, vp, vp, cf, vp, ci, vp, vp, ci, ci, vp]
    L.retention_layer_norm_bwd_workspace_size.restype = cs
    L.retention_layer_norm_bwd_workspace_size.argtypes = [ci, ci]
    L.retention_layer_norm_bwd.restype = ci
    L.retention_layer_norm_bwd.argtypes = [vp, ci, vp, ci, vp, vp, vp, vp, ci, vp, vp, vp, cs,
                                           ci, ci, vp]
    L.msr_norm_gate_bwd_workspace_size.restype = cs
    L.msr_norm_gate_bwd_workspace_size.argtypes = [ci, ci, ci]
    L.msr_norm_gate_bwd.restype = ci
    L.msr_norm_gate_bwd.argtypes = [vp, ci, ctypes.POINTER(NormGate), vp, vp, vp, ci, vp, vp, vp,
                                    cs, ci, ci, ci, vp]
    L.retention_check_device_error.restype = ci
    L.retention_check_device_error.argtypes = [vp]
    L.retention_selftest_wait_timeout.restype = ci
    L.retention_selftest_wait_timeout.argtypes = [vp]
    _lib = L
    return L


def status_string(status):
    return lib().retention_status_string(int(status)).decode()


def _check(status, where):
    if status != RET_OK:
        raise RetentionError(status, where)


def _dt(t):
    if t.dtype == torch.float32:
        return RET_F32
    if t.dtype == torch.bfloat16:
        return RET_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _wide(sizes):
    """Whether one of the or-ed sizes is negative or past a C int, of which ctypes would pass the
    low 32 bits."""
    return sizes >> 31


def _too_large(where):
    return RetentionError(RET_ERR_INVALID_ARG, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _gammas(gamma, H):
    vals = [float(x) for x in (gamma.tolist() if hasattr(gamma, "tolist") else gamma)]
    if len(vals) != H:
        raise ValueError(f"gamma needs {H} entries, got {len(vals)}")
    return (ctypes.c_double * H)(*vals)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def abi_version():
    return lib().retention_abi_version()


def parallel_workspace_size(dtype, B, T, H, dk, dv):
    """Bytes of workspace the parallel form needs (0: none, the CUDA-core kernel)."""
    code = RET_F32 if dtype == torch.float32 else RET_BF16
    if _wide(B | T | H | dk | dv):
        return 0
    return int(lib().retention_parallel_workspace_size(code, B, T, H, dk, dv))


def parallel_fwd(q, k, v, gamma, out_dtype=None, out=None, workspace=None, stream=None):
    """Parallel form; q,k: [B,T,H,dk], v: [B,T,H,dv] -> o [B,T,H,dv].  bf16
    inputs of the tensor-core head dims use a workspace (allocated here when
    not given)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes/dtypes disagree")
    if _wide(B | T | H | dk | dv):
        raise _too_large("retention_parallel_fwd")
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    else:
        _dev(out, "out")
        if tuple(out.shape) != (B, T, H, dv):
            raise ValueError("out has the wrong shape")
    need = lib().retention_parallel_workspace_size(_dt(q), B, T, H, dk, dv)
    if need and workspace is None:
        workspace = alloc_workspace(need, q.device)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().retention_parallel_fwd(_ptr(q), _ptr(k), _ptr(v), _dt(q), _gammas(gamma, H),
                                      _ptr(out), _dt(out), _ptr(workspace), nbytes,
                                      B, T, H, dk, dv, _stream(stream))
    _check(st, "retention_parallel_fwd")
    return out


def chunkwise_workspace_size(dtype, chunk, B, T, H, dk, dv, nseq=0):
    code = RET_F32 if dtype == torch.float32 else RET_BF16
    if _wide(chunk | B | T | H | dk | dv | nseq):
        return 0
    return int(lib().retention_chunkwise_workspace_size(code, chunk, B, T, H, dk, dv, nseq))


def chunkwise_executed_chunk(dtype, chunk, dk, dv):
    """The chunk length the chunkwise kernels evaluate for ``chunk`` (0 if
    unsupported); every chunk length gives the same result."""
    code = RET_F32 if dtype == torch.float32 else RET_BF16
    if _wide(chunk | dk | dv):
        return 0
    return int(lib().retention_chunkwise_executed_chunk(code, chunk, dk, dv))


def alloc_workspace(nbytes, device):
    """A caller-owned workspace buffer (uint8, 256-byte aligned by the allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def chunkwise_fwd_rope_workspace_size(chunk, B, T, H, dk, dv, nseq=0):
    if _wide(chunk | B | T | H | dk | dv | nseq):
        return 0
    return lib().retention_chunkwise_fwd_rope_workspace_size(chunk, B, T, H, dk, dv, nseq)


def chunkwise_fwd(q, k, v, gamma, chunk, cu_seqlens=None, state_in=None, return_state=False,
                  g=None, gn_weight=None, gn_bias=None, eps=1e-5, out_dtype=None, out=None,
                  state_out=None, workspace=None, stream=None, rope_base=None):
    """Chunkwise form (+ optional fused GroupNorm and swish gate when ``g`` is given).

    q,k: [B,T,H,dk]; v: [B,T,H,dv]; packed sequences: B = 1 and ``cu_seqlens``
    an int32 CUDA tensor [nseq+1].  Returns ``out`` ([B,T,H,dv]: o, or y when
    gated) and, with ``return_state``, the final fp32 states.  With
    ``rope_base`` (bf16 inputs only) q and k are first given the rotary
    position encoding of :func:`rope` inside the same call
    (``retention_chunkwise_fwd_rope``); q and k themselves are not modified.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes/dtypes disagree")
    nseq = 0
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens")
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor")
        nseq = cu_seqlens.numel() - 1
        if nseq < 1:
            raise ValueError("cu_seqlens needs at least two entries")
    if _wide(max(int(chunk), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_chunkwise_fwd")
    nstate = nseq if nseq else B
    if state_in is not None:
        _dev(state_in, "state_in")
        if state_in.dtype != torch.float32 or tuple(state_in.shape) != (nstate, H, dk, dv):
            raise ValueError(f"state_in must be float32 [{nstate},{H},{dk},{dv}]")
    if return_state and state_out is None:
        state_out = torch.empty(nstate, H, dk, dv, device=q.device, dtype=torch.float32)
    if state_out is not None:
        _dev(state_out, "state_out")
        if state_out.dtype != torch.float32 or tuple(state_out.shape) != (nstate, H, dk, dv):
            raise ValueError(f"state_out must be float32 [{nstate},{H},{dk},{dv}]")
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    else:
        _dev(out, "out")
        if tuple(out.shape) != (B, T, H, dv):
            raise ValueError("out has the wrong shape")
    ng = None
    keep = []
    if g is not None:
        _dev(g, "g")
        if g.numel() != B * T * H * dv:
            raise ValueError("g must hold B*T*H*dv elements")
        for t, n in ((gn_weight, "gn_weight"), (gn_bias, "gn_bias")):
            if t is not None:
                _dev(t, n)
                if t.dtype != torch.float32 or t.numel() != H * dv:
                    raise ValueError(f"{n} must be float32 with H*dv elements")
        ng = NormGate(g.data_ptr(), _dt(g), gn_weight.data_ptr() if gn_weight is not None else None,
                      gn_bias.data_ptr() if gn_bias is not None else None, float(eps))
        keep.append(ng)
    if rope_base is not None:
        if _dt(q) != RET_BF16:
            raise RetentionError(RET_ERR_UNSUPPORTED, "retention_chunkwise_fwd_rope")
        need = lib().retention_chunkwise_fwd_rope_workspace_size(chunk, B, T, H, dk, dv, nseq)
        where = "retention_chunkwise_fwd_rope_workspace_size"
    else:
        need = lib().retention_chunkwise_workspace_size(_dt(q), chunk, B, T, H, dk, dv, nseq)
        where = "retention_chunkwise_workspace_size"
    if need == 0:
        st = RET_ERR_UNSUPPORTED if _dt(q) == RET_BF16 else RET_ERR_INVALID_ARG
        raise RetentionError(st, where)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    head = (_ptr(q), _ptr(k), _ptr(v), _dt(q), _gammas(gamma, H), int(chunk),
            _ptr(cu_seqlens), nseq, _ptr(state_in), _ptr(state_out), _ptr(out), _dt(out),
            ctypes.byref(ng) if ng is not None else None)
    tail = (_ptr(workspace), workspace.numel() * workspace.element_size(), B, T, H, dk, dv,
            _stream(stream))
    if rope_base is not None:
        st = lib().retention_chunkwise_fwd_rope(*head, float(rope_base), *tail)
        _check(st, "retention_chunkwise_fwd_rope")
    else:
        st = lib().retention_chunkwise_fwd(*head, *tail)
        _check(st, "retention_chunkwise_fwd")
    return (out, state_out) if return_state else out


def chunkwise_states(k, v, gamma, chunk, cu_seqlens=None, state_in=None, state_out=None,
                     workspace=None, stream=None):
    """State phase only: per-chunk states into ``workspace`` (returned) and the
    final states into ``state_out`` (optional, float32 [nseq|B,H,dk,dv])."""
    for t, n in ((k, "k"), (v, "v")):
        _dev(t, n)
    B, T, H, dk = k.shape
    dv = v.shape[3]
    nseq = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens")
    if _wide(max(int(chunk), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_chunkwise_states")
    need = lib().retention_chunkwise_workspace_size(_dt(k), chunk, B, T, H, dk, dv, nseq)
    if need == 0:
        raise RetentionError(RET_ERR_UNSUPPORTED if _dt(k) == RET_BF16 else RET_ERR_INVALID_ARG,
                             "retention_chunkwise_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, k.device)
    for t, n in ((state_in, "state_in"), (state_out, "state_out")):
        if t is not None:
            _dev(t, n)
    st = lib().retention_chunkwise_states(
        _ptr(k), _ptr(v), _dt(k), _gammas(gamma, H), int(chunk), _ptr(cu_seqlens), nseq,
        _ptr(state_in), _ptr(state_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), B, T, H, dk, dv, _stream(stream))
    _check(st, "retention_chunkwise_states")
    return workspace


def chunkwise_outputs(q, k, v, gamma, chunk, workspace, cu_seqlens=None, has_state_in=False,
                      g=None, gn_weight=None, gn_bias=None, eps=1e-5, out_dtype=None, out=None,
                      stream=None):
    """Output phase only: reads the workspace of a preceding chunkwise_states call."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (workspace, "workspace")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    nseq = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if _wide(max(int(chunk), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_chunkwise_outputs")
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    ng = None
    if g is not None:
        _dev(g, "g")
        ng = NormGate(g.data_ptr(), _dt(g), gn_weight.data_ptr() if gn_weight is not None else None,
                      gn_bias.data_ptr() if gn_bias is not None else None, float(eps))
    st = lib().retention_chunkwise_outputs(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _gammas(gamma, H), int(chunk), _ptr(cu_seqlens), nseq,
        1 if has_state_in else 0, _ptr(out), _dt(out),
        ctypes.byref(ng) if ng is not None else None, _ptr(workspace),
        workspace.numel() * workspace.element_size(), B, T, H, dk, dv, _stream(stream))
    _check(st, "retention_chunkwise_outputs")
    return out


def chunkwise_fwd_static_ws(q, k, v, gamma, chunk, cu_seqlens=None, state_in=None,
                            state_out=None, g=None, gn_weight=None, gn_bias=None, eps=1e-5,
                            out=None, out_dtype=None, stream=None):
    """chunkwise_fwd without a workspace argument: the library uses its built-in
    device scratch (STATIC_WORKSPACE_BYTES) and allocates nothing itself.
    Outputs (and ``state_out``, if given) must be preallocated by the caller
    only if they are passed; here they are created with torch for convenience."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    nseq = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if _wide(max(int(chunk), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_chunkwise_fwd_static_ws")
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    ng = None
    if g is not None:
        _dev(g, "g")
        ng = NormGate(g.data_ptr(), _dt(g), gn_weight.data_ptr() if gn_weight is not None else None,
                      gn_bias.data_ptr() if gn_bias is not None else None, float(eps))
    st = lib().retention_chunkwise_fwd_static_ws(
        _ptr(q), _ptr(k), _ptr(v), _dt(q), _gammas(gamma, H), int(chunk), _ptr(cu_seqlens), nseq,
        _ptr(state_in), _ptr(state_out), _ptr(out), _dt(out),
        ctypes.byref(ng) if ng is not None else None, B, T, H, dk, dv, _stream(stream))
    _check(st, "retention_chunkwise_fwd_static_ws")
    return out


def chunkwise_bwd_workspace_size(dtype, chunk, B, T, H, dk, dv, nseq=0):
    code = RET_F32 if dtype == torch.float32 else RET_BF16
    if _wide(chunk | B | T | H | dk | dv | nseq):
        return 0
    return int(lib().retention_chunkwise_bwd_workspace_size(code, chunk, B, T, H, dk, dv, nseq))


def chunkwise_bwd(q, k, v, d_out, gamma, chunk, cu_seqlens=None, state_in=None,
                  d_state_out=None, return_d_state=False, workspace=None, stream=None):
    """Gradients of the chunkwise form (retention_chunkwise_bwd).

    q, k: [B,T,H,dk]; v, d_out: [B,T,H,dv], one dtype; packed sequences as in
    :func:`chunkwise_fwd`.  ``state_in`` is the forward's initial state and
    ``d_state_out`` the gradient of its final state (float32 [nseq|B,H,dk,dv],
    optional).  Returns float32 ``(dq, dk, dv)`` and, with ``return_d_state``,
    the gradient of the initial state.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d_out, "d_out")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if (k.shape != q.shape or v.shape[:3] != q.shape[:3] or d_out.shape != v.shape
            or len({q.dtype, k.dtype, v.dtype, d_out.dtype}) != 1):
        raise ValueError("q, k, v, d_out shapes/dtypes disagree")
    nseq = 0
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens")
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor with at least two entries")
        nseq = cu_seqlens.numel() - 1
    if _wide(max(int(chunk), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_chunkwise_bwd")
    nstate = nseq if nseq else B
    for t, n in ((state_in, "state_in"), (d_state_out, "d_state_out")):
        if t is not None:
            _dev(t, n)
            if t.dtype != torch.float32 or tuple(t.shape) != (nstate, H, dk, dv):
                raise ValueError(f"{n} must be float32 [{nstate},{H},{dk},{dv}]")
    dq = torch.empty(B, T, H, dk, device=q.device, dtype=torch.float32)
    dkk = torch.empty(B, T, H, dk, device=q.device, dtype=torch.float32)
    dvv = torch.empty(B, T, H, dv, device=q.device, dtype=torch.float32)
    dS0 = (torch.empty(nstate, H, dk, dv, device=q.device, dtype=torch.float32)
           if return_d_state else None)
    need = lib().retention_chunkwise_bwd_workspace_size(_dt(q), chunk, B, T, H, dk, dv, nseq)
    if need == 0:
        raise RetentionError(RET_ERR_UNSUPPORTED if max(dk, dv) > 256 else RET_ERR_INVALID_ARG,
                             "retention_chunkwise_bwd_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    st = lib().retention_chunkwise_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(d_out), _dt(q), _gammas(gamma, H), int(chunk),
        _ptr(cu_seqlens), nseq, _ptr(state_in), _ptr(d_state_out), _ptr(dq), _ptr(dkk),
        _ptr(dvv), _ptr(dS0), _ptr(workspace), workspace.numel() * workspace.element_size(),
        B, T, H, dk, dv, _stream(stream))
    _check(st, "retention_chunkwise_bwd")
    return (dq, dkk, dvv, dS0) if return_d_state else (dq, dkk, dvv)


def rope(q, k, base=10000.0, cu_seqlens=None, q_out=None, k_out=None, stream=None):
    """Rotary position encoding of q and k ([B,T,H,d], one dtype; packed
    sequences as in :func:`chunkwise_fwd`).  Returns ``(q_out, k_out)``; pass
    ``q_out=q, k_out=k`` to rotate in place."""
    _dev(q, "q")
    _dev(k, "k")
    if k.shape != q.shape or k.dtype != q.dtype or q.dim() != 4:
        raise ValueError("q and k must have one [B,T,H,d] shape and one dtype")
    B, T, H, d = q.shape
    nseq = 0
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens")
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor with at least two entries")
        nseq = cu_seqlens.numel() - 1
    if _wide(B | T | H | d | nseq):
        raise _too_large("retention_rope")
    q_out = torch.empty_like(q) if q_out is None else q_out
    k_out = torch.empty_like(k) if k_out is None else k_out
    for t, n in ((q_out, "q_out"), (k_out, "k_out")):
        _dev(t, n)
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{n} must match q")
    st = lib().retention_rope(_ptr(q), _ptr(k), _dt(q), _ptr(q_out), _ptr(k_out), float(base),
                              _ptr(cu_seqlens), nseq, B, T, H, d, _stream(stream))
    _check(st, "retention_rope")
    return q_out, k_out


def rla_fwd(q, k, v, window, cu_seqlens=None, out_dtype=None, out=None, workspace=None,
            stream=None):
    """Residual linear attention (retention_rla_fwd): o_t = softmax(q_t) S_(t-w-1)
    with S_t = S_(t-1) + softmax(k_t)^T v_t.  q, k: [B,T,H,dk]; v: [B,T,H,dv];
    packed sequences as in :func:`chunkwise_fwd`.  Returns o [B,T,H,dv]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes/dtypes disagree")
    nseq = 0
    if cu_seqlens is not None:
        _dev(cu_seqlens, "cu_seqlens")
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor with at least two entries")
        nseq = cu_seqlens.numel() - 1
    if _wide(max(int(window), 0) | B | T | H | dk | dv | nseq):
        raise _too_large("retention_rla_fwd")
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _dev(out, "out")
    need = lib().retention_rla_workspace_size(_dt(q), B, T, H, dk, dv, nseq)
    if need == 0:
        raise RetentionError(RET_ERR_UNSUPPORTED, "retention_rla_workspace_size")
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    st = lib().retention_rla_fwd(_ptr(q), _ptr(k), _ptr(v), _dt(q), int(window), _ptr(cu_seqlens),
                                 nseq, _ptr(out), _dt(out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), B, T, H, dk, dv,
                                 _stream(stream))
    _check(st, "retention_rla_fwd")
    return out


def recurrent_step(q, k, v, gamma, state, out_dtype=torch.float32, out=None, stream=None):
    """One decode step; updates ``state`` [N,H,dk,dv] in place and returns o [N,H,dv]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (state, "state")):
        _dev(t, n)
    N, H, dk = q.shape
    dv = v.shape[2]
    if state.dtype != torch.float32 or tuple(state.shape) != (N, H, dk, dv):
        raise ValueError(f"state must be float32 [{N},{H},{dk},{dv}]")
    if _wide(N | H | dk | dv):
        raise _too_large("retention_recurrent_step")
    if out is None:
        out = torch.empty(N, H, dv, device=q.device, dtype=out_dtype)
    st = lib().retention_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _dt(q), _gammas(gamma, H),
                                        _ptr(state), _ptr(out), _dt(out), N, H, dk, dv,
                                        _stream(stream))
    _check(st, "retention_recurrent_step")
    return out


def recurrent_steps(q, k, v, gamma, state, out_dtype=torch.float32, out=None, stream=None):
    """Tn (<= 16) decode steps in one pass over the state; q,k: [N,Tn,H,dk], v: [N,Tn,H,dv];
    updates ``state`` [N,H,dk,dv] in place and returns o [N,Tn,H,dv].  bf16 inputs with
    Tn >= 12, dk in {128, 256} and dv a multiple of 128 run on the tensor cores (tf32
    products on the float32 state, within the bf16-input tolerance); everything else runs
    in float32 on CUDA cores."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (state, "state")):
        _dev(t, n)
    N, Tn, H, dk = q.shape
    dv = v.shape[3]
    if state.dtype != torch.float32 or tuple(state.shape) != (N, H, dk, dv):
        raise ValueError(f"state must be float32 [{N},{H},{dk},{dv}]")
    if _wide(N | Tn | H | dk | dv):
        raise _too_large("retention_recurrent_steps")
    if out is None:
        out = torch.empty(N, Tn, H, dv, device=q.device, dtype=out_dtype)
    else:
        _dev(out, "out")
    g = _gammas(gamma, H)
    st = lib().retention_recurrent_steps(_ptr(q), _ptr(k), _ptr(v), _dt(q), g, _ptr(state),
                                         _ptr(out), _dt(out), N, Tn, H, dk, dv, _stream(stream))
    _check(st, "retention_recurrent_steps")
    return out


def norm_gate(o, g, weight=None, bias=None, eps=1e-5, out_dtype=None, out=None, stream=None):
    """Per-head GroupNorm + swish gate; o: [ntok,H,dv] (any leading dims), g same size.
    ``out`` (optional) is a preallocated contiguous output of o's size."""
    _dev(o, "o")
    _dev(g, "g")
    H, dv = o.shape[-2], o.shape[-1]
    ntok = o.numel() // (H * dv)
    if g.numel() != o.numel():
        raise ValueError("g must have as many elements as o")
    if _wide(ntok | H | dv):
        raise _too_large("msr_norm_gate")
    if out is None:
        y = torch.empty(o.shape, device=o.device, dtype=out_dtype or o.dtype)
    else:
        _dev(out, "out")
        if out.numel() != o.numel():
            raise ValueError("out must have as many elements as o")
        y = out
    ng = NormGate(g.data_ptr(), _dt(g), weight.data_ptr() if weight is not None else None,
                  bias.data_ptr() if bias is not None else None, float(eps))
    st = lib().msr_norm_gate(_ptr(o), _dt(o), ctypes.byref(ng), _ptr(y), _dt(y), ntok, H, dv,
                             _stream(stream))
    _check(st, "msr_norm_gate")
    return y


def _ready(stream, **tensors):
    """Checks the tensors of one call (None allowed): contiguous CUDA tensors, all on the
    current device, as is ``stream``.  Returns the raw stream to launch on."""
    cur = None
    for name, t in tensors.items():
        if t is None:
            continue
        if cur is None:
            _dev(t, name)
            cur = torch.cuda.current_device()
        if not (isinstance(t, torch.Tensor) and t.is_contiguous() and t.get_device() == cur):
            _dev(t, name)
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    if stream is None:
        return _current_raw_stream(cur)
    if stream.device.index != cur:
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{cur}")
    return stream.cuda_stream


def _current_raw_stream(device):
    # the stream as an integer, without building a Stream object (3 us of a 10 us call)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(device)


def _new(stream, shape, dtype, like):
    """An uninitialised tensor that belongs to the stream the kernels will run on."""
    if stream is None:
        if like.shape == shape:           # 1.3 us (another dtype: 1.6) instead of 2.0
            return torch.empty_like(like, dtype=dtype) if like.dtype != dtype else torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _at(t):
    """Device address as the integer ctypes takes for a pointer."""
    return None if t is None else t.data_ptr()


def _shaped(t, name, shape, dtype=None):
    if t is not None and (t.shape != shape or (dtype is not None and t.dtype != dtype)):
        kind = "" if dtype is None else f"{str(dtype)[6:]} "
        raise ValueError(f"{name} must be {kind}{list(shape)}")


def _offsets(cu_seqlens):
    if cu_seqlens is None:
        return 0
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor with at least two entries")
    return cu_seqlens.numel() - 1


def glr_chunk_slots(B, T, nseq=0):
    """Rows of ``chunk_states`` for these sizes (0 if they are invalid)."""
    return int(lib().retention_glr_chunk_slots(B, T, nseq)) if not _wide(B | T | nseq) else 0


def _glr_inputs(where, x, r, i, lam, cu_seqlens):
    if x.dim() != 3 or r.shape != x.shape or i.shape != x.shape or not x.dtype == r.dtype == i.dtype:
        raise ValueError("x, r, i must have one [B,T,D] shape and one dtype")
    B, T, D = x.shape
    _shaped(lam, "lam", (D,), torch.float32)
    nseq = _offsets(cu_seqlens)
    if nseq and B != 1:
        raise ValueError("packed sequences need B = 1")
    if _wide(B | T | D | nseq):
        raise _too_large(where)
    return B, T, D, nseq


def glr_fwd(x, r, i, lam, c=8.0, cu_seqlens=None, state_in=None, return_state=False,
            return_chunks=False, out_dtype=None, out=None, state_out=None, chunk_states=None,
            stream=None):
    """Gated linear recurrence h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t)) (retention_glr_fwd).

    x, r, i: [B,T,D], one dtype; lam: float32 [D]; packed sequences: B = 1 and ``cu_seqlens``
    as in :func:`chunkwise_fwd`.  ``state_in`` / ``state_out``: float32 [nseq|B,D].  Returns
    ``h`` [B,T,D], then the final states with ``return_state``, then with ``return_chunks``
    the states entering every 64 tokens (float32 [slots,D]), which :func:`glr_bwd` takes.
    """
    raw = _ready(stream, x=x, r=r, i=i, lam=lam, cu_seqlens=cu_seqlens, state_in=state_in, out=out,
                 state_out=state_out, chunk_states=chunk_states)
    B, T, D, nseq = _glr_inputs("retention_glr_fwd", x, r, i, lam, cu_seqlens)
    states = (nseq or B, D)
    slots = (glr_chunk_slots(B, T, nseq), D) if return_chunks or chunk_states is not None else None
    _shaped(state_in, "state_in", states, torch.float32)
    _shaped(state_out, "state_out", states, torch.float32)
    _shaped(out, "out", x.shape, out_dtype)
    _shaped(chunk_states, "chunk_states", slots, torch.float32)
    if out is None:
        out = _new(stream, x.shape, out_dtype or x.dtype, x)
    if return_state and state_out is None:
        state_out = _new(stream, states, torch.float32, x)
    if return_chunks and chunk_states is None:
        chunk_states = _new(stream, slots, torch.float32, x)
    st = lib().retention_glr_fwd(_at(x), _at(r), _at(i), _dt(x), _at(lam), float(c),
                                 _at(cu_seqlens), nseq, _at(state_in), _at(state_out), _at(out),
                                 _dt(out), _at(chunk_states), B, T, D, raw)
    _check(st, "retention_glr_fwd")
    if not (return_state or return_chunks):
        return out
    return (out,) + ((state_out,) if return_state else ()) + (
        (chunk_states,) if return_chunks else ())


def glr_bwd_workspace_size(B, T, D, nseq=0):
    if _wide(B | T | D | nseq):
        return 0
    return int(lib().retention_glr_bwd_workspace_size(B, T, D, nseq))


def glr_bwd(x, r, i, lam, chunk_states, d_h, c=8.0, cu_seqlens=None, d_state_out=None,
            return_d_state=False, grad_dtype=None, workspace=None, stream=None):
    """Gradients of :func:`glr_fwd` (retention_glr_bwd).

    ``chunk_states`` are the forward's (``return_chunks``), ``d_h`` [B,T,D] the gradient of h
    and ``d_state_out`` (float32 [nseq|B,D], optional) that of the final states.  Returns
    ``(dx, dr, di, d_lam)``, the first three in ``grad_dtype`` (default: x's dtype), and with
    ``return_d_state`` the gradient of the initial states.
    """
    raw = _ready(stream, x=x, r=r, i=i, lam=lam, chunk_states=chunk_states, d_h=d_h,
                 cu_seqlens=cu_seqlens, d_state_out=d_state_out, workspace=workspace)
    B, T, D, nseq = _glr_inputs("retention_glr_bwd", x, r, i, lam, cu_seqlens)
    states = (nseq or B, D)
    _shaped(d_h, "d_h", x.shape)
    _shaped(chunk_states, "chunk_states", (glr_chunk_slots(B, T, nseq), D), torch.float32)
    _shaped(d_state_out, "d_state_out", states, torch.float32)
    need = glr_bwd_workspace_size(B, T, D, nseq)
    gd = grad_dtype or x.dtype
    dx, dr, di = (_new(stream, x.shape, gd, x) for _ in range(3))
    d_lam = _new(stream, (D,), torch.float32, lam)
    dS = _new(stream, states, torch.float32, x) if return_d_state else None
    if workspace is None:
        workspace = _new(stream, (need,), torch.uint8, x)
    st = lib().retention_glr_bwd(_at(x), _at(r), _at(i), _dt(x), _at(lam), float(c),
                                 _at(cu_seqlens), nseq, _at(chunk_states), _at(d_h), _dt(d_h),
                                 _at(d_state_out), _at(dx), _at(dr), _at(di), _dt(dx), _at(d_lam),
                                 _at(dS), _at(workspace),
                                 workspace.numel() * workspace.element_size(), B, T, D, raw)
    _check(st, "retention_glr_bwd")
    return (dx, dr, di, d_lam, dS) if return_d_state else (dx, dr, di, d_lam)


def glr_step(x, r, i, lam, state, c=8.0, out_dtype=torch.float32, out=None, state_out=None,
             stream=None):
    """One token of the gated linear recurrence for N sequences: x, r, i [N,D], ``state``
    float32 [N,D], updated in place unless ``state_out`` is given.  Returns h [N,D]."""
    raw = _ready(stream, x=x, r=r, i=i, lam=lam, state=state, out=out, state_out=state_out)
    if x.dim() != 2 or r.shape != x.shape or i.shape != x.shape or not x.dtype == r.dtype == i.dtype:
        raise ValueError("x, r, i must have one [N,D] shape and one dtype")
    N, D = x.shape
    _shaped(lam, "lam", (D,), torch.float32)
    _shaped(state, "state", (N, D), torch.float32)
    _shaped(state_out, "state_out", (N, D), torch.float32)
    _shaped(out, "out", (N, D))
    if _wide(N | D):
        raise _too_large("retention_glr_step")
    if out is None:
        out = _new(stream, (N, D), out_dtype, x)
    if state_out is None:
        state_out = state
    st = lib().retention_glr_step(_at(x), _at(r), _at(i), _dt(x), _at(lam), float(c), _at(state),
                                  _at(state_out), _at(out), _dt(out), N, D, raw)
    _check(st, "retention_glr_step")
    return out


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out_dtype=None, out=None,
                   return_stats=False, stream=None):
    """Layer norm over the last dimension (retention_layer_norm_fwd); x: [...,D], weight and
    bias: float32 [D] or None.  Returns y and, with ``return_stats``, the float32 mean and
    1/sqrt(var + eps) of every row, which :func:`layer_norm_bwd` takes."""
    raw = _ready(stream, x=x, weight=weight, bias=bias, out=out)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension to normalise")
    D = x.shape[-1]
    ntok = x.numel() // D
    _shaped(weight, "weight", (D,), torch.float32)
    _shaped(bias, "bias", (D,), torch.float32)
    _shaped(out, "out", x.shape, out_dtype)
    if _wide(ntok | D):
        raise _too_large("retention_layer_norm_fwd")
    mean = rstd = None
    if out is None:
        out = _new(stream, x.shape, out_dtype or x.dtype, x)
    if return_stats:
        mean = _new(stream, x.shape[:-1], torch.float32, x)
        rstd = _new(stream, x.shape[:-1], torch.float32, mean)
    st = lib().retention_layer_norm_fwd(_at(x), _dt(x), _at(weight), _at(bias), float(eps),
                                        _at(out), _dt(out), _at(mean), _at(rstd), ntok, D, raw)
    _check(st, "retention_layer_norm_fwd")
    return (out, mean, rstd) if return_stats else out


def layer_norm_bwd_workspace_size(ntok, D):
    if _wide(ntok | D):
        return 0
    return int(lib().retention_layer_norm_bwd_workspace_size(ntok, D))


def layer_norm_bwd(x, d_y, mean, rstd, weight=None, return_d_affine=True, grad_dtype=None,
                   workspace=None, stream=None):
    """Gradients of :func:`layer_norm_fwd` (retention_layer_norm_bwd); ``mean`` and ``rstd`` as
    the forward returned them.  Returns ``(dx, d_weight, d_bias)`` (dx in ``grad_dtype``,
    default x's; the others float32 [D]), or dx alone without ``return_d_affine``."""
    raw = _ready(stream, x=x, d_y=d_y, mean=mean, rstd=rstd, weight=weight, workspace=workspace)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension to normalise")
    D = x.shape[-1]
    ntok = x.numel() // D
    _shaped(d_y, "d_y", x.shape)
    _shaped(mean, "mean", x.shape[:-1], torch.float32)
    _shaped(rstd, "rstd", x.shape[:-1], torch.float32)
    _shaped(weight, "weight", (D,), torch.float32)
    if _wide(ntok | D):
        raise _too_large("retention_layer_norm_bwd")
    dw = db = None
    dx = _new(stream, x.shape, grad_dtype or x.dtype, x)
    if return_d_affine:
        dw = _new(stream, (D,), torch.float32, x if weight is None else weight)
        db = _new(stream, (D,), torch.float32, dw)
        if workspace is None:
            workspace = _new(stream, (layer_norm_bwd_workspace_size(ntok, D),), torch.uint8, x)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().retention_layer_norm_bwd(_at(x), _dt(x), _at(d_y), _dt(d_y), _at(mean), _at(rstd),
                                        _at(weight), _at(dx), _dt(dx), _at(dw), _at(db),
                                        _at(workspace), nbytes, ntok, D, raw)
    _check(st, "retention_layer_norm_bwd")
    return (dx, dw, db) if return_d_affine else dx


def norm_gate_bwd_workspace_size(ntok, H, dv):
    if _wide(ntok | H | dv):
        return 0
    return int(lib().msr_norm_gate_bwd_workspace_size(ntok, H, dv))


def norm_gate_bwd(o, g, d_y, weight=None, bias=None, eps=1e-5, return_d_affine=True,
                  grad_dtype=None, workspace=None, stream=None):
    """Gradients of :func:`norm_gate` (msr_norm_gate_bwd); o and d_y: [...,H,dv], g the same
    size and d_y's dtype.  Returns ``(d_o, d_g, d_weight, d_bias)``: the first two in
    ``grad_dtype`` (default d_y's) and shaped as o and g, the others float32 [H*dv] and left
    out without ``return_d_affine``.  d_o is the ``d_out`` of :func:`chunkwise_bwd`."""
    raw = _ready(stream, o=o, g=g, d_y=d_y, weight=weight, bias=bias, workspace=workspace)
    if o.dim() < 2 or min(o.shape[-2:]) < 1:
        raise ValueError("o must be [...,H,dv]")
    H, dv = o.shape[-2], o.shape[-1]
    ntok = o.numel() // (H * dv)
    _shaped(d_y, "d_y", o.shape)
    if g.numel() != o.numel() or g.dtype != d_y.dtype:
        raise ValueError("g must have as many elements as o and d_y's dtype")
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != H * dv):
            raise ValueError(f"{n} must be float32 with H*dv elements")
    if _wide(ntok | H | dv):
        raise _too_large("msr_norm_gate_bwd")
    dw = db = None
    gd = grad_dtype or d_y.dtype
    d_o, d_g = _new(stream, o.shape, gd, o), _new(stream, g.shape, gd, g)
    if return_d_affine:
        dw = _new(stream, (H * dv,), torch.float32, o if weight is None else weight)
        db = _new(stream, (H * dv,), torch.float32, dw)
        if workspace is None:
            workspace = _new(stream, (norm_gate_bwd_workspace_size(ntok, H, dv),), torch.uint8,
                             o)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    ng = NormGate(g.data_ptr(), _dt(g), _at(weight), _at(bias), float(eps))
    st = lib().msr_norm_gate_bwd(_at(o), _dt(o), ctypes.byref(ng), _at(d_y), _at(d_o), _at(d_g),
                                 _dt(d_o), _at(dw), _at(db), _at(workspace), nbytes, ntok, H, dv,
                                 raw)
    _check(st, "msr_norm_gate_bwd")
    return (d_o, d_g, dw, db) if return_d_affine else (d_o, d_g)


def check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel reported a device-side error."""
    _check(lib().retention_check_device_error(_stream(stream)), "retention_check_device_error")


def selftest_wait_timeout(stream=None):
    """Enqueue the failure-detection self-test: one bounded wait that is never
    satisfied.  A following check_device_error() raises RET_ERR_TIMEOUT."""
    _check(lib().retention_selftest_wait_timeout(_stream(stream)), "retention_selftest_wait_timeout")

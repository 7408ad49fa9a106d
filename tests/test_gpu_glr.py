"""GPU parity of the gated linear recurrence (retention_glr_fwd, _bwd, _step)
against the fp64 oracle, through the C ABI.

Tolerances.  All arithmetic is float32 (unit roundoff u = 2^-24).  Every output
is a sum of products; its size is the same sum with every term taken positive
(the recurrence run on |x|, |S0|, |d_h|, |dS|).  A token's decay is off by at
most 8u y e^-y + 4u a <= 3u + 4u a (y carries the roundings of softplus,
sigmoid and the products; then one exponential) and its added term by ~10 u of
its own, so after T tokens an element is off by less than 16 u (T + 4) times the
largest size in its channel, whatever cancels.  Errors of different tokens have
independent signs, so over a whole tensor (1000 elements or more) the class
bound rel-L2 <= 1e-5 applies as well.  A bf16 store adds half a step, 2^-8 of
the value.  d_lam sums u_t over tokens with signs: its error is measured
against the sum of the sizes of u_t (1e-5: summation chains below 150 adds,
150 u = 9e-6).
"""

import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_retention_b200 import ops, workloads as W
from tests._util import BF16_U, F32_REL_L2, rel_l2
from tests.test_gpu_guards import assert_guards, guarded

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
C = 8.0


def make(B, T, D, dtype="f32", nstate=None, seed=0, lo=0.9, hi=0.999):
    gen = torch.Generator()
    gen.manual_seed(seed)
    td = W.torch_dtype(dtype)
    x, r, i, dh = (torch.randn(B, T, D, generator=gen).to(td) for _ in range(4))
    dec = torch.rand(D, generator=gen, dtype=torch.float64) * (hi - lo) + lo
    lam = torch.log(torch.expm1(-torch.log(dec) / C)).float()
    n = nstate or B
    S0, dS = torch.randn(n, D, generator=gen), torch.randn(n, D, generator=gen)
    return x, r, i, lam, dh, S0, dS


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(got, ref, size, T, what, floor=0.0):
    """size: as ref, every term positive; its largest per channel is the scale of the bound."""
    stored = got.dtype == torch.bfloat16
    g = W.to_f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{what}: non-finite"
    if not g.size:
        return
    if g.size >= 1000:
        e = rel_l2(g, ref)
        assert e <= F32_REL_L2 + (BF16_U if stored else 0.0), f"{what}: rel-L2 {e:.3e}"
    scale = size.reshape(-1, size.shape[-1]).max(axis=0)
    bound = 16 * U32 * (T + 4) * scale + (BF16_U * np.abs(ref) if stored else 0.0) + floor + 1e-36
    worst = (np.abs(g - ref) / bound).max(axis=tuple(range(g.ndim - 1)))
    assert worst.max() <= 1.0, f"{what}: channel {worst.argmax()} is {worst.max():.2f} times its bound off"


class Reference:
    """The oracle's outputs for one set of inputs, and the size of each."""

    def __init__(self, x, r, i, lam, dh, S0=None, dS=None, cu=None, floor=0.0):
        x, r, i, lam, dh, S0, dS = [None if t is None else W.to_f64(t) for t in (x, r, i, lam, dh, S0, dS)]
        B, T, D = x.shape
        segs = [(b, 0, T) for b in range(B)] if cu is None else [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]
        self.floor = floor
        self.S0 = np.zeros((len(segs), D)) if S0 is None else S0
        self.h, self.S = oracle.glr(x, r, i, lam, state=S0, cu_seqlens=cu)
        self.dx, self.dr, self.di, self.dlam, self.dS0 = oracle.glr_backward(
            x, r, i, lam, dh, state=S0, d_state=dS, cu_seqlens=cu)
        y, a, root, si = oracle.retention._glr_gates(r, i, lam, C)
        h, G = np.abs(x) * root * si, np.abs(dh)
        before, self.e_size = np.abs(self.S0).copy(), np.zeros_like(self.S0)
        self.h_size = [before]
        u = np.zeros_like(h)
        for s, (b, t0, t1) in enumerate(segs):
            e = np.zeros(D) if dS is None else np.abs(dS[s])
            for t in range(t1 - 1, t0 - 1, -1):
                G[b, t] += e
                e = a[b, t] * G[b, t]
            self.e_size[s] = e
            prev = before[s]
            for t in range(t0, t1):
                per = np.divide(y[b, t], root[b, t], out=np.zeros(D), where=root[b, t] > 0)
                u[b, t] = G[b, t] * (per * a[b, t] ** 2 * si[b, t] * np.abs(x[b, t]) + a[b, t] * y[b, t] * prev)
                prev = h[b, t] = a[b, t] * prev + h[b, t]
        self.h_size = np.concatenate([before, h.reshape(-1, D)])
        self.dx_size, self.u_size = G * root * si, u
        self.di_size = self.dx_size * np.abs(x)
        self.e_size = np.concatenate([self.e_size, G.reshape(-1, D)])
        self.dlam_size = u.sum(axis=(0, 1)) * oracle.retention._sigmoid(lam) / np.logaddexp(0, lam)

    def check_forward(self, h, S, T, chunks=None, cu=None):
        check(h, self.h, self.h_size, T, "h", self.floor)
        check(S, self.S, self.h_size, T, "state", self.floor)
        if chunks is not None:
            for (s, j), ref in oracle.glr_chunk_states(self.h, self.S0, 64, cu).items():
                first = s * T if cu is None else cu[s]
                check(chunks[first // 64 + s + j], ref, self.h_size, T, f"chunk {s},{j}", self.floor)

    def check_gradients(self, got, T):
        check(got[0], self.dx, self.dx_size, T, "dx", self.floor)
        check(got[1], self.dr, self.u_size, T, "dr", self.floor)
        check(got[2], self.di, self.di_size, T, "di", self.floor)
        err = np.abs(W.to_f64(got[3]) - self.dlam) / (self.dlam_size + self.floor + 1e-30)
        assert err.max() <= 1e-5, f"d_lam channel {err.argmax()}: off by {err.max():.2e} of its terms"
        if len(got) > 4:
            check(got[4], self.dS0, self.e_size, T, "d_state_in", self.floor)


SHAPES = [(1, 1, 1), (2, 7, 3), (2, 63, 5), (1, 64, 64), (3, 65, 130), (5, 2, 257), (2, 200, 33),
          (1, 1100, 96), (2, 513, 128), (1, 2600, 66)]


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("state", [False, True])
def test_forward_and_gradients(dtype, out, B, T, D, state):
    x, r, i, lam, dh, S0, dS = make(B, T, D, dtype, seed=T + D)
    if not state:
        S0 = dS = None
    ref = Reference(x, r, i, lam, dh, S0, dS)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    td = W.torch_dtype(out)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, return_state=True,
                               return_chunks=True, out_dtype=td)
    assert h.dtype == td
    ref.check_forward(h, S, T, chunks)
    assert torch.equal(ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, out_dtype=td), h)
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, d_state_out=dSd, return_d_state=True,
                      grad_dtype=td)
    assert all(g.dtype == td for g in got[:3])
    ref.check_gradients(got, T)
    ops.check_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("up", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("D", [4, 20, 33, 66, 100, 136])
def test_gradients_of_mixed_types(dtype, up, out, D):
    """Each type of the inputs, of d_h and of the gradients with rows that divide by 16 bytes in
    one type and not in the other (4, 20, 100), in both, and in neither."""
    B, T = 2, 150
    x, r, i, lam, dh, S0, dS = make(B, T, D, dtype, seed=D)
    dh = dh.to(W.torch_dtype(up))
    ref = Reference(x, r, i, lam, dh, S0, dS)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, return_state=True,
                               return_chunks=True, out_dtype=W.torch_dtype(out))
    ref.check_forward(h, S, T, chunks)
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, d_state_out=dSd, return_d_state=True,
                      grad_dtype=W.torch_dtype(out))
    ref.check_gradients(got, T)
    ops.check_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [33, 64, 129, 1100])
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 65])
def test_few_channels(dtype, T, D):
    """Rows shorter than a 16-byte piece share it with others; the tensor's last piece is cut."""
    x, r, i, lam, dh, S0, dS = make(1, T, D, dtype, seed=T + D)
    ref = Reference(x, r, i, lam, dh, S0, dS)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, return_state=True, return_chunks=True)
    ref.check_forward(h, S, T, chunks)
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, d_state_out=dSd, return_d_state=True)
    ref.check_gradients(got, T)
    ops.check_device_error()


PACKED = [[0, 1, 64, 65, 0, 300, 127], [5], [0, 0], [1] * 40, [3, 0, 0, 2, 1, 0] * 30, [700, 1, 1200]]


@pytest.mark.parametrize("lens", PACKED, ids=lambda l: f"{len(l)}seq{sum(l)}")
@pytest.mark.parametrize("dtype,D", [("f32", 70), ("bf16", 33), ("bf16", 192)])
def test_packed(lens, dtype, D):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x, r, i, lam, dh, S0, dS = make(1, T, D, dtype, nstate=len(lens), seed=len(lens) + D)
    ref = Reference(x, r, i, lam, dh, S0, dS, cu)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    cud = torch.from_numpy(cu).cuda()
    h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, cu_seqlens=cud, state_in=S0d, return_state=True,
                               return_chunks=True, out_dtype=torch.float32)
    ref.check_forward(h, S, T, chunks, cu)
    got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, cu_seqlens=cud, d_state_out=dSd,
                      return_d_state=True, grad_dtype=torch.float32)
    ref.check_gradients(got, T)
    ops.check_device_error()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 7), (5, 130), (2, 1024), (33, 96)])
def test_step_continues_the_forward(dtype, out, N, D):
    x, r, i, lam, dh, S0, _ = make(N, 4, D, dtype, seed=N + D)
    ref = Reference(x, r, i, lam, dh, S0)
    S = S0.cuda()
    ld = lam.cuda()
    for t in range(4):
        tok = [v[:, t].contiguous().cuda() for v in (x, r, i)]
        before = S.clone()
        new = torch.full_like(S, 9.0)
        h2 = ops.glr_step(*tok, ld, S, out_dtype=W.torch_dtype(out), state_out=new)
        assert torch.equal(S, before)                      # left alone when state_out is given
        h = ops.glr_step(*tok, ld, S, out_dtype=W.torch_dtype(out))
        assert torch.equal(S, new) and torch.equal(h, h2)
        check(h, ref.h[:, t], ref.h_size, t + 1, f"h {t}")
    check(S, ref.S, ref.h_size, 4, "state")


def test_gradients_match_differences():
    """Central differences of the library's own forward (float32, step 2^-6: truncation
    ~step^2/6 of third derivatives of order one, rounding ~1e-6 / step) to 2e-3."""
    B, T, D = 1, 70, 4
    x, r, i, lam, dh, S0, dS = cuda(*make(B, T, D, seed=5))
    _, _, chunks = ops.glr_fwd(x, r, i, lam, state_in=S0, return_state=True, return_chunks=True)
    g = ops.glr_bwd(x, r, i, lam, chunks, dh, d_state_out=dS, return_d_state=True)

    def loss(**over):
        a = dict(dict(x=x, r=r, i=i, lam=lam, S=S0), **over)
        h, S = ops.glr_fwd(a["x"], a["r"], a["i"], a["lam"], state_in=a["S"], return_state=True)
        return float((h.double() * dh.double()).sum() + (S.double() * dS.double()).sum())
    step = 2.0 ** -6
    scale = max(float(t.abs().max()) for t in g)
    for name, t, grad in (("x", x, g[0]), ("r", r, g[1]), ("i", i, g[2]), ("lam", lam, g[3]), ("S", S0, g[4])):
        flat, gf = t.reshape(-1), grad.reshape(-1)
        for k in sorted({0, flat.numel() // 2, flat.numel() - 1, 65 * D % flat.numel()}):
            up, dn = flat.clone(), flat.clone()
            up[k] += step
            dn[k] -= step
            fd = (loss(**{name: up.view(t.shape)}) - loss(**{name: dn.view(t.shape)})) / (2 * step)
            assert abs(fd - float(gf[k])) <= 2e-3 * scale, (name, k, fd, float(gf[k]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates(dtype):
    """Closed, open and saturated gates, decays of one and zero, against the oracle.  Where y
    falls below float32's smallest normal, 2^-126, it may count as zero: sqrt(1 - a^2) below
    sqrt(2^-125) = 1.6e-19 is lost, times |x| <= 5 in 150 tokens at most 1e-16 of h and of
    the gradients; that floor is allowed in those channels and in no others."""
    B, T, D = 1, 150, 40
    x, r, i, lam, dh, S0, dS = make(B, T, D, dtype, seed=9)
    r[:, :, 0], r[:, :, 1], r[:, :, 2], r[:, :, 3] = -100.0, 100.0, -30.0, -1e30
    i[:, :, 4], i[:, :, 5], i[:, :, 6], i[:, :, 7] = -80.0, 100.0, -1e30, -50.0
    lam[8], lam[9], lam[10], lam[11] = -120.0, 40.0, -60.0, 1e4
    r[:, :, 12], i[:, :, 12], lam[12] = 100.0, -80.0, 90.0
    r[:, :, 13], r[:, :, 14], i[:, :, 15] = float("-inf"), float("inf"), float("-inf")
    floor = np.zeros(D)
    floor[[0, 3, 8, 13]] = 1e-16
    for state in (False, True):
        s, d = (S0, dS) if state else (None, None)
        ref = Reference(x, r, i, lam, dh, s, d, floor=floor)
        xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, s, d)
        h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, state_in=S0d, return_state=True,
                                   return_chunks=True, out_dtype=torch.float32)
        got = ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, d_state_out=dSd, return_d_state=True,
                          grad_dtype=torch.float32)
        ref.check_forward(h, S, T, chunks)
        ref.check_gradients(got, T)


def test_nan_and_infinity_stay_in_their_channel_and_sequence():
    B, T, D = 3, 200, 70
    x, r, i, lam, dh, S0, dS = make(B, T, D, seed=2)
    clean = cuda(x, r, i, lam, dh, S0, dS)
    h0, S_0, c0 = ops.glr_fwd(*clean[:4], state_in=clean[5], return_state=True, return_chunks=True)
    g0 = ops.glr_bwd(*clean[:4], c0, clean[4], d_state_out=clean[6], return_d_state=True)
    x[1, 100, 9], r[1, 100, 20], i[1, 100, 30], x[1, 100, 40] = (float("nan"),) * 3 + (float("inf"),)
    bad = cuda(x, r, i, lam, dh, S0, dS)
    h, S, c = ops.glr_fwd(*bad[:4], state_in=bad[5], return_state=True, return_chunks=True)
    g = ops.glr_bwd(*bad[:4], c, bad[4], d_state_out=bad[6], return_d_state=True)
    hit = torch.zeros(D, dtype=torch.bool, device="cuda")
    hit[[9, 20, 30, 40]] = True
    assert not torch.isfinite(h[1, 100:][:, hit]).any() and not torch.isfinite(S[1][hit]).any()
    assert torch.equal(h[1, :100], h0[1, :100]) and torch.equal(h[[0, 2]], h0[[0, 2]])
    assert torch.equal(h[1][:, ~hit], h0[1][:, ~hit])
    for a, b in zip(g[:3], g0[:3]):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1][:, ~hit], b[1][:, ~hit])
    assert torch.equal(g[3][~hit], g0[3][~hit]) and torch.equal(g[4][:, ~hit], g0[4][:, ~hit])


def test_bad_offsets_are_reported_and_stay_in_bounds():
    D, T = 40, 100
    x, r, i, lam, dh, _, _ = cuda(*make(1, T, D, seed=1))
    for cu in ([0, 50, 30, 100], [0, 50, 1000], [-7, 50, 100], [0, 50, 90], [3, 100]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        n = len(cu) - 1
        h, hb = guarded((1, T, D), torch.float32)
        S, sb = guarded((n, D), torch.float32)
        ch, cb = guarded((ops.glr_chunk_slots(1, T, n), D), torch.float32)
        ch.zero_()
        ops.check_device_error()
        ops.glr_fwd(x, r, i, lam, cu_seqlens=cud, out=h, state_out=S, chunk_states=ch)
        with pytest.raises(ops.RetentionError) as info:
            ops.check_device_error()
        assert info.value.status == ops.RET_ERR_DEVICE_DATA
        for buf in (hb, sb, cb):
            assert_guards(buf, str(cu))
        ops.glr_bwd(x, r, i, lam, ch, dh, cu_seqlens=cud)
        with pytest.raises(ops.RetentionError):
            ops.check_device_error()


@pytest.mark.parametrize("dtype,B,T,D", [("f32", 2, 77, 33), ("bf16", 1, 130, 66), ("bf16", 2, 300, 128)])
def test_writes_only_its_outputs(dtype, B, T, D):
    x, r, i, lam, dh, S0, _ = cuda(*make(B, T, D, dtype, seed=4))
    h, hb = guarded((B, T, D), W.torch_dtype(dtype))
    S, sb = guarded((B, D), torch.float32)
    ch, cb = guarded((ops.glr_chunk_slots(B, T), D), torch.float32)
    ops.glr_fwd(x, r, i, lam, state_in=S0, out=h, state_out=S, chunk_states=ch)
    ws, wb = guarded((ops.glr_bwd_workspace_size(B, T, D),), torch.uint8)
    ops.glr_bwd(x, r, i, lam, ch, dh, workspace=ws)
    ops.check_device_error()
    for buf, what in ((hb, "h"), (sb, "state"), (cb, "chunks"), (wb, "workspace")):
        assert_guards(buf, what)
    st, tb = guarded((B, D), torch.float32)
    st.copy_(S0)
    o, ob = guarded((B, D), W.torch_dtype(dtype))
    ops.glr_step(*[v[:, 0].contiguous() for v in (x, r, i)], lam, st, out=o)
    assert_guards(tb, "step state")
    assert_guards(ob, "step h")


def test_two_streams_at_once_and_repeatable():
    """Two calls in flight on two streams, without the current stream waiting for them in
    between; every run gives the same bits."""
    sets = [cuda(*make(2, 900, 100, seed=s)) for s in (1, 2)]

    def once(a, stream=None):
        h, S, ch = ops.glr_fwd(*a[:4], state_in=a[5], return_state=True, return_chunks=True, stream=stream)
        return (h, S) + tuple(ops.glr_bwd(*a[:4], ch, a[4], d_state_out=a[6], return_d_state=True,
                                          stream=stream))
    want = [once(a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [once(a, s) for a, s in zip(sets, streams)]
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]   # reuses freed blocks
        torch.cuda.synchronize()
        del junk
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_captured_and_replayed():
    """A training pass in a graph, replayed on new inputs while eager calls go on."""
    a, b = cuda(*make(2, 300, 96, seed=1)), cuda(*make(2, 300, 96, seed=2))

    def once(a):
        h, S, ch = ops.glr_fwd(*a[:4], state_in=a[5], return_state=True, return_chunks=True)
        return (h, S) + tuple(ops.glr_bwd(*a[:4], ch, a[4], d_state_out=a[6], return_d_state=True))
    want = [once(a), once(b)]
    held = [t.clone() for t in a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(held)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = once(held)
        graphs.append((g, out))
    for k, src in ((1, b), (0, a), (1, b)):
        for t, s in zip(held, src):
            t.copy_(s)
        for g, out in graphs:
            g.replay()
        eager = once(src)
        torch.cuda.synchronize()
        for got in [out for _, out in graphs] + [eager]:
            assert all(torch.equal(p, q) for p, q in zip(got, want[k]))


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the end of the tensors against a short call from the stored state."""
    T, D = 264000, 8192                                   # 2.16e9 elements
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    x, r, i = (torch.randn(1, T, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    lam = make(1, 1, D)[3].cuda()
    h, S, ch = ops.glr_fwd(x, r, i, lam, return_state=True, return_chunks=True)
    row = (T - 1) // 64
    t0 = row * 64
    tail = [t[:, t0:].clone() for t in (x, r, i)]
    h2, S2, c2 = ops.glr_fwd(*tail, lam, state_in=ch[row:row + 1].clone(), return_state=True, return_chunks=True)
    torch.testing.assert_close(h[:, t0:].float(), h2.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(S, S2, rtol=1e-5, atol=1e-5)
    dx, dr, di, dlam = ops.glr_bwd(x, r, i, lam, ch, h)
    ex, er, ei, _ = ops.glr_bwd(*tail, lam, c2, h2)
    for a, b in ((dx, ex), (dr, er), (di, ei)):
        torch.testing.assert_close(a[:, t0:].float(), b.float(), rtol=2.0 ** -6, atol=1e-4)
    assert torch.isfinite(dlam).all()
    ops.check_device_error()


def test_binding_refusals():
    x, r, i, lam, dh, S0, _ = cuda(*make(2, 8, 16))
    with pytest.raises(ValueError, match="one .B,T,D. shape"):
        ops.glr_fwd(x, r[:, :4].contiguous(), i, lam)
    with pytest.raises(ValueError, match="one .B,T,D. shape"):
        ops.glr_fwd(x, r.bfloat16(), i, lam)
    with pytest.raises(ValueError, match="contiguous"):
        ops.glr_fwd(x.transpose(0, 1), r.transpose(0, 1), i.transpose(0, 1), lam)
    with pytest.raises(ValueError, match="lam must be"):
        ops.glr_fwd(x, r, i, lam.double())
    with pytest.raises(ValueError, match="state_in must be"):
        ops.glr_fwd(x, r, i, lam, state_in=S0[:1])
    with pytest.raises(ValueError, match="B = 1"):
        ops.glr_fwd(x, r, i, lam, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="1-D int32"):
        ops.glr_fwd(x[:1], r[:1], i[:1], lam, cu_seqlens=torch.tensor([0, 8], device="cuda"))
    with pytest.raises(TypeError, match="unsupported dtype"):
        ops.glr_fwd(x.half(), r.half(), i.half(), lam)
    with pytest.raises(ops.RetentionError):
        ops.glr_fwd(x, r, i, lam, c=0.0)
    with pytest.raises(ValueError, match="chunk_states must be"):
        ops.glr_bwd(x, r, i, lam, S0[:1].clone(), dh)
    with pytest.raises(ValueError, match="d_h must be"):
        ops.glr_bwd(x, r, i, lam, torch.zeros(ops.glr_chunk_slots(2, 8), 16, device="cuda"), dh[:1])
    with pytest.raises(ValueError, match="state must be"):
        ops.glr_step(x[:, 0].contiguous(), r[:, 0].contiguous(), i[:, 0].contiguous(), lam, S0.bfloat16())
    flat = torch.zeros(2 * 8 * 16 + 1, device="cuda")[1:].view(2, 8, 16)      # 4 bytes off 16
    with pytest.raises(ops.RetentionError):
        ops.glr_fwd(flat, r, i, lam)


@pytest.mark.parametrize("lens", [[70] * 128, [64 * (s % 7) + s % 3 for s in range(128)],
                                  [s % 90 for s in range(129)], [900] + [20] * 60 + [901]],
                         ids=["128equal", "128ties", "129given", "62ends"])
def test_sequences_that_start_in_another_order(lens):
    """Up to 128 packed sequences start longest first, more in their own order: equal lengths, empty
    ones and the longest at either end keep their states apart, and calls repeat."""
    D = 72
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x, r, i, lam, dh, S0, dS = make(1, T, D, "f32", nstate=len(lens), seed=len(lens))
    ref = Reference(x, r, i, lam, dh, S0, dS, cu)
    xd, rd, id_, ld, dhd, S0d, dSd = cuda(x, r, i, lam, dh, S0, dS)
    cud = torch.from_numpy(cu).cuda()

    def run():
        h, S, chunks = ops.glr_fwd(xd, rd, id_, ld, cu_seqlens=cud, state_in=S0d,
                                   return_state=True, return_chunks=True)
        return (h, S, chunks) + ops.glr_bwd(xd, rd, id_, ld, chunks, dhd, cu_seqlens=cud,
                                            d_state_out=dSd, return_d_state=True)
    out = run()
    ref.check_forward(*out[:2], T, out[2], cu)
    ref.check_gradients(out[3:], T)
    again = run()
    assert all(torch.equal(a, b) for a, b in zip(out[:2] + out[3:], again[:2] + again[3:]))
    ops.check_device_error()

"""Cases and plain forms of the training and serving operators beside retention.

Three families, in the layouts of ``include/retention.h``:

* ``glr``: the gated linear recurrence over [tokens, channels], with per-token gates.  With
  s_t = sigmoid(r_t), y_t = c softplus(lam) s_t, a_t = exp(-y_t), b_t = sqrt(1 - a_t^2) sigmoid(i_t):
      h_t = a_t h_(t-1) + b_t x_t
  ``glr_fwd`` is the forward over whole (padded or packed) sequences, ``glr_train`` the forward and
  its gradients, ``glr_step`` one token for each of many sequences;
* ``ln``: layer norm over the last dimension, ``ln_fwd`` and (with its gradients) ``ln_train``;
* ``ng``: the gradients of the per-head GroupNorm + Swish gate (``msr_norm_gate``), ``ng_bwd``.

``own`` selects between the elementary torch form and the library's calls.
"""

import math

import numpy as np
import torch

own = False

C_GATE = 8.0
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one generated token for each of 128 sequences, channels as wide as 16 heads of 256
        dict(name="glr_step_n128_d4096", op="glr_step", B=128, T=1, D=4096, dtype="bf16",
             out="bf16", packed=False, state=True),
        # a short prompt continued from a cached state; channels no vector load divides
        dict(name="glr_fwd_f32_b1_t77_d131", op="glr_fwd", B=1, T=77, D=131, dtype="f32",
             out="f32", packed=False, state=True),
        # prefill of one long sequence: little work across the batch, all of it along time
        dict(name="glr_fwd_b1_t16384_d1024", op="glr_fwd", B=1, T=16384, D=1024, dtype="bf16",
             out="bf16", packed=False, state=False),
        # the long-sequence training shape (2 x 8192 tokens, 16 heads of 256), forward and gradients
        dict(name="glr_train_b2_t8192_d4096", op="glr_train", B=2, T=8192, D=4096, dtype="bf16",
             out="bf16", packed=False, state=True),
        # packed ragged float32 batch (lengths from zero up), odd channel count
        dict(name="glr_train_f32_packed17_d1001", op="glr_train", B=17, T=9001, D=1001, dtype="f32",
             out="f32", packed=True, state=True),
        # the norm in front of one decode step of 128 sequences
        dict(name="ln_fwd_n128_d4096", op="ln_fwd", n=128, D=4096, dtype="bf16", affine=True),
        # the pre-norm of the long-sequence training shape
        dict(name="ln_train_n16384_d4096", op="ln_train", n=16384, D=4096, dtype="bf16", affine=True),
        # float32 training, 4 x 2048 tokens of 8 heads of 128
        dict(name="ln_train_f32_n8192_d1024", op="ln_train", n=8192, D=1024, dtype="f32", affine=True),
        # a ragged token count and a width that no vector load divides
        dict(name="ln_train_n4099_d1001", op="ln_train", n=4099, D=1001, dtype="bf16", affine=True),
        # gradients of the norm and gate, long-sequence shape (2 x 8192 tokens, 16 heads of 512)
        dict(name="ng_bwd_n16384_h16_d512", op="ng_bwd", n=16384, H=16, D=512, o="bf16", dtype="bf16",
             affine=True),
        # the same at 4 x 2048 tokens, 8 heads of 256, float32 retention output
        dict(name="ng_bwd_n8192_h8_d256", op="ng_bwd", n=8192, H=8, D=256, o="f32", dtype="bf16",
             affine=True),
        # float32, odd heads and channels, no affine weights
        dict(name="ng_bwd_f32_n1003_h5_d100", op="ng_bwd", n=1003, H=5, D=100, o="f32", dtype="f32",
             affine=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_train", "glr_train", "glr_step", "ln_fwd", "ln_train", "ng_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 1 << 25
    if op.startswith("glr"):
        D = _log_int(rng, 32, 8192)
        if rng.random() < 0.6:
            D = max(32, D // 32 * 32)
        B = _log_int(rng, 1, 256 if op == "glr_step" else 32)
        packed = op != "glr_step" and rng.random() < 0.4
        cap = max(1, most // (D if packed else B * D))
        T = 1 if op == "glr_step" else _log_int(rng, 1, max(1, min(16384, cap)))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, out=rng.choice([dtype, "f32"]), packed=packed,
                    state=op == "glr_step" or rng.random() < 0.5)
    if op.startswith("ln"):
        D = _log_int(rng, 32, 16384)
        if rng.random() < 0.6:
            D = max(32, D // 32 * 32)
        n = _log_int(rng, 1, max(1, min(32768, most // D)))
        return dict(op=op, n=n, D=D, dtype=dtype, affine=rng.random() < 0.7)
    H = rng.choice([1, 2, 3, 5, 8, 16, 32])
    D = _log_int(rng, 16, 1024)
    if rng.random() < 0.6:
        D = max(16, D // 16 * 16)
    n = _log_int(rng, 1, max(1, min(32768, most // (H * D))))
    return dict(op=op, n=n, H=H, D=D, o=rng.choice([dtype, "f32"]), dtype=dtype, affine=rng.random() < 0.7)


def _offsets(case, seed):
    """Host offsets [nseq+1] of the sequences on the flat token axis."""
    B, T = case["B"], case["T"]
    if not case["packed"]:
        return np.arange(B + 1, dtype=np.int64) * T
    cuts = np.sort(np.random.default_rng(seed).integers(0, T + 1, B - 1)) if B > 1 else []
    return np.concatenate([[0], cuts, [T]]).astype(np.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op, D = case["op"], case["D"]
    td = DTYPES[case["dtype"]]
    s = dict(case)
    if op.startswith("glr"):
        B, T = case["B"], case["T"]
        shape = (B, D) if op == "glr_step" else (1, T, D) if case["packed"] else (B, T, D)
        for name in ("x", "r", "i"):
            s[name] = normal(*shape).to(td)
        # slowest decays exp(-c softplus(lam)) uniform in [0.9, 0.999]
        u = torch.rand(D, generator=gen, device="cuda", dtype=torch.float64) * 0.099 + 0.9
        s["lam"] = torch.log(torch.expm1(-torch.log(u) / C_GATE)).float()
        s["h0"] = normal(B, D) if case["state"] else None
        off = _offsets(case, seed)
        s["reach"] = int((off[1:] - off[:-1]).max())
        s["cu"] = torch.from_numpy(off.astype(np.int32)).cuda() if case["packed"] else None
        s["offsets"] = torch.from_numpy(off).cuda()
        if op == "glr_train":
            s["dh"] = normal(*shape).to(td if case["out"] == "bf16" else torch.float32)
            s["dS"] = normal(B, D) if case["state"] else None
        if op == "glr_step":
            s["h1"] = torch.empty(B, D, device="cuda")
        return s
    n = case["n"]
    width = D if op.startswith("ln") else case["H"] * D
    s["w"] = 1.0 + 0.1 * normal(width) if case["affine"] else None
    s["b"] = 0.1 * normal(width) if case["affine"] else None
    if op.startswith("ln"):
        # a residual stream: channels with offsets of their own
        s["x"] = (normal(n, D) + 0.3 * normal(D)).to(td)
        if op == "ln_train":
            s["dy"] = normal(n, D).to(td)
        return s
    H = case["H"]
    s["x"] = (0.5 * normal(n, H, D)).to(DTYPES[case["o"]])
    s["g"] = normal(n, H * D).to(td)
    s["dy"] = normal(n, H, D).to(td)
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the library's calls ---------------------------------------------------

def _run_own(s):
    from linear_recurrent_sequence_retention_b200 import ops
    op = s["op"]
    if op == "glr_step":
        h = ops.glr_step(s["x"], s["r"], s["i"], s["lam"], s["h0"], c=C_GATE,
                         out_dtype=DTYPES[s["out"]], state_out=s["h1"])
        return h, s["h1"]
    if op == "glr_fwd":
        return ops.glr_fwd(s["x"], s["r"], s["i"], s["lam"], c=C_GATE, cu_seqlens=s["cu"],
                           state_in=s["h0"], return_state=True, out_dtype=DTYPES[s["out"]])
    if op == "glr_train":
        h, S, chunks = ops.glr_fwd(s["x"], s["r"], s["i"], s["lam"], c=C_GATE, cu_seqlens=s["cu"],
                                   state_in=s["h0"], return_state=True, return_chunks=True,
                                   out_dtype=DTYPES[s["out"]])
        grads = ops.glr_bwd(s["x"], s["r"], s["i"], s["lam"], chunks, s["dh"], c=C_GATE,
                            cu_seqlens=s["cu"], d_state_out=s["dS"], return_d_state=True)
        return (h, S) + tuple(grads)
    if op == "ln_fwd":
        return ops.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    if op == "ln_train":
        y, mean, rstd = ops.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS, return_stats=True)
        return (y,) + tuple(ops.layer_norm_bwd(s["x"], s["dy"], mean, rstd, s["w"]))
    return ops.norm_gate_bwd(s["x"], s["g"], s["dy"], s["w"], s["b"], eps=EPS)


# ---- plain forms: float32, rounded once at the end -------------------------

def _scan(A, V, reach):
    """h_t = A_t h_(t-1) + V_t along dim 0 by recursive doubling; A is zero where a sequence starts."""
    step = 1
    while step < reach:
        V = torch.cat([V[:step], V[step:] + A[step:] * V[:-step]])
        A = torch.cat([A[:step], A[step:] * A[:-step]])
        step *= 2
    return V


def _glr_gates(r, i, lam):
    sp = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))
    s, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    y = C_GATE * sp * s
    return sp, s, y, torch.exp(-y), torch.sqrt(-torch.expm1(-2 * y)), si


def _run_plain(s):
    op = s["op"]
    if op.startswith("glr"):
        return _glr_plain(s)
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    n = xc * rstd
    D = s["D"]
    w = b = None
    if s["w"] is not None:
        w, b = s["w"].view(x.shape[1:]), s["b"].view(x.shape[1:])
    z = n if w is None else n * w + b
    if op == "ln_fwd":
        return z.to(s["x"].dtype)
    dy = s["dy"].float()
    if op == "ng_bwd":
        g = s["g"].float().view(x.shape)
        sg = 1 / (1 + torch.exp(-g))
        dg = (dy * z * sg * (1 + g * (1 - sg))).to(s["g"].dtype).view(s["g"].shape)
        dy = dy * g * sg
    dw = (dy * n).sum(0, dtype=torch.float64).float()
    db = dy.sum(0, dtype=torch.float64).float()
    dn = dy if w is None else dy * w
    dx = rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    if op == "ng_bwd":
        return dx.to(s["dy"].dtype), dg, dw.view(-1), db.view(-1)
    return z.to(s["x"].dtype), dx.to(s["x"].dtype), dw, db


def _glr_plain(s):
    out = DTYPES[s["out"]]
    shape, D = s["x"].shape, s["D"]
    x, r, i = (s[k].float().view(-1, D) for k in ("x", "r", "i"))
    sp, sr, y, a, b0, si = _glr_gates(r, i, s["lam"])
    v = b0 * si * x
    if s["op"] == "glr_step":
        h = a * s["h0"] + v
        return h.to(out), h
    off = s["offsets"]
    full = off[1:] > off[:-1]
    first, last = off[:-1][full], off[1:][full] - 1
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(len(off) - 1, D, device=x.device)
    v[first] += a[first] * h0[full]
    af = a.clone()
    af[first] = 0
    h = _scan(af, v, s["reach"])
    S = h0.clone()
    S[full] = h[last]
    if s["op"] == "glr_fwd":
        return h.to(out).view(shape), S
    dh = s["dh"].float().view(-1, D)
    dS = s["dS"] if s["dS"] is not None else torch.zeros_like(S)
    dh = dh.clone()
    dh[last] += dS[full]
    # e_t = a_t (dh_t + e_(t+1)): the gradient passed to the token before
    ar = a.clone()
    ar[last] = 0
    e = torch.flip(_scan(torch.flip(ar, [0]), torch.flip(a * dh, [0]), s["reach"]), [0])
    after = torch.cat([e[1:], e[:1]])
    after[last] = 0
    G = dh + after
    hp = torch.cat([h[:1], h[:-1]])
    hp[first] = h0[full]
    dx = G * b0 * si
    di = dx * x * (1 - si)
    ratio = torch.where(b0 > 0, y / b0, 0)
    u = G * (ratio * a * a * si * x - a * y * hp)
    dr = u * (1 - sr)
    dlam = (u.sum(0, dtype=torch.float64) / (1 + torch.exp(-s["lam"].double())) / sp).float()
    dh0 = dS.clone()
    dh0[full] = e[first]
    grads = [t.to(s["x"].dtype).view(shape) for t in (dx, dr, di)]
    return (h.to(out).view(shape), S, *grads, dlam, dh0)


# ---- the definitions in 64 bits: a loop over tokens, gradients by differentiation -----

def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    leaf = {k: s[k].double().requires_grad_("train" in op or "bwd" in op)
            for k in ("x", "r", "i", "lam", "h0", "w", "b", "g") if s.get(k) is not None}
    if not op.startswith("glr"):
        x = leaf["x"]
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        z = (x - mean) / torch.sqrt(var + EPS)
        if s["w"] is None:
            leaf["w"] = torch.ones(x[0].numel(), dtype=torch.float64, device="cuda", requires_grad=True)
            leaf["b"] = torch.zeros_like(leaf["w"], requires_grad=True)
        z = z * leaf["w"].view(x.shape[1:]) + leaf["b"].view(x.shape[1:])
        if op == "ln_fwd":
            return z.detach()
        want = [leaf[k] for k in (("x", "w", "b") if op == "ln_train" else ("x", "g", "w", "b"))]
        if op == "ng_bwd":
            g = leaf["g"].view(x.shape)
            z = z * g * torch.sigmoid(g)
        grads = torch.autograd.grad(z, want, s["dy"].double())
        return (z.detach(), *grads) if op == "ln_train" else tuple(grads)
    lam = leaf["lam"]
    log_a = -C_GATE * torch.log1p(torch.exp(lam)) * torch.sigmoid(leaf["r"])
    a = torch.exp(log_a)
    v = torch.sqrt(1 - torch.exp(2 * log_a)) * torch.sigmoid(leaf["i"]) * leaf["x"]
    if op == "glr_step":
        h = a * leaf["h0"] + v
        return h, h
    if "h0" not in leaf:
        leaf["h0"] = torch.zeros(case["B"], D, dtype=torch.float64, device="cuda",
                                 requires_grad=op == "glr_train")
    hs, ends = [], []
    if case["packed"]:
        off = _offsets(case, seed)
        at, vt = a[0].unbind(0), v[0].unbind(0)
        for q in range(case["B"]):
            h = leaf["h0"][q]
            for t in range(int(off[q]), int(off[q + 1])):
                h = torch.addcmul(vt[t], at[t], h)
                hs.append(h)
            ends.append(h)
        H, S = torch.stack(hs)[None], torch.stack(ends)
    else:
        at, vt = a.unbind(1), v.unbind(1)
        h = leaf["h0"]
        for t in range(case["T"]):
            h = torch.addcmul(vt[t], at[t], h)
            hs.append(h)
        H, S = torch.stack(hs, 1), h
    if op == "glr_fwd":
        return H, S
    dS = s["dS"].double() if s["dS"] is not None else torch.zeros_like(S)
    grads = torch.autograd.grad([H, S], [leaf[k] for k in ("x", "r", "i", "lam", "h0")],
                                [s["dh"].double(), dS])
    return (H.detach(), S.detach(), *grads)


# ---- what one pass cannot do without ---------------------------------------

def work(case):
    op, D = case["op"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("glr"):
        el = (case["T"] if case["packed"] else case["B"] * case["T"]) * D
        eo = 2 if case["out"] == "bf16" else 4
        states = 4 * case["B"] * D
        if op == "glr_step":
            return {"bytes": el * (3 * e + eo) + 2 * states + 4 * D, "flops": 30 * el}
        n = el * (3 * e + eo) + 4 * D + states * (2 if case["state"] else 1)
        if op == "glr_fwd":
            return {"bytes": n, "flops": 30 * el}
        # x, r, i, d_h and h, dx, dr, di once each; lam and its gradient; the states and theirs
        return {"bytes": el * (6 * e + 2 * eo) + 8 * D + states * (4 if case["state"] else 2),
                "flops": 80 * el}
    if op.startswith("ln"):
        el, w = case["n"] * D, 8 * D if case["affine"] else 0
        if op == "ln_fwd":
            return {"bytes": 2 * el * e + w, "flops": 8 * el}
        return {"bytes": 4 * el * e + w + 8 * D, "flops": 22 * el}
    el, eo = case["n"] * case["H"] * D, 2 if case["o"] == "bf16" else 4
    return {"bytes": el * (eo + 4 * e) + 8 * case["H"] * D * (2 if case["affine"] else 1),
            "flops": 40 * el}

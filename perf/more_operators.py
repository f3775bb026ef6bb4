"""Cases of a recurrent block's operators, for training and for serving: the gated
linear recurrence (whole sequences, one token, forward with backward), the norms
after and before a block joined with its gate and the residual sum (forward and
backward), and the gradient of the causal convolution in front of the recurrence.

`run` computes a case in plain torch operations (fp32, rounded once at the end),
or with `own` set through the library's entry points.  `exact` gives the
operator's definition in 64 bits.  Layouts are those of the library: sequences
[b, L, C], states [b, C], rows [rows, C].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-5    # added to a row's mean square


# ------------------------------------------------------------------- cases
def _glr(name, op, b, L, C, dtype="bf16", gated=False, state=True, ragged=False):
    """op: glr_fwd, or glr_train (the forward pass and its backward)."""
    c = {"op": op, "b": b, "L": L, "C": C, "dtype": dtype, "gated": gated, "state": state, "ragged": ragged}
    return {"name": name, **c} if name else c


def _step(name, b, C, dtype="bf16", gated=False):
    c = {"op": "glr_step", "b": b, "C": C, "dtype": dtype, "gated": gated}
    return {"name": name, **c} if name else c


def _conv(name, b, L, C, W=4, dtype="bf16", bias=False, silu=True, state=True, ragged=False):
    c = {"op": "conv_bwd", "b": b, "L": L, "C": C, "W": W, "dtype": dtype, "bias": bias, "silu": silu,
         "state": state, "ragged": ragged}
    return {"name": name, **c} if name else c


def _norm(name, op, rows, C, dtype="bf16", residual="bf16", gated=False, scaled=True, post=True, pre=True):
    """op: norm_fwd or norm_bwd; residual: the residual stream's dtype."""
    c = {"op": op, "rows": rows, "C": C, "dtype": dtype, "residual": residual, "gated": gated, "scaled": scaled,
         "post": post, "pre": pre}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the benchmark's layer (4 x 8192 tokens, 64 heads of 64 = 4096 channels, a carried state):
        # prefill, or a forward pass of evaluation
        _glr("glr_long", "glr_fwd", 4, 8192, 4096),
        # one prompt of an odd length, gated, as a server prefills it alone
        _glr("glr_prompt", "glr_fwd", 1, 1237, 4096, gated=True, state=False),
        # a training step's part: forward and backward, gated
        _glr("glr_train_long", "glr_train", 4, 4096, 4096, gated=True),
        # a small fp32 model's padded batch, rows of every length from 0 to L
        _glr("glr_train_ragged_fp32", "glr_train", 6, 777, 1000, dtype="fp32", ragged=True),
        # decoding: one sequence, and 256 sequences, gated
        _step("step_one", 1, 4096),
        _step("step_b256", 256, 4096, gated=True),
        # the gradient of the library's long convolution (4 x 8192 tokens of 8192 channels), and of a
        # small one with bias on odd sizes
        _conv("conv_bwd_long", 4, 8192, 8192),
        _conv("conv_bwd_fp32", 3, 777, 1000, dtype="fp32", bias=True, ragged=True),
        # between two blocks of the long batch: gate, norm, scale, residual sum and the next norm;
        # and the same for the tokens of 256 decoded sequences, with an fp32 residual
        _norm("norm_long", "norm_fwd", 32768, 4096, gated=True),
        _norm("norm_decode", "norm_fwd", 256, 4096, residual="fp32"),
        # its gradient: the long batch, and an odd number of rows and channels with an fp32 residual
        _norm("norm_bwd_long", "norm_bwd", 32768, 4096, gated=True),
        _norm("norm_bwd_odd", "norm_bwd", 1237, 2049, residual="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(("glr_fwd", "glr_train", "glr_step", "conv_bwd", "norm_fwd", "norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    C = rng.choice((1, 8, 8, 8)) * _log(rng, 16, 1024)
    coin = lambda p=0.5: rng.random() < p  # noqa: E731
    if op in ("glr_fwd", "glr_train", "conv_bwd"):
        most = (4 * 8192 * 4096 if op == "glr_fwd" else 4 * 4096 * 4096) // (2 if dtype == "fp32" else 1)
        L = _log(rng, 1, 16384)
        while L * C > most:
            L //= 2
        b = _log(rng, 1, max(1, min(64, most // (L * C))))
    if op == "glr_step":
        return _step(None, _log(rng, 1, 512), C, dtype, coin())
    if op == "conv_bwd":
        return _conv(None, b, L, C, rng.choice((2, 3, 4, 4)), dtype, coin(), coin(0.8), coin(), coin(0.3))
    if op in ("glr_fwd", "glr_train"):
        return _glr(None, op, b, L, C, dtype, coin(), coin(0.7), coin(0.3))
    rows = _log(rng, 1, max(1, min(65536, 16384 * 4096 // C)))
    post = coin(0.7)
    return _norm(None, op, rows, C, dtype, dtype if coin() else "fp32", coin(), coin(), post, not post or coin(0.8))


# ------------------------------------------------------------------ inputs
def _lengths(c, gen):
    """Lengths 0 .. L in equal steps, in an order of the seed's (one row: the whole length)."""
    b, L = c["b"], c["L"]
    n = [L] if b == 1 else [L * i // (b - 1) for i in range(b)]
    return torch.tensor(n, dtype=torch.int32, device="cuda")[torch.randperm(b, generator=gen, device="cuda")]


def _total(c):
    """Tokens that are computed: the sum of the lengths."""
    b, L = c["b"], c["L"]
    return b * L if not c["ragged"] or b == 1 else sum(L * i // (b - 1) for i in range(b))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = {"generator": gen, "device": "cuda"}
    dt, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op in ("glr_fwd", "glr_train", "glr_step"):
        b, C = case["b"], case["C"]
        t = (b, C) if op == "glr_step" else (b, case["L"], C)
        # x as it leaves the convolution; r, i, z as they leave their projections
        s["x"] = torch.nn.functional.silu(torch.randn(*t, **kw)).to(dt)
        s["r"], s["i"] = torch.randn(*t, **kw).to(dt), torch.randn(*t, **kw).to(dt)
        s["z"] = torch.randn(*t, **kw).to(dt) if case["gated"] else None
        # log decay at an open gate: 8 log(u), u in [0.9, 0.999] (half lives of one to a thousand tokens)
        s["A"] = 8 * torch.log(0.9 + 0.099 * torch.rand(C, **kw))
        s["state"] = 0.5 * torch.randn(b, C, **kw) if case.get("state", True) else None
        s["lengths"] = _lengths(case, gen) if case.get("ragged") else None
        if op == "glr_train":
            s["dy"] = torch.randn(*t, **kw).to(dt)
            s["dfinal"] = torch.randn(b, C, **kw) if case["state"] else None
    elif op == "conv_bwd":
        b, L, C, W = case["b"], case["L"], case["C"], case["W"]
        s["x"], s["dy"] = torch.randn(b, L, C, **kw).to(dt), torch.randn(b, L, C, **kw).to(dt)
        s["weight"] = torch.randn(C, W, **kw) * W ** -0.5
        s["bias"] = torch.randn(C, **kw) * 0.1 if case["bias"] else None
        s["state"] = torch.randn(b, W - 1, C, **kw).to(dt) if case["state"] else None
        s["dfinal"] = torch.randn(b, W - 1, C, **kw).to(dt) if case["state"] else None
        s["lengths"] = _lengths(case, gen) if case["ragged"] else None
    else:
        rows, C, rd = case["rows"], case["C"], DTYPES[case["residual"]]
        s["x"] = torch.randn(rows, C, **kw).to(dt)
        s["z"] = torch.randn(rows, C, **kw).to(dt) if case["gated"] else None
        s["residual"] = (2 * torch.randn(rows, C, **kw)).to(rd)   # norm_bwd: the sum that was kept
        s["post_weight"] = 1 + 0.1 * torch.randn(C, **kw) if case["post"] else None
        s["pre_weight"] = 1 + 0.1 * torch.randn(C, **kw) if case["pre"] else None
        s["scale"] = 0.5 + 0.1 * torch.randn(C, **kw) if case["scaled"] else None
        if op == "norm_bwd":
            s["dresidual"] = torch.randn(rows, C, **kw).to(rd)
            s["dy"] = torch.randn(rows, C, **kw).to(dt) if case["pre"] else None
    return s


# ------------------------------------------------------------- plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t from zero along dim 1: sums over spans of 1, 2, 4, ... tokens.  Overwrites both."""
    n = 1
    while n < a.shape[1]:
        u[:, n:] += a[:, n:] * u[:, :-n]
        a[:, n:] = a[:, n:] * a[:, :-n]
        n *= 2
    return u


def _recurrence(s, x, r, i):
    """(a, s of s^2 = 1 - a^2, gates sigma(r), sigma(i)) in fp32."""
    sr, si = _sigmoid(r.float()), _sigmoid(i.float())
    la = s["A"] * sr
    return la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), sr, si


def _plain_glr(s):
    c = s["case"]
    b, L, C = s["x"].shape
    dt, x = s["x"].dtype, s["x"].float()
    la, a, m, sr, si = _recurrence(s, s["x"], s["r"], s["i"])
    here = None
    if s["lengths"] is not None:  # tokens past a row's length leave its state as it is
        here = (torch.arange(L, device=x.device) < s["lengths"][:, None])[..., None]
        a, m = torch.where(here, a, 1.0), torch.where(here, m, 0.0)
    h0 = s["state"] if s["state"] is not None else torch.zeros(b, C, device=x.device)
    u = m * si * x
    u[:, 0] += a[:, 0] * h0
    h = _scan(a.clone(), u)
    gate = _sigmoid(s["z"].float()) if c["gated"] else None
    y = h if gate is None else h * s["z"].float() * gate
    if here is not None:
        y = torch.where(here, y, 0.0)
    out = {"y": y.to(dt), "state": h[:, -1].clone()}
    if c["op"] == "glr_fwd":
        return out
    dy = s["dy"].float()
    if here is not None:
        dy = torch.where(here, dy, 0.0)
    if gate is not None:
        z = s["z"].float()
        out["dz"] = (dy * h * gate * (1 + z * (1 - gate))).to(dt)
        dy = dy * z * gate
    if s["dfinal"] is not None:
        dy = dy.clone()
        dy[:, -1] += s["dfinal"]
    # dh_t = dy_t + a_{t+1} dh_{t+1}: the scan from the other end
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    dh = _scan(after.flip(1), dy.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    out["dstate"] = a[:, 0] * dh[:, 0]
    q = torch.where(m > 0, -la / m, 0.0)                    # -la / s
    e = dh * (la * a * before + q * a * a * si * x)         # la d(la)
    if here is not None:
        e = torch.where(here, e, 0.0)
    out["dx"] = (dh * m * si).to(dt)
    out["dr"] = (e * (1 - sr)).to(dt)
    out["di"] = (dh * m * si * (1 - si) * x).to(dt)
    out["dA"] = e.sum((0, 1)) / s["A"]
    return out


def _plain_step(s):
    la, a, m, sr, si = _recurrence(s, s["x"], s["r"], s["i"])
    h = a * s["state"] + m * si * s["x"].float()
    y = h if s["z"] is None else h * s["z"].float() * _sigmoid(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": h}


def _plain_conv(s):
    c = s["case"]
    b, L, C = s["x"].shape
    W, w, dt = c["W"], s["weight"], s["x"].dtype
    state = s["state"] if s["state"] is not None else torch.zeros(b, W - 1, C, device=w.device, dtype=dt)
    x = torch.cat([state, s["x"]], 1).float()
    d = s["dy"].float()
    if c["silu"]:
        p = sum(x[:, k:k + L] * w[:, k] for k in range(W))
        if s["bias"] is not None:
            p = p + s["bias"]
        g = _sigmoid(p)
        d = d * g * (1 + p * (1 - g))
    n = torch.full((b,), L, device=w.device)
    if s["lengths"] is not None:
        n = s["lengths"].long()
        d = torch.where((torch.arange(L, device=w.device) < n[:, None])[..., None], d, 0.0)
    dx = torch.zeros_like(x)
    for k in range(W):
        dx[:, k:k + L] += d * w[:, k]
    if s["dfinal"] is not None:  # the last W - 1 inputs of each row
        at = (n[:, None] + torch.arange(W - 1, device=w.device))[..., None].expand(-1, -1, C)
        dx.scatter_add_(1, at, s["dfinal"].float())
    out = {"dx": dx[:, W - 1:].to(dt), "dweight": torch.stack([(d * x[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)}
    if s["bias"] is not None:
        out["dbias"] = d.sum((0, 1))
    if s["state"] is not None:
        out["dstate"] = dx[:, :W - 1].to(dt)
    return out


def _rstd(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)


def _plain_norm(s):
    c = s["case"]
    p = s["x"].float()
    if c["post"]:
        p = p * _rstd(p) * s["post_weight"]
    if c["gated"]:
        z = s["z"].float()
        p = p * z * _sigmoid(z)
    if c["scaled"]:
        p = p * s["scale"]
    r = s["residual"].float() + p
    out = {"residual": r.to(s["residual"].dtype)}
    if c["pre"]:
        out["y"] = (r * _rstd(r) * s["pre_weight"]).to(s["x"].dtype)
    return out


def _plain_norm_bwd(s):
    c, dt = s["case"], s["x"].dtype
    out = {}
    d = s["dresidual"].float()
    if c["pre"]:
        r, dy = s["residual"].float(), s["dy"].float()
        k = _rstd(r)
        r = r * k
        out["dpre_weight"] = (dy * r).sum(0)
        g = dy * s["pre_weight"]
        d = d + k * (g - r * (g * r).mean(-1, keepdim=True))
    out["dresidual"] = d.to(s["dresidual"].dtype)
    x = s["x"].float()
    k = _rstd(x) if c["post"] else 1.0
    x = x * k
    n = x * s["post_weight"] if c["post"] else x
    z = gate = None
    if c["gated"]:
        z = s["z"].float()
        gate = _sigmoid(z)
    if c["scaled"]:
        out["dscale"] = (d * n * z * gate if c["gated"] else d * n).sum(0)
        d = d * s["scale"]
    if c["gated"]:
        out["dz"] = (d * n * gate * (1 + z * (1 - gate))).to(dt)
        d = d * z * gate
    if c["post"]:
        out["dpost_weight"] = (d * x).sum(0)
        d = d * s["post_weight"]
        d = k * (d - x * (d * x).mean(-1, keepdim=True))
    out["dx"] = d.to(dt)
    return out


# -------------------------------------------------------------------- run
_bd = None


def _binding():
    global _bd
    if _bd is None:
        from mamba_chunked_ssd_gb300 import binding
        binding.load_library()
        _bd = binding
    return _bd


def _own(s):
    bd, c, op = _binding(), s["case"], s["case"]["op"]
    if op == "glr_step":
        y, h = bd.mamba2_glr_step(s["x"], s["r"], s["i"], s["A"], z=s["z"], state_in=s["state"])
        return {"y": y, "state": h}
    if op in ("glr_fwd", "glr_train"):
        train = op == "glr_train"
        y, h, chunks = bd.mamba2_glr_fwd(s["x"], s["r"], s["i"], s["A"], z=s["z"], initial_state=s["state"],
                                         lengths=s["lengths"], want_chunk_states=train)
        out = {"y": y, "state": h}
        if train:
            dx, dr, di, dz, dA, dh = bd.mamba2_glr_bwd(s["dy"], s["x"], s["r"], s["i"], s["A"], chunks, z=s["z"],
                                                       dfinal_state=s["dfinal"], lengths=s["lengths"])
            if dz is not None:
                out["dz"] = dz
            out.update({"dstate": dh, "dx": dx, "dr": dr, "di": di, "dA": dA})
        return out
    if op == "conv_bwd":
        has = s["state"] is not None
        dx, dw, db, ds = bd.mamba2_causal_conv_bwd(s["dy"], s["x"], s["weight"], bias=s["bias"], silu=c["silu"],
                                                   initial_state=s["state"], lengths=s["lengths"],
                                                   dfinal_state=s["dfinal"], want_dinitial_state=has)
        out = {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}
    elif op == "norm_fwd":
        r, y = bd.mamba2_block_norm_fwd(s["x"], s["residual"], z=s["z"], post_weight=s["post_weight"],
                                        scale=s["scale"], pre_weight=s["pre_weight"], eps=NORM_EPS, post=c["post"],
                                        pre=c["pre"])
        out = {"residual": r, "y": y}
    else:
        dx, dz, dr, dpost, dscale, dpre = bd.mamba2_block_norm_bwd(
            s["dresidual"], s["dy"], s["x"], s["residual"], z=s["z"], post_weight=s["post_weight"], scale=s["scale"],
            pre_weight=s["pre_weight"], eps=NORM_EPS, post=c["post"], pre=c["pre"])
        out = {"dpre_weight": dpre, "dresidual": dr, "dscale": dscale, "dz": dz, "dpost_weight": dpost, "dx": dx}
    return {n: t for n, t in out.items() if t is not None}


def run(state):
    if own:
        return _own(state)
    return {"glr_fwd": _plain_glr, "glr_train": _plain_glr, "glr_step": _plain_step, "conv_bwd": _plain_conv,
            "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op in ("glr_fwd", "glr_train", "glr_step"):
        b, C, g = case["b"], case["C"], int(case["gated"])
        rows = b if op == "glr_step" else b * case["L"]     # outputs are written past a row's length too
        tok = b if op == "glr_step" else _total(case)
        states = 2 if case.get("state", True) else 1
        if op != "glr_train":
            return {"bytes": (tok * (3 + g) + rows) * C * e + 4 * C + 4 * states * b * C, "flops": tok * C * (16 + 5 * g)}
        return {"bytes": (tok * (4 + g) + rows * (4 + g)) * C * e + 8 * C + 8 * states * b * C,
                "flops": tok * C * (46 + 12 * g)}
    if op == "conv_bwd":
        b, C, W = case["b"], case["C"], case["W"]
        states = 3 if case["state"] else 0
        return {"bytes": (2 * _total(case) + b * case["L"]) * C * e + states * b * (W - 1) * C * e
                + 4 * C * (2 * W + 2 * case["bias"]),
                "flops": _total(case) * C * (4 * W + (2 * W + 8) * case["silu"])}
    n, r = case["rows"] * case["C"], 2 if case["residual"] == "bf16" else 4
    weights = 4 * case["C"] * (case["post"] + case["pre"] + case["scaled"])
    if op == "norm_fwd":
        return {"bytes": n * (e * (1 + case["gated"] + case["pre"]) + 2 * r) + weights,
                "flops": n * (2 + 4 * case["post"] + 4 * case["pre"] + 5 * case["gated"])}
    return {"bytes": n * (e * (2 + 2 * case["gated"] + case["pre"]) + r * (2 + case["pre"])) + 2 * weights,
            "flops": n * (2 + 9 * case["post"] + 9 * case["pre"] + 10 * case["gated"] + 2 * case["scaled"])}


# ------------------------------------------------------------------ exact
def _leaf(t):
    return None if t is None else t.double().detach().requires_grad_()


def _exact_glr(s):
    """Token by token from the definition; gradients by differentiating that."""
    c, step, train = s["case"], s["case"]["op"] == "glr_step", s["case"]["op"] == "glr_train"
    names = ("x", "r", "i", "z")
    x, r, i, z = (None if s[n] is None else s[n].double()[:, None] if step else s[n].double() for n in names)
    b, L, C = x.shape
    A = s["A"].double()
    h = s["state"].double() if s["state"] is not None else x.new_zeros(b, C)
    n = s["lengths"] if s["lengths"] is not None else torch.full((b,), L, device=x.device)
    leaves = {"x": x, "r": r, "i": i, "A": A, "state": h, "z": z}
    with torch.set_grad_enabled(train):
        if train:
            for t in leaves.values():
                if t is not None:
                    t.requires_grad_()
        log_a = A * torch.sigmoid(r)
        a, u = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * (torch.sigmoid(i) * x)
        a_t, u_t = a.unbind(1), u.unbind(1)
        hs = []
        for t in range(L):
            h = torch.where((t < n)[:, None], torch.addcmul(u_t[t], a_t[t], h), h)
            hs.append(h)
        y = torch.stack(hs, 1)
        if z is not None:
            y = y * (z * torch.sigmoid(z))
        y = torch.where((torch.arange(L, device=x.device) < n[:, None])[..., None], y, 0.0)
        out = {"y": y.detach()[:, 0] if step else y.detach(), "state": h.detach()}
        if train:
            total = (y * s["dy"].double()).sum()
            if s["dfinal"] is not None:
                total = total + (h * s["dfinal"].double()).sum()
            live = {k: t for k, t in leaves.items() if t is not None}
            out.update({"d" + k: g for k, g in zip(live, torch.autograd.grad(total, list(live.values())))})
    return out


def _exact_conv(s):
    """Batch row by batch row, differentiating the definition."""
    c = s["case"]
    b, L, C = s["x"].shape
    W, w, bias = c["W"], _leaf(s["weight"]), _leaf(s["bias"])
    dx, ds = [], []
    for k in range(b):
        n = L if s["lengths"] is None else int(s["lengths"][k])
        x = _leaf(s["x"][k])
        past = _leaf(s["state"][k]) if s["state"] is not None else None
        seen = torch.cat([past if past is not None else x.new_zeros(W - 1, C), x[:n]])
        y = 0 if bias is None else bias
        for d in range(W):
            y = y + seen[d:d + n] * w[:, d]
        if c["silu"]:
            y = y * torch.sigmoid(y)
        total = (y * s["dy"][k, :n].double()).sum()
        if s["dfinal"] is not None:
            total = total + (seen[n:] * s["dfinal"][k].double()).sum()
        if total.requires_grad:
            total.backward()
        dx.append(torch.zeros_like(x) if x.grad is None else x.grad)
        if past is not None:
            ds.append(torch.zeros_like(past) if past.grad is None else past.grad)
    out = {"dx": torch.stack(dx), "dweight": w.grad}
    if bias is not None:
        out["dbias"] = bias.grad
    if ds:
        out["dstate"] = torch.stack(ds)
    return out


def _exact_norm(s):
    c, bwd = s["case"], s["case"]["op"] == "norm_bwd"
    names = ("x", "z", "post_weight", "scale", "pre_weight", "residual")
    x, z, w1, al, w2, res = (_leaf(s[n]) if bwd else None if s[n] is None else s[n].double() for n in names)
    unit = lambda t: t / torch.sqrt(torch.mean(t ** 2, -1, keepdim=True) + NORM_EPS)  # noqa: E731
    p = unit(x) * w1 if c["post"] else x
    if z is not None:
        p = p * (z * torch.sigmoid(z))
    if al is not None:
        p = p * al
    if not bwd:
        r = res + p
        return {"residual": r, "y": unit(r) * w2} if c["pre"] else {"residual": r}
    # the sum that was kept is given, so the second norm is differentiated there
    d = s["dresidual"].double()
    out = {}
    if c["pre"]:
        g = torch.autograd.grad((unit(res) * w2 * s["dy"].double()).sum(), (res, w2))
        d, out["dpre_weight"] = d + g[0], g[1]
    out["dresidual"] = d
    leaves = {"dscale": al, "dz": z, "dpost_weight": w1, "dx": x}
    leaves = {k: t for k, t in leaves.items() if t is not None}
    if p is x:
        return {**out, "dx": d}
    out.update(dict(zip(leaves, torch.autograd.grad((p * d).sum(), list(leaves.values())))))
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("glr"):
        return _exact_glr(s)
    return _exact_conv(s) if op == "conv_bwd" else _exact_norm(s)

"""Cases of the gated-delta-rule operators: the chunked and the recurrent gated
delta rule, the causal convolution in front of them and the gated group norm
behind them.

`run` computes a case in plain torch operations (fp32, rounded once at the
end), or with `own` set through the library's entry points.  `exact` gives the
operator's definition in 64 bits.  Layouts are those of the library: q, k
[b, L, G, S], v, y [b, L, nh, H], g, beta [b, L, nh], states [b, nh, S, H].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
L2_EPS = 1e-6      # added to the sum of squares of a normalised q or k row
NORM_EPS = 1e-5    # added to a group's mean square or variance


# ------------------------------------------------------------------- cases
def _gdr(name, b, L, nh, G, H, S, dtype="bf16", l2norm=True, state=True, ragged=False):
    c = {"op": "gdr_fwd", "b": b, "L": L, "nh": nh, "G": G, "H": H, "S": S, "dtype": dtype,
         "l2norm": l2norm, "state": state, "ragged": ragged}
    return {"name": name, **c} if name else c


def _step(name, b, nh, G, H, S, dtype="bf16", l2norm=True):
    c = {"op": "gdr_step", "b": b, "nh": nh, "G": G, "H": H, "S": S, "dtype": dtype, "l2norm": l2norm}
    return {"name": name, **c} if name else c


def _conv(name, b, L, C, W=4, dtype="bf16", bias=False, state=True, ragged=False):
    c = {"op": "conv_fwd", "b": b, "L": L, "C": C, "W": W, "dtype": dtype, "bias": bias,
         "state": state, "ragged": ragged}
    return {"name": name, **c} if name else c


def _conv_step(name, b, C, W=4, dtype="bf16", bias=False):
    c = {"op": "conv_step", "b": b, "C": C, "W": W, "dtype": dtype, "bias": bias}
    return {"name": name, **c} if name else c


def _norm(name, rows, C, groups, mode, mean=False, bias=False, dtype="bf16"):
    c = {"op": "norm", "rows": rows, "C": C, "groups": groups, "mode": mode, "mean": mean,
         "bias": bias, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the long-sequence layer of the library's benchmark (4 x 8192 tokens, 64 heads of 64, state
        # 128, a carried state) with four heads to a q/k group
        _gdr("gdr_long", 4, 8192, 64, 16, 64, 128),
        # heads of 128 columns, two to a q/k group: prefill of four long prompts
        _gdr("gdr_wide", 4, 4096, 32, 16, 128, 128),
        # one prompt of an odd length, as a server prefills it alone
        _gdr("gdr_prompt", 1, 1237, 32, 16, 128, 128, state=False),
        # a padded batch of prompts of every length from 0 to L
        _gdr("gdr_ragged", 16, 1024, 16, 8, 128, 128, ragged=True),
        # a small fp32 problem, every head with its own q and k, inputs already scaled
        _gdr("gdr_fp32", 2, 777, 8, 8, 64, 64, dtype="fp32", l2norm=False),
        # decoding: one sequence, and 256 sequences of the benchmark's layer
        _step("step_one", 1, 32, 16, 128, 128),
        _step("step_b256", 256, 64, 16, 64, 128),
        # the convolution over q, k and v of gdr_long (2 x 16 x 128 + 64 x 64 channels), and one
        # token of 256 sequences
        _conv("conv_long", 4, 8192, 8192),
        _conv_step("conv_step_b256", 256, 8192),
        # the gated norm behind gdr_long (a group per head), the one of the state-space layer (one
        # group, gated first), and a few rows with mean, bias and activation in fp32
        _norm("norm_heads_long", 32768, 4096, 64, "after"),
        _norm("norm_whole_gate_first", 8192, 4096, 1, "before"),
        _norm("norm_mean_silu_fp32", 37, 4096, 16, "silu", mean=True, bias=True, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(("gdr_fwd", "gdr_fwd", "gdr_step", "conv_fwd", "conv_step", "norm", "norm"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op in ("gdr_fwd", "gdr_step"):
        S, H = rng.choice((64, 128, 128, 128, 96, 256)), rng.choice((64, 64, 128, 128, 40))
        G = rng.choice((1, 2, 4, 8, 16))
        nh = G * rng.choice((1, 2, 3, 4))
    if op == "gdr_fwd":
        L = _log(rng, 1, 8192)
        most = 4 * 8192 * 64 * 64 * 128 // 4
        b = _log(rng, 1, max(1, min(64, most // (L * nh * S * H))))
        return _gdr(None, b, L, nh, G, H, S, dtype, rng.random() < 0.7, rng.random() < 0.7, rng.random() < 0.3)
    if op == "gdr_step":
        return _step(None, _log(rng, 1, 256), nh, G, H, S, dtype, rng.random() < 0.7)
    if op == "conv_fwd":
        L, C = _log(rng, 1, 16384), rng.choice((1, 8, 8, 8)) * _log(rng, 16, 1024)
        b = _log(rng, 1, max(1, min(64, 4 * 8192 * 8192 // (L * C))))
        return _conv(None, b, L, C, rng.choice((2, 3, 4, 4)), dtype, rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.3)
    if op == "conv_step":
        return _conv_step(None, _log(rng, 1, 512), rng.choice((1, 8, 8, 8)) * _log(rng, 16, 1024),
                          rng.choice((2, 3, 4, 4)), dtype, rng.random() < 0.5)
    groups, size = rng.choice((1, 2, 8, 16, 32)), rng.choice((64, 128, 256, 100, 33, 512, 2048))
    rows = _log(rng, 1, max(1, min(65536, 32768 * 4096 // (groups * size))))
    return _norm(None, rows, groups * size, groups, rng.choice(("none", "silu", "after", "before")),
                 rng.random() < 0.3, rng.random() < 0.5, dtype)


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
    if op in ("gdr_fwd", "gdr_step"):
        b, nh, G, H, S = (case[n] for n in ("b", "nh", "G", "H", "S"))
        t = (b, case["L"]) if op == "gdr_fwd" else (b,)
        silu = torch.nn.functional.silu
        # q, k, v as they leave the convolution and its activation
        q, k = silu(torch.randn(*t, G, S, **kw)), silu(torch.randn(*t, G, S, **kw))
        if not case["l2norm"]:  # rows that the caller has scaled
            q, k = (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + L2_EPS) for x in (q, k))
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), silu(torch.randn(*t, nh, H, **kw)).to(dt)
        # log decay -A softplus(a + bias): A in [1, 16], steps of 1e-3 to 0.1 at a = 0
        A = 1 + 15 * torch.rand(nh, **kw)
        step = torch.exp(torch.rand(nh, **kw) * math.log(100.0)) * 1e-3
        a = torch.randn(*t, nh, **kw)
        s["g"] = -A * torch.nn.functional.softplus(a + step + torch.log(-torch.expm1(-step)))
        s["beta"] = torch.sigmoid(torch.randn(*t, nh, **kw))
        s["state"] = torch.randn(b, nh, S, H, **kw) * 0.1 if case.get("state", True) else None
        s["scale"] = S ** -0.5
        s["lengths"] = _lengths(case, gen) if case.get("ragged") else None
    elif op in ("conv_fwd", "conv_step"):
        b, C, W = case["b"], case["C"], case["W"]
        t = (b, case["L"]) if op == "conv_fwd" else (b,)
        s["x"] = torch.randn(*t, C, **kw).to(dt)
        s["weight"] = torch.randn(C, W, **kw) * W ** -0.5
        s["bias"] = torch.randn(C, **kw) * 0.1 if case["bias"] else None
        s["state"] = torch.randn(b, W - 1, C, **kw).to(dt) if case.get("state", True) else None
        s["lengths"] = _lengths(case, gen) if case.get("ragged") else None
    else:
        rows, C = case["rows"], case["C"]
        s["x"] = torch.randn(rows, C, **kw).to(dt)
        s["z"] = torch.randn(rows, C, **kw).to(dt) if case["mode"] in ("after", "before") else None
        s["weight"] = 1 + 0.1 * torch.randn(C, **kw)
        s["bias"] = 0.1 * torch.randn(C, **kw) if case["bias"] else None
    return s


# ------------------------------------------------------------- plain forms
def _unit(x, eps):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + eps)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _heads(x, nh):
    """[.., G, S] -> [.., nh, S]: each group's row for its nh / G heads."""
    return x.repeat_interleave(nh // x.shape[-2], dim=-2)


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A (size a power of two): the inverses of the diagonal
    blocks of size n give those of size 2 n, [[P, 0], [-R C P, R]]."""
    T = A.shape[-1]
    inv = torch.eye(T, device=A.device, dtype=A.dtype).expand_as(A).contiguous()
    n = 1
    while n < T:
        blocks = inv.unflatten(-1, (T // (2 * n), 2 * n)).unflatten(-3, (T // (2 * n), 2 * n))
        i = torch.arange(T // (2 * n), device=A.device)
        diag = blocks[..., i, :, i, :]          # [T / 2n, ..., 2n, 2n]
        low = A.unflatten(-1, (T // (2 * n), 2 * n)).unflatten(-3, (T // (2 * n), 2 * n))[..., i, :, i, :]
        diag[..., n:, :n] = -(diag[..., n:, n:] @ (low[..., n:, :n] @ diag[..., :n, :n]))
        blocks[..., i, :, i, :] = diag
        n *= 2
    return inv


def _plain_gdr(s):
    c = s["case"]
    b, L, nh, H, S = (c[n] for n in ("b", "L", "nh", "H", "S"))
    q, k, v, g, beta = s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"]
    if c["l2norm"]:
        q, k = _unit(q, L2_EPS), _unit(k, L2_EPS)
    if s["lengths"] is not None:  # tokens past a row's length leave its state as it is
        here = (torch.arange(L, device=g.device) < s["lengths"][:, None])[..., None]
        g, beta = torch.where(here, g, 0.0), torch.where(here, beta, 0.0)
    T = 64
    while T // 2 >= L:
        T //= 2
    n = -(-L // T)

    def chunks(x):  # [b, L, nh, d] -> [b, nh, n, T, d], zeros past the last token
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * T - L))
        return x.unflatten(1, (n, T)).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v = chunks(_heads(q * s["scale"], nh)), chunks(_heads(k, nh)), chunks(v)
    g, beta = chunks(g[..., None]), chunks(beta[..., None])
    G = g.cumsum(-2)                                  # log decay from the chunk's start
    lower = torch.ones(T, T, dtype=torch.bool, device=g.device).tril()
    decay = torch.exp(torch.where(lower, G - G.transpose(-1, -2), -math.inf))
    A = (beta * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inv = _unit_lower_inverse(A)
    U, W = inv @ (beta * v), inv @ (beta * torch.exp(G) * k)
    P = decay * (q @ k.transpose(-1, -2))
    q = torch.exp(G) * q
    last = G[..., -1:, :]
    k = (torch.exp(last - G) * k).transpose(-1, -2)
    last = torch.exp(last)
    h = s["state"] if s["state"] is not None else torch.zeros(b, nh, S, H, device=g.device)
    y = torch.empty_like(v)
    for i in range(n):
        new = U[:, :, i] - W[:, :, i] @ h
        y[:, :, i] = q[:, :, i] @ h + P[:, :, i] @ new
        h = last[:, :, i] * h + k[:, :, i] @ new
    y = y.permute(0, 2, 3, 1, 4).reshape(b, n * T, nh, H)[:, :L]
    if s["lengths"] is not None:
        y = torch.where(here[..., None], y, 0.0)
    return {"y": y.to(s["v"].dtype).contiguous(), "state": h}


def _plain_step(s):
    c = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["l2norm"]:
        q, k = _unit(q, L2_EPS), _unit(k, L2_EPS)
    q, k = _heads(q * s["scale"], c["nh"]), _heads(k, c["nh"])
    h = torch.exp(s["g"])[..., None, None] * s["state"]
    new = s["beta"][..., None] * (v - (k[..., None] * h).sum(-2))
    h = h + k[..., None] * new[..., None, :]
    return {"y": (q[..., None] * h).sum(-2).to(s["v"].dtype), "state": h}


def _plain_conv(s):
    c = s["case"]
    W, step = c["W"], c["op"] == "conv_step"
    x = s["x"][:, None] if step else s["x"]
    b, L, C = x.shape
    state = s["state"] if s["state"] is not None else torch.zeros(b, W - 1, C, device=x.device, dtype=x.dtype)
    x = torch.cat([state, x], 1)
    y = sum(x[:, w:w + L].float() * s["weight"][:, w] for w in range(W))
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _silu(y).to(x.dtype)
    if s["lengths"] is None:
        return {"y": y[:, 0] if step else y, "state": x[:, L:].contiguous()}
    n = s["lengths"].long()[:, None]
    y = torch.where((torch.arange(L, device=x.device) < n)[..., None], y, 0.0)
    at = n + torch.arange(W - 1, device=x.device)
    return {"y": y, "state": torch.gather(x, 1, at[..., None].expand(-1, -1, C))}


def _plain_norm(s):
    c = s["case"]
    x, z = s["x"].float(), s["z"]
    if c["mode"] == "before":
        x = x * _silu(z.float())
    x = x.unflatten(-1, (c["groups"], -1))
    if c["mean"]:
        x = x - x.mean(-1, keepdim=True)
    x = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)).flatten(-2) * s["weight"]
    if s["bias"] is not None:
        x = x + s["bias"]
    if c["mode"] == "after":
        x = x * _silu(z.float())
    if c["mode"] == "silu":
        x = _silu(x)
    return {"y": x.to(s["x"].dtype)}


# -------------------------------------------------------------------- run
_bd = None


def _binding():
    global _bd
    if _bd is None:
        from mamba_chunked_ssd_gb300 import binding
        binding.load_library()
        _bd = binding
    return _bd


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"gdr_fwd": _plain_gdr, "gdr_step": _plain_step, "conv_fwd": _plain_conv,
                "conv_step": _plain_conv, "norm": _plain_norm}[op](s)
    bd = _binding()
    if op == "gdr_fwd":
        y, h = bd.mamba2_gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], qk_l2norm=c["l2norm"],
                                 initial_state=s["state"], lengths=s["lengths"])
        return {"y": y, "state": h}
    if op == "gdr_step":
        y, h = bd.mamba2_gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], state_in=s["state"], scale=s["scale"],
                                  qk_l2norm=c["l2norm"])
        return {"y": y, "state": h}
    if op == "conv_fwd":
        y, h = bd.mamba2_causal_conv_fwd(s["x"], s["weight"], bias=s["bias"], silu=True, initial_state=s["state"],
                                         lengths=s["lengths"])
        return {"y": y, "state": h}
    if op == "conv_step":
        y, h = bd.mamba2_causal_conv_step(s["x"], s["weight"], state_in=s["state"], bias=s["bias"], silu=True)
        return {"y": y, "state": h}
    y = bd.mamba2_group_norm(s["x"], s["weight"], c["groups"], z=s["z"], bias=s["bias"], eps=NORM_EPS,
                             subtract_mean=c["mean"], mode=c["mode"])
    return {"y": y}


# ------------------------------------------------------------------- work
def work(case):
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op in ("gdr_fwd", "gdr_step"):
        b, nh, G, H, S = (case[n] for n in ("b", "nh", "G", "H", "S"))
        rows = case["b"] * case["L"] if op == "gdr_fwd" else b   # y is written past a row's length too
        tok = _total(case) if op == "gdr_fwd" else b
        states = 2 if case.get("state", True) else 1
        return {"bytes": tok * (2 * G * S * e + nh * H * e + 8 * nh) + rows * nh * H * e + 4 * states * b * nh * S * H,
                "flops": 6 * tok * nh * S * H}
    if op in ("conv_fwd", "conv_step"):
        b, C, W = case["b"], case["C"], case["W"]
        rows = case["b"] * case["L"] if op == "conv_fwd" else b
        tok = _total(case) if op == "conv_fwd" else b
        states = 2 if case.get("state", True) else 1
        return {"bytes": (tok + rows) * C * e + states * b * (W - 1) * C * e + 4 * C * (W + case["bias"]),
                "flops": tok * C * (2 * W + 4)}
    n = case["rows"] * case["C"]
    gated = case["mode"] in ("after", "before")
    return {"bytes": (2 + gated) * n * e + 4 * case["C"] * (1 + case["bias"]), "flops": 8 * n}


# ------------------------------------------------------------------ exact
def _exact_gdr(s):
    """Token by token: h <- e^g h + k (beta (v - (e^g h)^T k))^T, y = scale h^T q."""
    c, step = s["case"], s["case"]["op"] == "gdr_step"
    q, k, v, g, beta = (s[n].double() if not step else s[n].double()[:, None] for n in ("q", "k", "v", "g", "beta"))
    b, L, nh, H = v.shape
    if c["l2norm"]:
        q, k = (x / torch.sqrt(torch.einsum("blgs,blgs->blg", x, x)[..., None] + L2_EPS) for x in (q, k))
    of = torch.arange(nh, device=v.device) // (nh // c["G"])  # each head's group
    h = torch.zeros(b, nh, c["S"], H, dtype=torch.float64, device=v.device)
    if s["state"] is not None:
        h = h + s["state"].double()
    n = s["lengths"] if s["lengths"] is not None else torch.full((b,), L, device=v.device)
    y = torch.zeros_like(v)
    for t in range(L):
        live = (t < n)[:, None]
        kt, qt = k[:, t, of], q[:, t, of]
        at = torch.where(live, torch.exp(g[:, t]), 1.0)
        h = h * at[..., None, None]
        err = v[:, t] - torch.einsum("bnsh,bns->bnh", h, kt)
        err = torch.where(live[..., None], err * beta[:, t, :, None], 0.0)
        h = torch.addcmul(h, kt[..., None], err[..., None, :])
        y[:, t] = torch.where(live[..., None], torch.einsum("bnsh,bns->bnh", h, qt) * s["scale"], 0.0)
    return {"y": y[:, 0] if step else y, "state": h}


def _exact_conv(s):
    c, step = s["case"], s["case"]["op"] == "conv_step"
    x = (s["x"][:, None] if step else s["x"]).double()
    b, L, C = x.shape
    W, w = c["W"], s["weight"].double()
    past = s["state"].double() if s["state"] is not None else x.new_zeros(b, W - 1, C)
    y = x.new_zeros(b, L, C)
    for d in range(W):  # the input d tokens back
        y[:, d:] += x[:, :max(0, L - d)] * w[:, W - 1 - d]
        m = min(d, L)
        y[:, :m] += past[:, W - 1 - d:W - 1 - d + m] * w[:, W - 1 - d]
    if s["bias"] is not None:
        y += s["bias"].double()
    y *= torch.sigmoid(y)
    n = s["lengths"].tolist() if s["lengths"] is not None else [L] * b
    state = torch.stack([torch.cat([past[i], x[i, :n[i]]])[-(W - 1):] for i in range(b)])
    for i in range(b):
        y[i, n[i]:] = 0
    return {"y": y[:, 0] if step else y, "state": state}


def _exact_norm(s):
    c = s["case"]
    x = s["x"].double().reshape(c["rows"], c["groups"], -1)
    gate = None if s["z"] is None else s["z"].double().reshape(x.shape)
    if gate is not None:
        gate = gate * torch.sigmoid(gate)
    if c["mode"] == "before":
        x = x * gate
    m = x.mean(-1, keepdim=True) if c["mean"] else 0.0
    d = torch.sqrt(torch.mean((x - m) ** 2, -1, keepdim=True) + NORM_EPS)
    y = (x - m) / d * s["weight"].double().reshape(c["groups"], -1)
    if s["bias"] is not None:
        y = y + s["bias"].double().reshape(c["groups"], -1)
    if c["mode"] == "after":
        y = y * gate
    if c["mode"] == "silu":
        y = y * torch.sigmoid(y)
    return {"y": y.reshape(c["rows"], c["C"])}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gdr_fwd", "gdr_step"):
        return _exact_gdr(s)
    return _exact_norm(s) if op == "norm" else _exact_conv(s)

"""Plain fp64 forms of the recurrent block's operators for the tests, on the CPU and
straight from their definitions (torch, token by token, so that they can be
differentiated), and the gradients by their formulas."""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu").double()


def counts(lengths, b, L):
    return [L] * b if lengths is None else [min(max(int(n), 0), L) for n in lengths]


def silu(z):
    return z * torch.sigmoid(z)


def glr(x, r, i, A, z=None, init=None, lengths=None):
    """(y [b, L, C], final state [b, C], states after each token [b, L, C])."""
    b, L, C = x.shape
    n = torch.tensor(counts(lengths, b, L))
    h = torch.zeros(b, C, dtype=x.dtype) if init is None else init
    la = A * torch.sigmoid(r)
    hs = []
    for t in range(L):
        new = torch.exp(la[:, t]) * h + torch.sqrt(-torch.expm1(2 * la[:, t])) * torch.sigmoid(i[:, t]) * x[:, t]
        h = torch.where((t < n)[:, None], new, h)
        hs.append(h)
    hs = torch.stack(hs, 1) if L else torch.zeros(b, 0, C, dtype=x.dtype)
    y = hs if z is None else hs * silu(z)
    here = (torch.arange(L) < n[:, None])[..., None]
    return torch.where(here, y, torch.zeros_like(y)), h, hs


def glr_grads(dy, x, r, i, A, z=None, init=None, lengths=None, dfinal=None):
    """Gradients by the formulas, from the other end, and the sums of dA's terms' absolute values."""
    b, L, C = x.shape
    n = counts(lengths, b, L)
    h0 = torch.zeros(b, C, dtype=x.dtype) if init is None else init
    _, _, hs = glr(x, r, i, A, z, init, lengths)
    out = {k: torch.zeros(b, L, C, dtype=x.dtype) for k in ("dx", "dr", "di", "dz")}
    dA, size = torch.zeros(C, dtype=x.dtype), torch.zeros(C, dtype=x.dtype)
    dinit = torch.zeros(b, C, dtype=x.dtype)
    for k in range(b):
        c = torch.zeros(C, dtype=x.dtype) if dfinal is None else dfinal[k]
        for t in reversed(range(n[k])):
            sr, si = torch.sigmoid(r[k, t]), torch.sigmoid(i[k, t])
            la = A * sr
            a = torch.exp(la)
            s = torch.sqrt(-torch.expm1(2 * la))
            before = hs[k, t - 1] if t else h0[k]
            dh = dy[k, t]
            if z is not None:
                sz = torch.sigmoid(z[k, t])
                out["dz"][k, t] = dy[k, t] * hs[k, t] * sz * (1 + z[k, t] * (1 - sz))
                dh = dh * z[k, t] * sz
            dh = dh + c
            e = dh * (la * a * before - la * a * a / s * si * x[k, t])
            out["dx"][k, t], out["dr"][k, t] = dh * s * si, e * (1 - sr)
            out["di"][k, t] = dh * s * x[k, t] * si * (1 - si)
            dA, size = dA + e / A, size + (e / A).abs()
            c = a * dh
        dinit[k] = c
    if z is None:
        del out["dz"]
    return {**out, "dA": dA, "dinit": dinit}, size


def conv(x, weight, bias=None, act=True, init=None, lengths=None):
    """(y [b, L, C], final state [b, W - 1, C])."""
    b, L, C = x.shape
    W = weight.shape[1]
    n = counts(lengths, b, L)
    ys, states = [], []
    for k in range(b):
        past = torch.zeros(W - 1, C, dtype=x.dtype) if init is None else init[k]
        seen = torch.cat([past, x[k, :n[k]]])
        s = sum(seen[w:w + n[k]] * weight[:, w] for w in range(W))
        if bias is not None:
            s = s + bias
        ys.append(torch.cat([silu(s) if act else s, torch.zeros(L - n[k], C, dtype=x.dtype)]))
        states.append(seen[n[k]:])
    return torch.stack(ys), torch.stack(states)


def conv_grads(dy, x, weight, bias=None, act=True, init=None, lengths=None, dfinal=None):
    """Gradients by the formulas, tap by tap, and the sums of the weights' terms' absolute values."""
    b, L, C = x.shape
    W = weight.shape[1]
    n = counts(lengths, b, L)
    dx, dinit = torch.zeros_like(x), torch.zeros(b, W - 1, C, dtype=x.dtype)
    dw, size = torch.zeros(C, W, dtype=x.dtype), torch.zeros(C, W, dtype=x.dtype)
    db, bsize = torch.zeros(C, dtype=x.dtype), torch.zeros(C, dtype=x.dtype)
    for k in range(b):
        past = torch.zeros(W - 1, C, dtype=x.dtype) if init is None else init[k]
        seen = torch.cat([past, x[k, :n[k]]])
        g = torch.zeros_like(seen)
        for t in range(n[k]):
            d = dy[k, t]
            if act:
                p = (seen[t:t + W] * weight.T).sum(0) + (0 if bias is None else bias)
                s = torch.sigmoid(p)
                d = d * s * (1 + p * (1 - s))
            for w in range(W):
                g[t + w] += weight[:, w] * d
                dw[:, w] += d * seen[t + w]
                size[:, w] += (d * seen[t + w]).abs()
            db, bsize = db + d, bsize + d.abs()
        if dfinal is not None:
            g[n[k]:] += dfinal[k]
        dinit[k], dx[k, :n[k]] = g[:W - 1], g[W - 1:]
    return {"dx": dx, "dweight": dw, "dbias": db, "dinit": dinit}, {"dweight": size, "dbias": bsize}


def unit(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def block_norm(x, residual=None, z=None, post_weight=None, scale=None, pre_weight=None, eps=1e-5, post=True, pre=True):
    """(residual_out, y or None)."""
    p = unit(x, eps) if post else x
    for w in (post_weight, None if z is None else silu(z), scale):
        if w is not None:
            p = p * w
    r = p if residual is None else residual + p
    if not pre:
        return r, None
    y = unit(r, eps)
    return r, y if pre_weight is None else y * pre_weight


def block_norm_grads(dr, dy, x, out=None, z=None, post_weight=None, scale=None, pre_weight=None, eps=1e-5, post=True,
                     pre=True):
    """Gradients by the formulas, from the sum `out` that the forward pass wrote, and the sums
    of their terms' absolute values."""
    one = torch.ones(x.shape[-1], dtype=x.dtype)
    w1, al, w2 = (one if w is None else w for w in (post_weight, scale, pre_weight))
    res, size = {}, {}

    def terms(name, t):
        t = t.reshape(-1, t.shape[-1])
        res[name], size[name] = t.sum(0), t.abs().sum(0)

    D = torch.zeros_like(x) if dr is None else dr
    if pre:
        k = 1 / torch.sqrt((out * out).mean(-1, keepdim=True) + eps)
        u = out * k
        terms("dpre_weight", dy * u)
        m = (dy * w2 * u).mean(-1, keepdim=True)
        size["dresidual"] = D.abs() + k * ((dy * w2).abs() + (u * m).abs())
        D = D + k * (dy * w2 - u * m)
    res["dresidual"] = D
    size.setdefault("dresidual", D.abs())
    k = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if post else 1.0
    u = x * k
    n = u * w1
    g = 1.0 if z is None else silu(z)
    terms("dscale", D * n * g)
    size["dscale"] = size["dscale"] + ((n * g).abs() * size["dresidual"]).reshape(-1, x.shape[-1]).sum(0)
    d = D * al
    if z is not None:
        s = torch.sigmoid(z)
        res["dz"] = d * n * s * (1 + z * (1 - s))
        d = d * g
    if post:
        terms("dpost_weight", d * u)
        size["dpost_weight"] = size["dpost_weight"] + (al * g * u * size["dresidual"]).abs().reshape(-1, x.shape[-1]).sum(0)
        d = d * w1
        m = (d * u).mean(-1, keepdim=True)
        size["dx"] = k * (d.abs() + (u * m).abs())
        d = k * (d - u * m)
    res["dx"] = d
    # (the errors of D's terms go on into what is made of it)
    size["dx"] = size.get("dx", d.abs()) + (k * al * g * w1).abs() * size["dresidual"]
    if z is not None:
        size["dz"] = res["dz"].abs() + (al * n * s * (1 + z * (1 - s))).abs() * size["dresidual"]
    return res, size

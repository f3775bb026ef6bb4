"""Plain fp64 forms of the gated-delta-rule operators for the tests, on the CPU
and straight from their definitions (numpy, token by token)."""
from __future__ import annotations

import numpy as np


def f64(t):
    return None if t is None else t.detach().to("cpu").double().numpy()


def _unit(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def gdr(q, k, v, g, beta, scale, l2norm=False, eps=1e-6, init=None, lengths=None):
    """(y [b, L, nh, H], final state [b, nh, S, H]) of the recurrence
    h <- e^g h;  h <- h + k (beta (v - h^T k))^T;  y = scale h^T q."""
    q, k, v, g, beta, init = (f64(t) for t in (q, k, v, g, beta, init))
    b, L, nh, H = v.shape
    S, r = q.shape[-1], nh // q.shape[-2]
    h = np.zeros((b, nh, S, H)) if init is None else init.copy()
    y = np.zeros((b, L, nh, H))
    n = np.full(b, L) if lengths is None else np.clip(lengths.cpu().numpy(), 0, L)
    for i in range(b):
        for t in range(n[i]):
            qt, kt = q[i, t], k[i, t]
            if l2norm:
                qt, kt = _unit(qt, eps), _unit(kt, eps)
            qt, kt = np.repeat(qt, r, 0), np.repeat(kt, r, 0)
            h[i] *= np.exp(g[i, t])[:, None, None]
            w = beta[i, t][:, None] * (v[i, t] - np.einsum("nsh,ns->nh", h[i], kt))
            h[i] += kt[:, :, None] * w[:, None, :]
            y[i, t] = scale * np.einsum("nsh,ns->nh", h[i], qt)
    return y, h


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-x))


def conv(x, weight, bias=None, act=True, init=None, lengths=None):
    x, weight, bias, init = (f64(t) for t in (x, weight, bias, init))
    b, L, C = x.shape
    W = weight.shape[1]
    n = np.full(b, L) if lengths is None else np.clip(lengths.cpu().numpy(), 0, L)
    y = np.zeros((b, L, C))
    state = np.zeros((b, W - 1, C))
    for i in range(b):
        past = np.zeros((W - 1, C)) if init is None else init[i]
        z = np.concatenate([past, x[i, :n[i]]])
        for t in range(n[i]):
            s = (z[t:t + W] * weight.T).sum(0) + (0 if bias is None else bias)
            y[i, t] = silu(s) if act else s
        state[i] = z[n[i]:]
    return y, state


def norm(x, groups, weight=None, bias=None, z=None, eps=1e-5, mean=False, mode="none"):
    x, weight, bias, z = (f64(t) for t in (x, weight, bias, z))
    u = x * silu(z) if mode == "before" else x
    u = u.reshape(*x.shape[:-1], groups, -1)
    if mean:
        u = u - u.mean(-1, keepdims=True)
    u = (u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)).reshape(x.shape)
    if weight is not None:
        u = u * weight
    if bias is not None:
        u = u + bias
    if mode == "after":
        u = u * silu(z)
    return silu(u) if mode == "silu" else u

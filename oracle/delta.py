"""fp64 oracle of the gated delta rule and of the group norm with an
activation: the definitions of ``include/wkv.h`` token by token in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code
with the CUDA library.  Layouts are the C ABI's: r, k (B, T, Hk*N), v
(B, T, H*N), w, beta (B, T, H), states (B, H, N, N).
"""
import numpy as np


def _heads(x, N, share):
    """(B, T, heads*N) -> (T, B, H, N) float64, each key head repeated."""
    B, T, C = x.shape
    return np.repeat(np.asarray(x, np.float64).reshape(B, T, C // N, N), share, axis=2).transpose(1, 0, 2, 3)


def _flat(x):
    """(T, B, H, N) -> (B, T, H*N)."""
    T, B, H, N = x.shape
    return x.transpose(1, 0, 2, 3).reshape(B, T, H * N)


def _parts(w, beta, r, k, v, H):
    N = v.shape[2] // H
    share = H // (k.shape[2] // N)
    a = np.exp(-np.asarray(w, np.float64)).transpose(1, 0, 2)
    b = np.asarray(beta, np.float64).transpose(1, 0, 2)
    return N, share, a, b, _heads(r, N, share), _heads(k, N, share), _heads(v, N, 1)


def _state(state, B, H, N):
    return np.zeros((B, H, N, N)) if state is None else np.asarray(state, np.float64).copy()


def delta_forward(w, beta, r, k, v, H, state_in=None):
    """(y, state_out)."""
    N, _, a, b, r, k, v = _parts(w, beta, r, k, v, H)
    S = _state(state_in, v.shape[1], H, N)
    y = np.empty_like(v)
    for t in range(v.shape[0]):
        S = a[t][..., None, None] * S
        e = v[t] - np.einsum("bhij,bhi->bhj", S, k[t])
        S = S + np.einsum("bhi,bhj->bhij", k[t], b[t][..., None] * e)
        y[t] = np.einsum("bhij,bhi->bhj", S, r[t])
    return _flat(y), S


def delta_backward(w, beta, r, k, v, H, state_in, dy, dstate_out=None):
    """(dr, dk, dv, dw, dbeta, dstate_in): the chain rule through the recurrence."""
    N, share, a, b, r, k, v = _parts(w, beta, r, k, v, H)
    T, B = v.shape[:2]
    dy = _heads(dy, N, 1)
    S = [_state(state_in, B, H, N)]
    err = []
    for t in range(T):
        faded = a[t][..., None, None] * S[-1]
        err.append(v[t] - np.einsum("bhij,bhi->bhj", faded, k[t]))
        S.append(faded + np.einsum("bhi,bhj->bhij", k[t], b[t][..., None] * err[t]))
    D = _state(dstate_out, B, H, N)
    dr, dk, dv = (np.empty_like(v) for _ in range(3))
    dw, db = np.empty_like(a), np.empty_like(b)
    for t in reversed(range(T)):
        D = D + np.einsum("bhi,bhj->bhij", r[t], dy[t])
        dr[t] = np.einsum("bhij,bhj->bhi", S[t + 1], dy[t])
        du = np.einsum("bhij,bhi->bhj", D, k[t])
        db[t] = (du * err[t]).sum(-1)
        dv[t] = b[t][..., None] * du
        faded = a[t][..., None, None] * S[t]
        dk[t] = np.einsum("bhij,bhj->bhi", D, b[t][..., None] * err[t]) - np.einsum("bhij,bhj->bhi", faded, dv[t])
        D = D - np.einsum("bhi,bhj->bhij", k[t], dv[t])
        dw[t] = -(D * faded).sum((-1, -2))
        D = a[t][..., None, None] * D

    def shared(x):
        return _flat(x.reshape(T, B, H // share, share, N).sum(3))

    return shared(dr), shared(dk), _flat(dv), dw.transpose(1, 0, 2), db.transpose(1, 0, 2), D


def _act(kind, x):
    s = 1 / (1 + np.exp(-x))
    if kind == "none":
        return x, np.ones_like(x)
    return (x * s, s * (1 + x * (1 - s))) if kind == "silu" else (s, s * (1 - s))


def _norm(x, G, weight, bias, eps):
    C = x.shape[-1]
    x = np.asarray(x, np.float64).reshape(*x.shape[:-1], G, C // G)
    d = x - x.mean(-1, keepdims=True)
    inv = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    hat = (d * inv).reshape(*x.shape[:-2], C)
    wt = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    z = hat * wt + (0 if bias is None else np.asarray(bias, np.float64))
    return hat, inv, wt, z


def group_norm(x, G, weight=None, bias=None, gate=None, act="none", eps=1e-5):
    z = _norm(x, G, weight, bias, eps)[3]
    return _act(act, z)[0] if gate is None else z * _act(act, np.asarray(gate, np.float64))[0]


def group_norm_backward(x, G, weight=None, bias=None, gate=None, dy=None, act="none", eps=1e-5):
    """(dx, dweight, dbias, dgate)."""
    hat, inv, wt, z = _norm(x, G, weight, bias, eps)
    dy = np.asarray(dy, np.float64)
    value, slope = _act(act, z if gate is None else np.asarray(gate, np.float64))
    dz = dy * (slope if gate is None else value)
    dgate = None if gate is None else dy * z * slope
    shape = (*x.shape[:-1], G, x.shape[-1] // G)
    h, g = hat.reshape(shape), (dz * wt).reshape(shape)
    dx = inv * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx.reshape(x.shape), (dz * hat).sum(rows), dz.sum(rows), dgate

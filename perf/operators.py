"""Cases that measure the gated delta rule (forward, single-token step, backward) and the group norm with an activation.

Each case names an operator (``op``) with its sizes.  ``run`` makes the call a user makes where ``own`` is true, and
otherwise computes the same result from elementary torch operations in 32 bits.  ``exact`` computes it in 64 bits,
token by token, from the operators' definitions.
"""
import math

import torch

own = False

DEV = "cuda"
BIG = 1e4       # e^-BIG is 0: a decay rate of infinity (a reset of the state) counts as this much
CHUNK = 64      # tokens per chunk of the plain delta rule
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _delta(name, op, B, T, Hk, H, N, dtype, state=True, resets=False):
    return {"name": name, "op": op, "B": B, "T": T, "Hk": Hk, "H": H, "N": N, "dtype": dtype, "state": state,
            "resets": resets}


def _norm(name, op, B, T, C, G, dtype, act="silu", gate=True):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "G": G, "dtype": dtype, "act": act, "gate": gate}


def listed():
    return [
        # the shortest prompt: a few tokens through two small heads, where the call's latency is all
        _delta("delta_fwd_prompt", "fwd", 1, 17, 2, 2, 32, "f32"),
        # the training configuration's layer: width 2048 in 32 heads of 64, context 4096, 8 sequences
        _delta("delta_fwd_layer", "fwd", 8, 4096, 32, 32, 64, "bf16", state=False),
        # the wide layer: width 5120 in 80 heads of 64, context 8192, documents packed (the state is reset at each)
        _delta("delta_fwd_wide_packed", "fwd", 4, 8192, 80, 80, 64, "bf16", resets=True),
        # a chunk of a long document on one sequence, wide heads, two value heads to a key head, an odd length
        _delta("delta_fwd_shared", "fwd", 1, 4095, 16, 32, 128, "bf16"),
        # a small ragged training batch in 32 bits
        _delta("delta_bwd_ragged", "bwd", 2, 130, 4, 4, 64, "f32"),
        # the training configuration's layer, reverse mode
        _delta("delta_bwd_layer", "bwd", 8, 4096, 32, 32, 64, "bf16", state=False),
        # wide heads that share keys, reverse mode, an odd length and packed documents
        _delta("delta_bwd_shared", "bwd", 1, 2047, 8, 16, 128, "bf16", resets=True),
        # one layer of one conversation: the smallest decode call
        {"name": "delta_step_one", "op": "step", "L": 1, "B": 1, "Hk": 32, "H": 32, "N": 64, "dtype": "bf16"},
        # 24 layers x 256 sequences of width 4096: the batched decode step
        {"name": "delta_step_batch", "op": "step", "L": 24, "B": 256, "Hk": 64, "H": 64, "N": 64, "dtype": "bf16"},
        # the norm of one decode step's heads, gated
        _norm("norm_decode", "norm", 256, 1, 4096, 64, "bf16"),
        # the training layer's norm and gate
        _norm("norm_layer", "norm", 8, 4096, 2048, 32, "bf16"),
        # the training layer's norm and gate, reverse mode
        _norm("norm_bwd_layer", "norm_bwd", 8, 4096, 2048, 32, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("fwd", "bwd"):
        N = rng.choice([32, 64, 64, 128])
        Hk, ratio = _log(rng, 1, 32), rng.choice([1, 1, 2, 4])
        H = Hk * ratio
        B, T = _log(rng, 1, 8), _log(rng, 1, 16384)
        most = 4 * 8192 * 80 * 64 * 64 if op == "fwd" else 8 * 4096 * 32 * 64 * 64
        T = max(1, min(T, most // (2 * B * H * N * max(N, 64))))
        return {"op": op, "B": B, "T": T, "Hk": Hk, "H": H, "N": N, "dtype": dtype,
                "state": rng.random() < 0.7, "resets": rng.random() < 0.4}
    if op == "step":
        N = rng.choice([32, 64, 64, 128])
        Hk, ratio = _log(rng, 1, 32), rng.choice([1, 1, 2, 4])
        L, B = _log(rng, 1, 24), _log(rng, 1, 256)
        most = 24 * 256 * 64 * 64 * 64
        B = max(1, min(B, most // (L * Hk * ratio * N * N)))
        return {"op": op, "L": L, "B": B, "Hk": Hk, "H": Hk * ratio, "N": N, "dtype": dtype}
    G, size = _log(rng, 1, 80), rng.choice([rng.randint(8, 130), 32, 64, 64, 128])
    B, T = _log(rng, 1, 64), _log(rng, 1, 8192)
    T = max(1, min(T, 8 * 4096 * 2048 // (2 * B * G * size)))
    return {"op": op, "B": B, "T": T, "C": G * size, "G": G, "dtype": dtype,
            "act": rng.choice(["none", "silu", "silu", "sigmoid"]), "gate": rng.random() < 0.6}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    if case["op"] in ("norm", "norm_bwd"):
        B, T, C = case["B"], case["T"], case["C"]
        # heads' outputs differ in size by the state they carry, and lie off zero a little
        s = {"x": randn(B, T, C, scale=2.0).add_(0.25).to(dt), "weight": 1 + 0.2 * randn(C), "bias": 0.2 * randn(C),
             "gate": randn(B, T, C, dtype=dt) if case["gate"] else None}
        if case["op"] == "norm_bwd":
            s["dy"] = randn(B, T, C, dtype=dt)
        return {"case": case, **s}
    lead = (case["L"], case["B"]) if case["op"] == "step" else (case["B"], case["T"])
    Hk, H, N = case["Hk"], case["H"], case["N"]
    r = randn(*lead, Hk * N, dtype=dt, scale=N ** -0.5)
    k = randn(*lead, Hk, N)
    k = (k / k.norm(dim=-1, keepdim=True)).reshape(*lead, Hk * N).to(dt)  # keys of length one
    v = randn(*lead, H * N, dtype=dt)
    # decay rates from a per-head level and the token's own part: states that last from one token to dozens
    level = torch.rand((*([1] * len(lead)), H), generator=gen, device=DEV) * 4 - 4
    w = torch.exp(level + 0.5 * randn(*lead, H))
    if case.get("resets"):  # a document begins: nothing of the state before it is left
        w = w.masked_fill(torch.rand((*lead, 1), generator=gen, device=DEV) < 1 / 512, math.inf)
    beta = torch.sigmoid(randn(*lead, H))
    s = {"case": case, "w": w, "beta": beta, "r": r, "k": k, "v": v}
    if case["op"] == "step":
        s["state"] = randn(*lead, H, N, N, scale=0.3)
        return s
    s["state_in"] = randn(lead[0], H, N, N, scale=0.3) if case["state"] else None
    if case["op"] == "bwd":
        s["dy"] = randn(*lead, H * N, dtype=dt)
        s["dstate_out"] = randn(lead[0], H, N, N, scale=0.3) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A (..., L, L), L a power of two: the inverses of the diagonal blocks of
    size h give those of size 2 h, inv([[P, 0], [Q, R]]) = [[P', 0], [-R' Q P', R']]."""
    L = A.shape[-1]
    i = torch.arange(L, device=A.device)
    X = torch.eye(L, device=A.device).expand_as(A)
    h = 1
    while h < L:
        below = (i[:, None] // (2 * h) == i[None, :] // (2 * h)) & (i[:, None] // h > i[None, :] // h)
        X = X - X @ torch.where(below, A, 0.0) @ X
        h *= 2
    return X


def _plain_delta(w, beta, r, k, v, H, state_in):
    """The delta rule in chunks.  Within a chunk that starts from S the tokens' updates U solve
    (I + A) U = beta (V - e^-g K S), A[t, s] = beta_t e^-(g_t - g_s) k_t.k_s for s < t, g the running sum of w."""
    B, T, N = v.shape[0], v.shape[1], v.shape[2] // H
    share = H // (k.shape[2] // N)
    L = CHUNK
    while L // 2 >= T:
        L //= 2
    n = -(-T // L)

    def chunks(x):  # (B, T, heads, ...) -> (B, heads, n, L, ...), empty tokens behind the last
        x = torch.cat([x, x.new_zeros(B, n * L - T, *x.shape[2:])], 1) if n * L > T else x
        return x.reshape(B, n, L, *x.shape[2:]).movedim(3, 1)

    kk, rr, vv = (chunks(x.reshape(B, T, -1, N)) for x in (k, r, v))
    kk, rr = (x.repeat_interleave(share, 1) if share > 1 else x for x in (kk, rr))
    g = chunks(w.clamp(max=BIG).double()).cumsum(-1)    # 64 bits: the differences of long sums
    b = chunks(beta)
    i = torch.arange(L, device=w.device)
    gap = (g[..., :, None] - g[..., None, :]).float().masked_fill(i[:, None] < i[None, :], math.inf)
    fade = torch.exp(-gap)                              # e^-(g_t - g_s), 0 above the diagonal
    A = (b[..., None] * fade * (kk @ kk.transpose(-1, -2))).tril(-1)
    X = _inverse(A)
    eg = torch.exp(-g.float())[..., None]
    W = X @ (b[..., None] * eg * kk)
    U0 = X @ (b[..., None] * vv)
    P = fade * (rr @ kk.transpose(-1, -2))
    rg = eg * rr
    kg = fade[..., -1, :, None] * kk
    S = state_in if state_in is not None else vv.new_zeros(B, H, N, N)
    ys = []
    for c in range(n):
        U = U0[:, :, c] - W[:, :, c] @ S
        ys.append(rg[:, :, c] @ S + P[:, :, c] @ U)
        S = eg[:, :, c, -1:] * S + kg[:, :, c].transpose(-1, -2) @ U
    y = torch.stack(ys, 2).movedim(1, 3).reshape(B, n * L, H * N)[:, :T]
    return y, S


def _plain_step(s):
    case = s["case"]
    N, share, S = case["N"], case["H"] // case["Hk"], s["state"]
    k, r = (s[n].float().unflatten(-1, (-1, N)).repeat_interleave(share, 2) for n in ("k", "r"))
    v = s["v"].float().unflatten(-1, (-1, N))
    S.mul_(torch.exp(-s["w"])[..., None, None])
    u = s["beta"][..., None] * (v - (k[..., None, :] @ S)[..., 0, :])
    S.add_(k[..., :, None] * u[..., None, :])
    y = (r[..., None, :] @ S)[..., 0, :]
    return {"y": y.flatten(-2).to(s["v"].dtype), "state": S}


def _act(name, x):
    return x if name == "none" else x * torch.sigmoid(x) if name == "silu" else torch.sigmoid(x)


def _plain_norm(case, x, weight, bias, gate):
    xg = x.unflatten(-1, (case["G"], -1))
    d = xg - xg.mean(-1, keepdim=True)
    z = (d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)).flatten(-2) * weight + bias
    return _act(case["act"], z) if gate is None else z * _act(case["act"], gate)


def _leaf(x):
    return None if x is None else x.float().requires_grad_()


def _gradients(out, dout, names, leaves, types):
    have = [n for n in names if leaves[n] is not None]
    grads = torch.autograd.grad(out, [leaves[n] for n in have], dout)
    return {"d" + n: g.to(types[n]) for n, g in zip(have, grads)}


def _plain(s):
    case = s["case"]
    if case["op"] == "fwd":
        y, S = _plain_delta(s["w"], s["beta"], s["r"].float(), s["k"].float(), s["v"].float(), case["H"],
                            s["state_in"])
        return {"y": y.to(s["v"].dtype), "state": S}
    if case["op"] == "step":
        return _plain_step(s)
    if case["op"] == "norm":
        g = s["gate"]
        y = _plain_norm(case, s["x"].float(), s["weight"], s["bias"], None if g is None else g.float())
        return {"y": y.to(s["x"].dtype)}
    if case["op"] == "norm_bwd":
        x = {n: _leaf(s[n]) for n in ("x", "weight", "bias", "gate")}
        y = _plain_norm(case, x["x"], x["weight"], x["bias"], x["gate"])
        types = {"x": s["x"].dtype, "gate": s["x"].dtype, "weight": torch.float32, "bias": torch.float32}
        return _gradients([y], [s["dy"].float()], list(x), x, types)
    x = {n: _leaf(s[n]) for n in ("r", "k", "v", "w", "beta", "state_in")}
    if x["state_in"] is None:
        B, H, N = case["B"], case["H"], case["N"]
        x["state_in"] = torch.zeros((B, H, N, N), device=DEV, requires_grad=True)
    y, S = _plain_delta(x["w"], x["beta"], x["r"], x["k"], x["v"], case["H"], x["state_in"])
    out, dout = [y], [s["dy"].float()]
    if s["dstate_out"] is not None:
        out, dout = [y, S], [s["dy"].float(), s["dstate_out"]]
    types = {n: s["v"].dtype if n in "rkv" else torch.float32 for n in x}
    return _gradients(out, dout, list(x), x, types)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if not own:
        return _plain(s)
    import rwkv_wkv_recurrence_02_b200 as wkv
    case = s["case"]
    if case["op"] == "fwd":
        y, S = wkv.wkv_delta_forward(s["w"], s["beta"], s["r"], s["k"], s["v"], case["H"], s["state_in"])
        return {"y": y, "state": S}
    if case["op"] == "step":
        y = wkv.wkv_delta_step(s["w"], s["beta"], s["r"], s["k"], s["v"], s["state"])
        return {"y": y, "state": s["state"]}
    if case["op"] == "bwd":
        g = wkv.wkv_delta_backward(s["w"], s["beta"], s["r"], s["k"], s["v"], case["H"], s["state_in"], dy=s["dy"],
                                   dstate_out=s["dstate_out"])
        return dict(zip(("dr", "dk", "dv", "dw", "dbeta", "dstate_in"), g))
    if case["op"] == "norm":
        return {"y": wkv.wkv_group_norm(s["x"], case["G"], s["weight"], s["bias"], s["gate"], act=case["act"],
                                        eps=1e-5)}
    g = wkv.wkv_group_norm_backward(s["x"], case["G"], s["weight"], s["bias"], s["gate"], dy=s["dy"], act=case["act"],
                                    eps=1e-5)
    return {n: x for n, x in zip(("dx", "dweight", "dbias", "dgate"), g) if x is not None}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("norm", "norm_bwd"):
        n = case["B"] * case["T"] * case["C"]
        if case["op"] == "norm":
            return {"bytes": n * e * (3 if case["gate"] else 2) + 8 * case["C"], "flops": 12 * n}
        return {"bytes": n * e * (5 if case["gate"] else 3) + 16 * case["C"], "flops": 30 * n}
    tokens = case["B"] * (case["L"] if case["op"] == "step" else case["T"])
    keys, values, scalars = tokens * case["Hk"] * case["N"], tokens * case["H"] * case["N"], tokens * case["H"]
    if case["op"] == "step":
        return {"bytes": e * (2 * keys + 2 * values) + 8 * scalars + 8 * values * case["N"],
                "flops": 6 * values * case["N"]}
    state = 4 * case["B"] * case["H"] * case["N"] ** 2 * (2 if case["state"] else 1)
    if case["op"] == "fwd":
        # S^T k, the update and S^T r: three multiply-adds for each value of the state
        return {"bytes": e * (2 * keys + 2 * values) + 8 * scalars + state, "flops": 6 * values * case["N"]}
    # the updates again (2), the gradient state's walk (4), the state's walk (3)
    return {"bytes": e * (4 * keys + 3 * values) + 16 * scalars + 2 * state, "flops": 18 * values * case["N"]}


# ---------------------------------------------------------------------------
# 64 bits, token by token
# ---------------------------------------------------------------------------
def _exact_heads(x, share, N):
    """(B, T, heads N) -> (T, B, H, N) in 64 bits."""
    return x.double().unflatten(-1, (-1, N)).repeat_interleave(share, 2).transpose(0, 1).contiguous()


def _advance(S, a, b, k, v):
    """One token on states S (B, H, N, N): the new states and e = v - a S^T k."""
    S = a[..., None, None] * S
    e = v - (S * k[..., :, None]).sum(-2)
    return S + k[..., :, None] * (b[..., None] * e)[..., None, :], e


def _exact_bwd(case, s):
    N, H, share = case["N"], case["H"], case["H"] // case["Hk"]
    r, k = (_exact_heads(s[n], share, N) for n in ("r", "k"))
    v, dy = (_exact_heads(s[n], 1, N) for n in ("v", "dy"))
    a, b = torch.exp(-s["w"].double()).transpose(0, 1), s["beta"].double().transpose(0, 1)
    T, B = v.shape[:2]
    S = torch.zeros((B, H, N, N), dtype=torch.float64, device=DEV) if s["state_in"] is None else s["state_in"].double()
    D = torch.zeros_like(S) if s["dstate_out"] is None else s["dstate_out"].double()
    seg, kept = 32, []
    for t in range(T):
        if t % seg == 0:
            kept.append(S)
        S, _ = _advance(S, a[t], b[t], k[t], v[t])
    dr, dk, dv = (torch.empty_like(v) for _ in range(3))
    da, db = torch.empty_like(a), torch.empty_like(b)
    for c in reversed(range(len(kept))):
        states, errs = [kept[c]], []
        for t in range(c * seg, min(T, c * seg + seg)):
            S, e = _advance(states[-1], a[t], b[t], k[t], v[t])
            states.append(S)
            errs.append(e)
        for t in reversed(range(c * seg, min(T, c * seg + seg))):
            old, new, e = states[t - c * seg], states[t - c * seg + 1], errs[t - c * seg]
            D = D + r[t][..., :, None] * dy[t][..., None, :]
            dr[t] = (new * dy[t][..., None, :]).sum(-1)
            du = (D * k[t][..., :, None]).sum(-2)
            db[t] = (du * e).sum(-1)
            de = b[t][..., None] * du
            dv[t] = de
            faded = a[t][..., None, None] * old
            dk[t] = (D * (b[t][..., None] * e)[..., None, :]).sum(-1) - (faded * de[..., None, :]).sum(-1)
            D = D - k[t][..., :, None] * de[..., None, :]  # with respect to a S
            da[t] = (D * old).sum((-1, -2))
            D = a[t][..., None, None] * D
    back = lambda x: x.transpose(0, 1).flatten(2)  # noqa: E731
    shared = lambda x: back(x.unflatten(2, (-1, share)).sum(3))  # noqa: E731
    return {"dr": shared(dr), "dk": shared(dk), "dv": back(dv), "dw": -(a * da).transpose(0, 1).contiguous(),
            "dbeta": db.transpose(0, 1).contiguous(), "dstate_in": D}


def _exact_norm(case, s, dy):
    B, T, C, G = case["B"], case["T"], case["C"], case["G"]
    x = s["x"].double().view(B, T, G, C // G)
    var, mean = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
    inv = 1 / torch.sqrt(var + 1e-5)
    hat = (x - mean) * inv
    wt, z = s["weight"].double(), hat.view(B, T, C) * s["weight"].double() + s["bias"].double()
    arg = z if s["gate"] is None else s["gate"].double()
    sig = 1 / (1 + torch.exp(-arg))
    value = {"none": arg, "silu": arg * sig, "sigmoid": sig}[case["act"]]
    if dy is None:
        return {"y": value if s["gate"] is None else z * value}
    slope = {"none": torch.ones_like(arg), "silu": sig * (1 + arg * (1 - sig)), "sigmoid": sig * (1 - sig)}[case["act"]]
    dy = dy.double()
    dz = dy * slope if s["gate"] is None else dy * value
    out = {"dweight": (dz * hat.view(B, T, C)).sum((0, 1)), "dbias": dz.sum((0, 1))}
    dh = (dz * wt).view(B, T, G, C // G)
    out["dx"] = (inv * (dh - dh.mean(-1, keepdim=True) - hat * (dh * hat).mean(-1, keepdim=True))).view(B, T, C)
    if s["gate"] is not None:
        out["dgate"] = dy * z * slope
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, s, s.get("dy"))
    if case["op"] == "bwd":
        return _exact_bwd(case, s)
    N, H, share = case["N"], case["H"], case["H"] // case["Hk"]
    if case["op"] == "step":
        flat = lambda x, h: x.double().unflatten(-1, (-1, N)).repeat_interleave(h, 2)  # noqa: E731
        S, _ = _advance(s.pop("state").double(), torch.exp(-s["w"].double()), s["beta"].double(), flat(s["k"], share),
                        flat(s["v"], 1))
        return {"y": (S * flat(s["r"], share)[..., :, None]).sum(-2).flatten(-2), "state": S}
    r, k, v = _exact_heads(s["r"], share, N), _exact_heads(s["k"], share, N), _exact_heads(s["v"], 1, N)
    a, b = torch.exp(-s["w"].double()).transpose(0, 1), s["beta"].double().transpose(0, 1)
    S = torch.zeros((v.shape[1], H, N, N), dtype=torch.float64, device=DEV)
    S = S if s["state_in"] is None else s["state_in"].double()
    y = torch.empty_like(v)
    for t in range(v.shape[0]):
        S, _ = _advance(S, a[t], b[t], k[t], v[t])
        y[t] = (S * r[t][..., :, None]).sum(-2)
    return {"y": y.transpose(0, 1).flatten(2), "state": S}

"""The gated delta rule (forward, step, backward) against the fp64 oracle.

Errors are measured against the largest magnitude of the tensor (of dw:
of what its sum adds up, which can cancel).  Tolerance of float32
arithmetic: 2e-5, the bound of this library's other float32 results: every
token rounds sums of at most N terms, spread over lanes, at about
(N / 8 + 8) 2^-24 = 1.4e-6 for N = 128, and states that last about 50 tokens
keep the errors of so many, of either sign: 1.4e-6 sqrt(50) = 1e-5.  A
bfloat16 output adds half a step of its own, 2^-8 of its value."""
import numpy as np
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv
from oracle import delta as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dr", "dk", "dv", "dw", "dbeta", "dstate_in")


def case(B, T, Hk, H, N, dtype, state=True, seed=0, w=None, beta=None, lead=None):
    g = torch.Generator().manual_seed(seed + 1000 * T + N)
    lead = lead or (B, T)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    k = n(*lead, Hk, N)
    k = (k / k.norm(dim=-1, keepdim=True)).reshape(*lead, Hk * N)
    d = {"w": torch.exp(torch.rand((*lead, H), generator=g) * 4 - 3.5) if w is None else torch.full((*lead, H), float(w)),
         "beta": torch.sigmoid(n(*lead, H)) if beta is None else torch.full((*lead, H), float(beta)),
         "r": (n(*lead, Hk * N) * N ** -0.5).to(dtype), "k": k.to(dtype), "v": n(*lead, H * N).to(dtype)}
    d = {a: x.to(DEV) for a, x in d.items()}
    d["state_in"] = (0.3 * n(B, H, N, N)).to(DEV) if state else None
    d["dy"] = n(*lead, H * N).to(dtype).to(DEV)
    d["ds"] = (0.3 * n(B, H, N, N)).to(DEV)
    return d


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def ref_fwd(d, H):
    return D.delta_forward(*(f64(d[n]) for n in ("w", "beta", "r", "k", "v")), H, f64(d["state_in"]))


def ref_bwd(d, H, ds=True):
    return D.delta_backward(*(f64(d[n]) for n in ("w", "beta", "r", "k", "v")), H, f64(d["state_in"]), f64(d["dy"]),
                            f64(d["ds"]) if ds else None)


def forward(d, H, **kw):
    return wkv.wkv_delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], H, d["state_in"], **kw)


def backward(d, H, ds=True, **kw):
    return wkv.wkv_delta_backward(d["w"], d["beta"], d["r"], d["k"], d["v"], H, d["state_in"], dy=d["dy"],
                                  dstate_out=d["ds"] if ds else None, **kw)


def close(got, ref, name="", scale=None):
    g = f64(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g)), name
    if not g.size:
        return
    scale = max(np.abs(ref).max() if scale is None else scale, 1e-30)
    tol = 2e-5 * scale + (2.0 ** -8 * np.abs(ref) if got.dtype == BF16 else 0)
    err = np.abs(g - ref)
    assert np.all(err <= tol), f"{name}: {np.max(err / scale):.3e} of the largest magnitude"


SHAPES = [
    # B, T, Hk, H, N, dtype, state
    (1, 1, 1, 1, 32, F32, False),
    (1, 1, 1, 2, 64, BF16, True),
    (2, 2, 1, 1, 128, F32, True),
    (2, 15, 2, 2, 32, BF16, True),
    (1, 16, 1, 1, 64, F32, False),
    (3, 17, 1, 3, 64, F32, True),       # one key head under three value heads
    (1, 63, 2, 4, 128, BF16, True),
    (1, 64, 1, 1, 32, F32, True),
    (2, 65, 2, 2, 64, BF16, False),
    (1, 130, 1, 2, 128, F32, True),
    (2, 200, 3, 3, 32, F32, True),
    (1, 257, 2, 4, 64, F32, True),
    (1, 300, 5, 5, 64, BF16, True),
]


@pytest.mark.parametrize("B,T,Hk,H,N,dtype,state", SHAPES)
def test_forward(B, T, Hk, H, N, dtype, state):
    d = case(B, T, Hk, H, N, dtype, state)
    y, s = forward(d, H)
    yr, sr = ref_fwd(d, H)
    close(y, yr, "y")
    close(s, sr, "state")
    # no state wanted: the same outputs
    y2, none = forward(d, H, want_state=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("B,T,Hk,H,N,dtype,state", SHAPES)
def test_backward(B, T, Hk, H, N, dtype, state):
    d = case(B, T, Hk, H, N, dtype, state)
    got = backward(d, H)
    for name, g, r in zip(NAMES, got, ref_bwd(d, H)):
        close(g, r, name)
    again = backward(d, H)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for name, g, r in zip(NAMES, backward(d, H, ds=False, want_dstate_in=False), ref_bwd(d, H, ds=False)):
        if name == "dstate_in":
            assert g is None
        else:
            close(g, r, name)
    if not state:
        assert torch.count_nonzero(backward(d, H)[3][:, 0]) == 0   # nothing to decay before the first token


# strong decays and resets leave a block's product of decays, products at the
# edge of the scaled form (16 tokens of 3.4: 2^-78; of 3.6: 2^-83) and none
@pytest.mark.parametrize("w", [0.0, 1e-6, 3.4, 3.6, 30.0, 200.0, 1e30, float("inf")])
@pytest.mark.parametrize("N", [32, 64, 128])
def test_decays(w, N):
    d = case(1, 40, 1, 2, N, F32, w=w)
    y, s = forward(d, 2)
    yr, sr = ref_fwd(d, 2)
    close(y, yr, "y")
    close(s, sr, "state")
    ref = ref_bwd(d, 2)
    # dw is a difference of sums of r . dr and dv . v: its errors are theirs
    terms = np.abs((ref[0] * f64(d["r"])).sum(-1)).max() + np.abs((ref[2] * f64(d["v"])).sum(-1)).max()
    for name, g, r in zip(NAMES, backward(d, 2), ref):
        close(g, r, name, scale=max(terms, np.abs(r).max()) if name == "dw" else None)
    if w >= 200:
        assert torch.count_nonzero(backward(d, 2)[3]) == 0


def test_resets_in_the_middle():
    d = case(2, 100, 2, 4, 64, F32)
    d["w"][:, 37] = float("inf")
    d["w"][0, 64] = float("inf")
    d["w"][1, 99, 2] = float("inf")
    y, s = forward(d, 4)
    yr, sr = ref_fwd(d, 4)
    close(y, yr, "y")
    close(s, sr, "state")
    for name, g, r in zip(NAMES, backward(d, 4), ref_bwd(d, 4)):
        close(g, r, name)


@pytest.mark.parametrize("N,dtype", [(32, F32), (64, BF16), (128, F32)])
def test_padding_leaves_the_state(N, dtype):
    d = case(2, 50, 1, 2, N, dtype)
    d["w"][:, 31:] = 0
    d["beta"][:, 31:] = 0
    cut = {n: x[:, :31].contiguous() if n not in ("state_in", "ds") else x for n, x in d.items()}
    s, s_cut = forward(d, 2)[1], forward(cut, 2)[1]
    close(s, f64(s_cut), "state")
    for name, g, r in zip(NAMES, backward(d, 2), ref_bwd(d, 2)):
        close(g, r, name)


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0, -0.5])
def test_learning_rates(beta):
    d = case(1, 70, 1, 1, 64, F32, beta=beta)
    close(forward(d, 1)[0], ref_fwd(d, 1)[0], "y")
    for name, g, r in zip(NAMES, backward(d, 1), ref_bwd(d, 1)):
        close(g, r, name)


def test_no_tokens():
    d = case(2, 0, 1, 2, 64, F32)
    y, s = forward(d, 2)
    assert y.shape == (2, 0, 128) and torch.equal(s, d["state_in"])
    assert torch.count_nonzero(wkv.wkv_delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], 2)[1]) == 0
    g = backward(d, 2)
    assert torch.equal(g[5], d["ds"]) and g[0].shape == (2, 0, 64)
    e = case(0, 5, 1, 2, 64, F32)
    assert forward(e, 2)[0].shape == (0, 5, 128)


@pytest.mark.parametrize("N,dtype", [(32, BF16), (64, F32), (128, F32)])
def test_chunks_in_place_and_steps_equal_one_pass(N, dtype):
    d = case(2, 45, 2, 4, N, dtype)
    yr, sr = ref_fwd(d, 4)
    st, ys = d["state_in"].clone(), []
    for t0, t1 in ((0, 1), (1, 17), (17, 17), (17, 45)):
        c = {n: d[n][:, t0:t1].contiguous() for n in ("w", "beta", "r", "k", "v")}
        y, out = wkv.wkv_delta_forward(c["w"], c["beta"], c["r"], c["k"], c["v"], 4, st, state_out=st)
        assert out is st
        ys.append(y)
    close(torch.cat(ys, 1), yr, "y")
    close(st, sr, "state")
    st, ys = d["state_in"].clone()[None], []
    for t in range(45):
        c = {n: d[n][None, :, t].contiguous() for n in ("w", "beta", "r", "k", "v")}
        ys.append(wkv.wkv_delta_step(c["w"], c["beta"], c["r"], c["k"], c["v"], st)[0])
    close(torch.stack(ys, 1), yr, "y of steps")
    close(st[0], sr, "state of steps")


@pytest.mark.parametrize("L,B,Hk,H,N,dtype", [(1, 1, 1, 1, 32, F32), (2, 3, 1, 3, 64, BF16), (3, 1, 2, 2, 128, F32),
                                              (1, 5, 2, 4, 128, BF16), (4, 2, 3, 3, 32, BF16)])
def test_step(L, B, Hk, H, N, dtype):
    d = case(L * B, 1, Hk, H, N, dtype, lead=(L, B))
    d["w"][0, 0, 0] = float("inf")
    st = d["state_in"].view(L, B, H, N, N)
    one = lambda x: f64(x).reshape(L * B, 1, -1)  # noqa: E731
    yr, sr = D.delta_forward(*(one(d[n]) for n in ("w", "beta", "r", "k", "v")), H, f64(d["state_in"]))
    y = wkv.wkv_delta_step(d["w"], d["beta"], d["r"], d["k"], d["v"], st)
    close(y.view(L * B, 1, -1), yr, "y")
    close(st.view(L * B, H, N, N), sr, "state")


def odd(t):
    """The same values one element behind an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("N,dtype", [(32, BF16), (64, BF16), (64, F32), (128, F32)])
def test_unaligned(N, dtype):
    d = case(2, 37, 1, 2, N, dtype)
    o = {n: odd(x) for n, x in d.items()}
    for a, b in zip(forward(d, 2) + backward(d, 2), forward(o, 2) + backward(o, 2)):
        assert torch.equal(a, b)
    st, so = d["state_in"].clone()[None], odd(d["state_in"][None])
    c = {n: d[n][None, :, 0].contiguous() for n in ("w", "beta", "r", "k", "v")}
    ya = wkv.wkv_delta_step(c["w"], c["beta"], c["r"], c["k"], c["v"], st)
    yb = wkv.wkv_delta_step(*(odd(c[n]) for n in ("w", "beta", "r", "k", "v")), so)
    assert torch.equal(ya, yb) and torch.equal(st, so)


def test_refuses_what_it_cannot_read():
    d = case(1, 8, 1, 1, 64, F32)
    with pytest.raises(ValueError, match="contiguous"):
        wkv.wkv_delta_forward(d["w"], d["beta"], d["r"], d["k"].transpose(1, 2).contiguous().transpose(1, 2), d["v"], 1)
    with pytest.raises(TypeError):
        wkv.wkv_delta_forward(d["w"].double(), d["beta"], d["r"], d["k"], d["v"], 1)
    with pytest.raises(TypeError):
        wkv.wkv_delta_forward(d["w"], d["beta"], d["r"].bfloat16(), d["k"], d["v"], 1)
    with pytest.raises(wkv.WkvError, match="SHAPE"):
        x = torch.zeros(1, 8, 48, device=DEV)
        wkv.wkv_delta_forward(d["w"], d["beta"], x, x, x, 1)
    with pytest.raises(wkv.WkvError, match="ALIAS"):
        forward(d, 1, y=d["v"])
    with pytest.raises(ValueError, match="state_in"):
        wkv.wkv_delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], 1, torch.zeros(1, 1, 32, 32, device=DEV))


def test_another_stream_and_two_calls_at_once():
    d, e = case(2, 90, 2, 2, 64, BF16, seed=1), case(1, 70, 1, 2, 64, BF16, seed=2)
    want = [backward(d, 2), backward(e, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [backward(x, 2, stream=s) for x, s in zip((d, e), streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    # and as the current stream, with one workspace for calls in order
    ws = wkv.Workspace()
    with torch.cuda.stream(streams[0]):
        got = [backward(x, 2, workspace=ws) for x in (d, e, d)]
    torch.cuda.synchronize()
    for a, b in zip(want + want[:1], got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_of_forward_and_backward_replay():
    d, e = case(1, 50, 1, 2, 64, BF16, seed=3), case(1, 66, 1, 2, 64, BF16, seed=4)
    run = lambda x: forward(x, 2) + backward(x, 2)  # noqa: E731
    want = [run(d), run(e)]
    graphs, outs = [], []
    for x in (d, e):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(x))
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    # new inputs in the captured tensors
    d["v"].copy_(-d["v"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(run(d), outs[0]))


def test_offsets_beyond_32_bits():
    """The last sequence of a call of over 2^31 values equals a call of its own."""
    B, T, H, N = 513, 1024, 64, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn((B, T, H * N), generator=g, device=DEV, dtype=BF16) for _ in range(2))
    k *= N ** -0.5
    w, beta = (torch.rand((B, T, H), generator=g, device=DEV) for _ in range(2))
    y, s = wkv.wkv_delta_forward(w, beta, k, k, v, H)
    y1, s1 = wkv.wkv_delta_forward(w[-1:], beta[-1:], k[-1:], k[-1:], v[-1:], H)
    assert torch.equal(y[-1:], y1) and torch.equal(s[-1:], s1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_with_norm_and_gate(dtype):
    """The delta rule, the group norm of its heads and the gate as a layer
    runs them, forward and back through both, against the oracle's chain on
    the values the operators hand on."""
    H, N = 4, 64
    d = case(2, 77, 2, H, N, dtype, seed=8)
    gate, weight, bias = torch.randn_like(d["v"]), torch.rand(H * N, device=DEV) + 0.5, torch.randn(H * N, device=DEV)
    y, s = forward(d, H)
    o = wkv.wkv_group_norm(y, H, weight, bias, gate, act="silu")
    dx, dwt, db, dg = wkv.wkv_group_norm_backward(y, H, weight, bias, gate, dy=d["dy"], act="silu")
    got = wkv.wkv_delta_backward(d["w"], d["beta"], d["r"], d["k"], d["v"], H, d["state_in"], dy=dx, dstate_out=d["ds"])
    close(y, ref_fwd(d, H)[0], "y")
    close(o, D.group_norm(f64(y), H, f64(weight), f64(bias), f64(gate), "silu"), "o")
    for name, a, b in zip(("dx", "dweight", "dbias", "dgate"), (dx, dwt, db, dg),
                          D.group_norm_backward(f64(y), H, f64(weight), f64(bias), f64(gate), f64(d["dy"]), "silu")):
        close(a, b, name)
    for name, a, b in zip(NAMES, got, ref_bwd({**d, "dy": dx}, H)):
        close(a, b, name)


@pytest.mark.parametrize("B,T,Hk,H,N,dtype", [(7, 1100, 8, 64, 64, BF16), (11, 777, 16, 16, 128, BF16), (13, 513, 30, 60, 32, F32),
                                              (6, 2048, 50, 50, 64, F32)])
def test_walks_in_parts_equal_whole_ones(B, T, Hk, H, N, dtype):
    """More heads than the GPU holds at once go in parts of the tokens, with
    the same arithmetic: the same bits as one walk a CTA, on calls that share
    a workspace, and each sequence's as in a call of its own."""
    g = torch.Generator(device=DEV).manual_seed(B)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    d = {"w": torch.rand((B, T, H), generator=g, device=DEV), "beta": torch.rand((B, T, H), generator=g, device=DEV),
         "r": n(B, T, Hk * N).to(dtype), "k": (n(B, T, Hk * N) * N ** -0.5).to(dtype), "v": n(B, T, H * N).to(dtype),
         "state_in": n(B, H, N, N), "dy": n(B, T, H * N).to(dtype), "ds": n(B, H, N, N)}
    ws = wkv.Workspace()
    y, s = forward(d, H, use_workspace=False)
    for _ in range(2):
        y1, s1 = forward(d, H, workspace=ws)
        assert torch.equal(y, y1) and torch.equal(s, s1)
        assert ws.status() == 0
    got = backward(d, H)
    for b in (0, B // 2, B - 1):
        one = {x: t[b:b + 1].contiguous() for x, t in d.items()}
        for x, t in zip(NAMES, backward(one, H)):
            assert torch.equal(got[NAMES.index(x)][b:b + 1], t), (x, b)

"""Refusals of the gated delta rule's and the group norm's entry points on the
host: bad arguments are errors before anything is launched or written."""
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

OK, NULLPTR, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE = 0, -1, -2, -3, -4, -5, -8
F32, BF16 = 0, 1
# fake, well-aligned device addresses: every call fails its checks or is a
# no-op before it could use them
P = [(1 << 40) + (i << 32) for i in range(24)]


@pytest.fixture(scope="module")
def L():
    return wkv.lib()


def fwd(L, B=2, T=9, Hk=2, H=4, N=64, dt=BF16, w=P[0], beta=P[1], r=P[2], k=P[3], v=P[4], s_in=None, y=P[6],
        s_out=None, ws=None, nws=0):
    return L.wkv_delta_forward(B, T, Hk, H, N, dt, w, beta, r, k, v, s_in, y, s_out, ws, nws, None)


def test_forward_refusals(L):
    assert fwd(L, dt=5) == DTYPE
    for bad in ({"B": -1}, {"T": -1}, {"N": 48}, {"N": 0}, {"H": 3}, {"Hk": 0}, {"H": 0}, {"T": 1 << 60},
                {"H": 1 << 62, "Hk": 1}):
        assert fwd(L, **bad) == SHAPE, bad
    for name in ("w", "beta", "r", "k", "v", "y"):
        assert fwd(L, **{name: None}) == NULLPTR, name
    assert fwd(L, r=P[2] + 1) == ALIGN
    assert fwd(L, w=P[0] + 2) == ALIGN
    assert fwd(L, s_in=P[5] + 2) == ALIGN
    assert fwd(L, y=P[4]) == ALIAS
    assert fwd(L, y=P[3] + 64) == ALIAS
    assert fwd(L, s_out=P[0]) == ALIAS
    assert fwd(L, s_out=P[6] + 16) == ALIAS
    assert fwd(L, s_in=P[5], s_out=P[5] + 64) == ALIAS
    assert fwd(L, B=0, w=None) == OK
    assert fwd(L, T=0) == OK
    many = dict(B=40, T=2048)      # 160 heads
    need = L.wkv_delta_forward_workspace_bytes(40, 2048, 4, 64)
    assert need > 0 and L.wkv_delta_forward_workspace_bytes(2, 2048, 4, 64) == 0
    assert L.wkv_delta_forward_workspace_bytes(40, 2048, 4, 63) == 0
    assert fwd(L, ws=P[8] + 8, nws=need, **many) == ALIGN
    assert fwd(L, ws=P[6], nws=need, **many) == ALIAS
    assert fwd(L, ws=P[5], nws=need, s_in=P[5], **many) == ALIAS
    assert fwd(L, T=0, s_in=P[5], s_out=P[5]) == OK


def step(L, Lr=2, B=3, Hk=2, H=4, N=64, dt=F32, w=P[0], beta=P[1], r=P[2], k=P[3], v=P[4], s=P[5], y=P[6]):
    return L.wkv_delta_step(Lr, B, Hk, H, N, dt, w, beta, r, k, v, s, y, None)


def test_step_refusals(L):
    assert step(L, dt=9) == DTYPE
    for bad in ({"Lr": -1}, {"B": -1}, {"N": 65}, {"Hk": 3}, {"B": 1 << 62}):
        assert step(L, **bad) == SHAPE, bad
    for name in ("w", "beta", "r", "k", "v", "s", "y"):
        assert step(L, **{name: None}) == NULLPTR, name
    assert step(L, k=P[3] + 2) == ALIGN
    assert step(L, s=P[4]) == ALIAS
    assert step(L, y=P[5] + 4) == ALIAS
    assert step(L, Lr=0) == OK


def bwd(L, B=2, T=9, Hk=2, H=4, N=64, dt=BF16, ws=P[20], nws=1 << 30, **kw):
    a = dict(zip(("w", "beta", "r", "k", "v", "s_in", "dy", "ds", "dr", "dk", "dv", "dw", "dbeta", "dsi"), P))
    a.update(kw)
    return L.wkv_delta_backward(B, T, Hk, H, N, dt, *a.values(), ws, nws, None)


def test_backward_refusals(L):
    assert bwd(L, dt=2) == DTYPE
    assert bwd(L, N=16) == SHAPE
    for name in ("w", "beta", "r", "k", "v", "dy", "dr", "dk", "dv", "dw", "dbeta"):
        assert bwd(L, **{name: None}) == NULLPTR, name
    need = L.wkv_delta_backward_workspace_bytes(2, 9, 2, 4, 64)
    assert need > 0
    assert bwd(L, nws=need - 1) == WORKSPACE
    assert bwd(L, ws=None) == WORKSPACE
    assert bwd(L, ws=P[20] + 16) == ALIGN
    assert bwd(L, dr=P[9]) == ALIAS      # dk's
    assert bwd(L, dv=P[6]) == ALIAS      # dy's
    assert bwd(L, dsi=P[7]) == ALIAS     # dstate_out's
    assert bwd(L, dsi=P[5]) == ALIAS     # state_in's
    assert bwd(L, dw=P[20] + 256) == ALIAS
    assert L.wkv_delta_backward_workspace_bytes(2, 9, 2, 4, 63) == 0
    assert L.wkv_delta_backward_workspace_bytes(-2, 9, 2, 4, 64) == 0


def norm(L, rows=4, C=96, G=3, dt=BF16, act=1, eps=1e-5, x=P[0], wt=P[1], b=P[2], gate=P[3], y=P[4]):
    return L.wkv_group_norm(rows, C, G, dt, act, eps, x, wt, b, gate, y, None)


def test_norm_refusals(L):
    assert norm(L, dt=3) == DTYPE
    for bad in ({"G": 5}, {"G": 0}, {"G": -3}, {"rows": -1}, {"act": 3}, {"act": -1}, {"eps": 0.0},
                {"eps": float("nan")}, {"eps": float("inf")}, {"rows": 1 << 60}):
        assert norm(L, **bad) == SHAPE, bad
    assert norm(L, x=None) == NULLPTR
    assert norm(L, y=None) == NULLPTR
    assert norm(L, x=P[0] + 1) == ALIGN
    assert norm(L, wt=P[1] + 2) == ALIGN
    assert norm(L, y=P[0]) == ALIAS
    assert norm(L, y=P[3] + 2) == ALIAS
    assert norm(L, rows=0) == OK


def norm_bwd(L, rows=4, C=96, G=3, dt=BF16, act=1, eps=1e-5, ws=P[20], nws=1 << 30, **kw):
    a = dict(zip(("x", "wt", "b", "gate", "dy", "dx", "dwt", "db", "dgate"), P))
    a.update(kw)
    return L.wkv_group_norm_backward(rows, C, G, dt, act, eps, *a.values(), ws, nws, None)


def test_norm_backward_refusals(L):
    assert norm_bwd(L, dt=3) == DTYPE
    assert norm_bwd(L, G=7) == SHAPE
    for name in ("x", "dy", "dx", "dgate"):
        assert norm_bwd(L, **{name: None}) == NULLPTR, name
    assert norm_bwd(L, gate=None) == NULLPTR           # dgate of no gate
    need = L.wkv_group_norm_backward_workspace_bytes(4, 96, 3, BF16)
    assert norm_bwd(L, nws=need - 1) == WORKSPACE
    assert norm_bwd(L, ws=None) == WORKSPACE
    assert norm_bwd(L, dx=P[0]) == ALIAS
    assert norm_bwd(L, dgate=P[5]) == ALIAS
    assert L.wkv_group_norm_backward_workspace_bytes(4, 96, 5, BF16) == 0


def test_binding_refuses_host_tensors_and_shapes():
    r = torch.zeros(1, 2, 64)
    s = torch.zeros(1, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        wkv.wkv_delta_forward(s, s, r, r, r, 1)
    with pytest.raises(ValueError, match="heads"):
        wkv.wkv_delta_forward(s, s, r, r, r, 3)
    with pytest.raises(ValueError, match="share"):
        wkv.wkv_delta_forward(s, s, r, torch.zeros(1, 2, 48), r, 2)
    with pytest.raises(ValueError, match="three dimensions"):
        wkv.wkv_delta_backward(s, s, r, r[0], r, 1, dy=r)
    with pytest.raises(ValueError, match="state"):
        wkv.wkv_delta_step(s, s, r, r, r, torch.zeros(1, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        wkv.wkv_group_norm(r, 1)
    with pytest.raises(ValueError, match="groups"):
        wkv.wkv_group_norm(r, 3)
    with pytest.raises(ValueError, match="act"):
        wkv.wkv_group_norm(r, 2, act="relu")

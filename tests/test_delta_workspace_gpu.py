"""Workspaces of the delta rule and the group norm: one shared with
wkv_forward's look-back, the error word, and a wait between a walk's parts
that runs out."""
import os
import subprocess
import sys

import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_workspace_shared_with_the_look_back():
    """Calls that leave their own contents in a workspace come between two
    look-back calls of one workspace: the same bits, and no error."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, device=dev)
    T, C, H, N = 64 * 40, 64, 2, 32
    w, u, k, v = torch.exp(n(C)), n(C), n(1, T, C), n(1, T, C)
    ws = wkv.Workspace()
    y0, s0 = wkv.wkv_forward(w, u, k, v, workspace=ws)
    dw, db = torch.exp(n(1, 99, H)), torch.sigmoid(n(1, 99, H))
    dr, dk, dv, dy = (0.2 * n(1, 99, H * N) for _ in range(4))
    g0 = wkv.wkv_delta_backward(dw, db, dr, dk, dv, H, dy=dy)
    x, gate, gy = n(50, 96), n(50, 96), n(50, 96)
    one = torch.ones(96, device=dev)
    b0 = wkv.wkv_group_norm_backward(x, 3, one, one, gate, dy=gy, act="silu")
    for _ in range(2):
        g1 = wkv.wkv_delta_backward(dw, db, dr, dk, dv, H, dy=dy, workspace=ws)
        b1 = wkv.wkv_group_norm_backward(x, 3, one, one, gate, dy=gy, act="silu", workspace=ws)
        y1, s1 = wkv.wkv_forward(w, u, k, v, workspace=ws)
        for a, b in zip((y0, s0, *g0, *b0), (y1, s1, *g1, *b1)):
            assert torch.equal(a, b)
        assert ws.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["forward", "backward"])
def test_c_workspace_keeps_its_error_word(op):
    """The first 256 bytes of a workspace stay as wkv_workspace_init left them."""
    import ctypes
    dev = torch.device("cuda")
    B, T, H, N = 3, 512, 100, 64      # walks in parts
    L = wkv.lib()
    nbytes = (L.wkv_delta_forward_workspace_bytes(B, T, H, N) if op == "forward"
              else L.wkv_delta_backward_workspace_bytes(B, T, H, H, N))
    buf = torch.full((nbytes + 256,), 0x5A, dtype=torch.uint8, device=dev)
    ptr = (buf.data_ptr() + 255) & ~255
    assert L.wkv_workspace_init(ptr, 256, None) == 0
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)
    f = lambda *s: torch.zeros(s, device=dev)
    w, beta, r, k, v, dy, y = f(B, T, H), f(B, T, H), *(z(B, T, H * N) for _ in range(5))
    p = lambda t: t.data_ptr()
    if op == "forward":
        rc = L.wkv_delta_forward(B, T, H, H, N, wkv.WKV_BF16, p(w), p(beta), p(r), p(k), p(v), None, p(y), None, ptr, nbytes, None)
    else:
        o = [z(B, T, H * N) for _ in range(3)] + [f(B, T, H) for _ in range(2)]
        rc = L.wkv_delta_backward(B, T, H, H, N, wkv.WKV_BF16, p(w), p(beta), p(r), p(k), p(v), None, p(dy), None,
                                  *map(p, o), None, ptr, nbytes, None)
    assert rc == 0
    assert L.wkv_workspace_status(ptr, None) == 0


EXPIRED = r"""
import sys, torch
sys.path.insert(0, %r)
import rwkv_wkv_recurrence_02_b200 as wkv
B, T, H, N = 3, 2048, 100, 64     # more walks than the GPU holds
dev = torch.device("cuda")
x = [torch.randn(B, T, H * N, device=dev).bfloat16() * 0.1 for _ in range(4)]
w = torch.rand(B, T, H, device=dev); beta = torch.rand(B, T, H, device=dev)
ws = wkv.Workspace()
if %r == "forward":
    out = wkv.wkv_delta_forward(w, beta, *x[:3], H, workspace=ws)
else:
    out = wkv.wkv_delta_backward(w, beta, *x[:3], H, dy=x[3], workspace=ws)
print("STATUS", ws.status(), "NAN", any(bool(torch.isnan(t).any().item()) for t in out))
ws.reset()
print("AFTER_RESET", ws.status())
"""


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["forward", "backward"])
def test_expired_wait_between_parts_is_reported(op):
    """With a limit of 1 ns the first part that is taken before the one ahead of
    it has ended gives up: an error and NaN, and no hang."""
    r = subprocess.run([sys.executable, "-c", EXPIRED % (ROOT, op)], env=dict(os.environ, WKV_WAIT_LIMIT_NS="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    out = dict(zip(r.stdout.split()[::2], r.stdout.split()[1::2]))
    assert out["STATUS"] == "-7" and out["NAN"] == "True" and out["AFTER_RESET"] == "0"

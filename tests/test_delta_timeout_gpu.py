"""A wait for the reverse mode's tensor-core products that runs out: with a limit
of 0 every batch is asked for once, while it is under way."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUN = r"""
import sys, torch
sys.path.insert(0, %r)
import rwkv_wkv_recurrence_02_b200 as wkv
from torch import isfinite
B, T, Hk, H, N = 3, 150, %d, 4, 64
g = torch.Generator(device="cuda").manual_seed(0)
n = lambda *s: torch.randn(s, generator=g, device="cuda")
w, beta = torch.exp(n(B, T, H)), torch.sigmoid(n(B, T, H))
r, k = ((0.2 * n(B, T, Hk * N)).bfloat16() for _ in range(2))
v, dy = (n(B, T, H * N).bfloat16() for _ in range(2))
ws = wkv.Workspace()
dr, dk, dv, dw, dbeta, ds = wkv.wkv_delta_backward(w, beta, r, k, v, H, dy=dy, workspace=ws)
print("STATUS", ws.status())
print("NAN", all(bool(torch.isnan(t).all()) for t in (dr, dk, dw)))
print("FINITE", all(bool(isfinite(t).all()) for t in (dv, dbeta, ds)))
ws.reset()
print("RESET", ws.status())
y, s = wkv.wkv_delta_forward(w, beta, r, k, v, H, workspace=ws)
print("FORWARD", bool(isfinite(y).all()), ws.status())
"""


@pytest.mark.gpu
@pytest.mark.parametrize("Hk", [4, 2])
def test_products_that_do_not_come(Hk):
    r = subprocess.run([sys.executable, "-c", RUN % (ROOT, Hk)], env=dict(os.environ, WKV_WAIT_LIMIT_NS="0"), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:5] == ["STATUS -7", "NAN True", "FINITE True", "RESET 0", "FORWARD True 0"]

"""A wait that ran out is reported where the call's workspace is gone: the
device's own record of the delta rule, with a limit of 0 for every wait."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUN = r"""
import sys, torch
sys.path.insert(0, %r)
import rwkv_wkv_recurrence_02_b200 as wkv
print(wkv.wkv_delta_status())
if %r == "parts":                   # four walks more than the GPU holds: the first of their parts are waited for
    B, T, H, dt = 3, 2048, 100, torch.bfloat16
else:
    B, T, H, dt = 1, 200, 2, torch.bfloat16
x = [torch.randn(B, T, H * 64, device="cuda").to(dt) * 0.1 for _ in range(4)]
w, beta = torch.rand(B, T, H, device="cuda"), torch.rand(B, T, H, device="cuda")
if %r == "parts":
    out = wkv.wkv_delta_forward(w, beta, *x[:3], H)
else:
    out = wkv.wkv_delta_backward(w, beta, *x[:3], H, dy=x[3])
print(any(bool(torch.isnan(t).any()) for t in out))
print(wkv.wkv_delta_status(), wkv.wkv_delta_status(clear=True, device="cuda:0"), wkv.wkv_delta_status())
"""


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["parts", "products"])
def test_calls_without_a_workspace(case):
    r = subprocess.run([sys.executable, "-c", RUN % (ROOT, case, case)], env=dict(os.environ, WKV_WAIT_LIMIT_NS="0"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["0", "True", "-7", "-7", "0"]

"""Calls of the delta rule and the group norm leave a workspace's first 256 bytes
as they were, whatever was in them, until there is an error."""
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

pytestmark = pytest.mark.gpu


def workspace(nbytes):
    buf = torch.randint(0, 256, (nbytes + 256,), dtype=torch.uint8, device="cuda")
    ptr = (buf.data_ptr() + 255) & ~255
    return buf, ptr, buf[ptr - buf.data_ptr():][:256]


def ptrs(*tensors):
    return [t if t is None else t.data_ptr() for t in tensors]


# 300 heads are walked in parts, 6 are not
@pytest.mark.parametrize("H", [2, 100])
@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, wkv.WKV_BF16), (torch.float32, wkv.WKV_F32)])
@pytest.mark.parametrize("op", ["forward", "backward"])
def test_delta(op, H, dtype, code):
    B, T, N, L = 3, 600, 64, wkv.lib()
    need = (L.wkv_delta_forward_workspace_bytes(B, T, H, N) if op == "forward"
            else L.wkv_delta_backward_workspace_bytes(B, T, H, H, N))
    if need == 0:
        assert H == 2 and op == "forward"
        return
    buf, ptr, header = workspace(need)
    before = header.clone()
    z = [torch.zeros(B, T, H * N, dtype=dtype, device="cuda") for _ in range(7)]
    f = [torch.zeros(B, T, H, device="cuda") for _ in range(4)]
    for _ in range(2):
        if op == "forward":
            rc = L.wkv_delta_forward(B, T, H, H, N, code, *ptrs(*f[:2], *z[:3], None, z[3], None), ptr, need, None)
        else:
            rc = L.wkv_delta_backward(B, T, H, H, N, code, *ptrs(*f[:2], *z[:3], None, z[3], None, *z[4:], *f[2:], None), ptr, need, None)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(header, before)


@pytest.mark.parametrize("C,G", [(192, 3), (1200, 1)])     # groups in registers, and too large for them
def test_group_norm(C, G):
    rows, L = 500, wkv.lib()
    need = L.wkv_group_norm_backward_workspace_bytes(rows, C, G, wkv.WKV_F32)
    buf, ptr, header = workspace(need)
    before = header.clone()
    x, dy, dx = (torch.randn(rows, C, device="cuda") for _ in range(3))
    wt, b, dwt, db = (torch.ones(C, device="cuda") for _ in range(4))
    rc = L.wkv_group_norm_backward(rows, C, G, wkv.WKV_F32, 1, 1e-5, *ptrs(x, wt, b, None, dy, dx, dwt, db, None), ptr, need, None)
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(header, before)

"""The reverse mode's segments of bfloat16 heads of 64 (tcgen05.mma): decays,
resets, many segments, shared key heads, and next to the other operator that
allocates tensor memory.  Tolerances are test_delta_gpu's: outputs in bfloat16
half a step (2^-8), float32 accuracy (2e-5 of the largest) for the rest."""
import numpy as np
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv
from test_delta_gpu import BF16, DEV, NAMES, backward, case, close, f64, ref_bwd

pytestmark = pytest.mark.gpu


def check(d, H):
    ref = ref_bwd(d, H)
    # dw is a difference of sums of r . dr and dv . v: its errors are theirs
    share = d["v"].shape[2] // d["r"].shape[2]
    rd = np.abs((f64(d["r"]) * ref[0]).reshape(*d["r"].shape[:2], -1, 64).sum(-1)).max() * share
    vd = np.abs((f64(d["v"]) * ref[2]).reshape(*d["v"].shape[:2], -1, 64).sum(-1)).max()
    for name, g, r in zip(NAMES, backward(d, H), ref):
        close(g, r, name, scale=max(rd, vd, np.abs(r).max()) if name == "dw" else None)


@pytest.mark.parametrize("w", [0.0, 1e-6, 0.1, 3.5, 30.0, 200.0, float("inf")])
def test_decays(w):
    d = case(1, 140, 1, 2, 64, BF16, w=w)
    check(d, 2)
    if w >= 200:
        assert torch.count_nonzero(backward(d, 2)[3]) == 0


@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (2, 63, 1, 1), (1, 64, 2, 2), (3, 129, 1, 3), (2, 191, 3, 6), (1, 1000, 2, 2), (5, 66, 7, 7)])
def test_lengths_and_shared_keys(B, T, Hk, H):
    check(case(B, T, Hk, H, 64, BF16), H)


def test_resets():
    d = case(2, 200, 2, 4, 64, BF16)
    d["w"][:, 37] = float("inf")
    d["w"][0, 64] = float("inf")
    d["w"][1, 127, 2] = float("inf")
    d["w"][1, 128] = float("inf")
    check(d, 4)


def test_what_a_sequence_has_does_not_reach_others():
    """NaN in one sequence stays there."""
    d = case(3, 150, 2, 2, 64, BF16)
    want = backward(d, 2)
    d["v"][1, 100] = float("nan")
    for a, b in zip(want, backward(d, 2)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_beside_the_other_user_of_tensor_memory():
    """The matrix-state forward and the reverse mode on two streams at once."""
    d = case(4, 1500, 16, 16, 64, BF16)
    g = torch.Generator(device=DEV).manual_seed(1)
    B, T, C, H = 8, 1024, 2048, 32
    r, k, v = (torch.randn((B, T, C), generator=g, device=DEV).to(BF16) for _ in range(3))
    w, u = torch.rand(C, generator=g, device=DEV), torch.randn(C, generator=g, device=DEV)
    want, (y0, s0) = backward(d, 16), wkv.wkv5_forward(w, u, r, k, v, H)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            got = [backward(d, 16) for _ in range(2)]
        with torch.cuda.stream(streams[1]):
            y, s = wkv.wkv5_forward(w, u, r, k, v, H)
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(s, s0)
        assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))

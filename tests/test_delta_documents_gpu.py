"""Decay rates' gradients of documents packed into one sequence: what follows a
reset (w = inf) is no part of the gradients before it, and its rounding must not
reach them either.  Tolerance: test_delta_gpu's 2e-5, of each document's own scale."""
import pytest
import torch

from test_delta_gpu import BF16, F32, NAMES, backward, case, close, f64, ref_bwd

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("N,dtype", [(32, BF16), (64, BF16), (128, BF16), (64, F32), (128, F32)])


@KINDS
@pytest.mark.parametrize("T,at", [(64, 30), (64, 1), (200, 63), (200, 64), (200, 65), (200, 190)])
def test_a_document_without_gradient(T, at, N, dtype):
    """Nothing comes from outputs with dy = 0: every gradient before the border is 0."""
    d = case(2, T, 1, 2, N, dtype)
    d["w"][:, at] = float("inf")
    d["dy"][:, :at] = 0
    got = dict(zip(NAMES, backward(d, 2)))
    for name in ("dr", "dk", "dv", "dw", "dbeta"):
        assert torch.count_nonzero(got[name][:, :at]) == 0, name
    assert torch.count_nonzero(got["dstate_in"]) == 0


@KINDS
@pytest.mark.parametrize("at", [(30,), (20, 21, 50), (64, 100), (5, 70, 71)])
def test_documents_of_their_own_size(at, N, dtype):
    """Gradients of 2^20 in every other document leave the others' as they are by themselves."""
    H, T = 2, 140
    d = case(1, T, 1, H, N, dtype, state=False)
    d["w"][:, list(at)] = float("inf")
    borders = [0, *at, T]
    for i in range(len(at) + 1):
        if i % 2:
            d["dy"][:, borders[i]:borders[i + 1]] *= 2.0 ** 20
    got = backward(d, H, ds=False)
    for t0, t1 in zip(borders, borders[1:]):
        part = {n: x[:, t0:t1].contiguous() if x is not None and n not in ("state_in", "ds") else x for n, x in d.items()}
        ref = ref_bwd(part, H, ds=False)
        # dw is a difference of sums of r . dr and dv . v: its errors are theirs
        size = max(abs(f64(part["r"]) * ref[0]).sum(-1).max(), abs(f64(part["v"]) * ref[2]).sum(-1).max(), abs(ref[3]).max())
        close(got[3][:, t0:t1], ref[3], "dw", scale=size)

"""The gated delta rule over thousands of tokens, with states that hardly fade,
against the fp64 oracle.

Tolerance: a token rounds its sums at about (N / 8 + 8) 2^-24 = 1.4e-6 for N = 128
(test_delta_gpu).  With no decay an error lasts until the keys have erased it: a token
takes beta (2 - beta) = 3/4 of the square along one of N directions, so amplitudes
last about 2 N / 0.75 = 340 tokens, and errors of either sign add up to
1.4e-6 sqrt(340) = 2.6e-5.  The bound is 4e-5 of the largest magnitude; a bfloat16
output adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from test_delta_gpu import BF16, F32, NAMES, backward, case, f64, forward, ref_bwd, ref_fwd

pytestmark = pytest.mark.gpu


def close(got, ref, name, scale=None):
    g = f64(got)
    scale = np.abs(ref).max() if scale is None else scale
    err = np.abs(g - ref)
    assert np.all(err <= 4e-5 * scale + (2.0 ** -8 * np.abs(ref) if got.dtype == BF16 else 0)), f"{name}: {np.max(err) / scale:.3e}"


@pytest.mark.parametrize("w", [0.0, 1e-6, None])
@pytest.mark.parametrize("N,dtype", [(32, BF16), (64, BF16), (128, BF16), (64, F32), (128, F32)])
def test_long(N, dtype, w):
    T, Hk, H = 2100, 1, 2
    d = case(1, T, Hk, H, N, dtype, w=w)
    for name, g, r in zip(("y", "state"), forward(d, H), ref_fwd(d, H)):
        close(g, r, name)
    ref = ref_bwd(d, H)
    # dw is a difference of sums of r . dr and dv . v: its errors are theirs
    terms = np.abs((f64(d["r"]) * ref[0]).sum(-1)).max() * H + np.abs((f64(d["v"]) * ref[2]).reshape(1, T, H, N).sum(-1)).max()
    for name, g, r in zip(NAMES, backward(d, H), ref):
        close(g, r, name, max(terms, np.abs(r).max()) if name == "dw" else None)

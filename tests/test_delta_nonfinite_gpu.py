"""Values that are not finite (NaN, infinities): what they reach is what the
definition, token by token, lets them reach.  Outputs that the oracle has finite
keep test_delta_gpu's tolerances, all others are not finite either."""
import warnings

import numpy as np
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv
from test_delta_gpu import BF16, F32, NAMES, backward, case, f64, forward, ref_bwd, ref_fwd

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("N,dtype", [(32, BF16), (64, BF16), (128, BF16), (32, F32), (64, F32), (128, F32)])
NAN, INF = float("nan"), float("inf")


def same(got, ref, name, scale=None):
    g = f64(got)
    ok = np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), ok), f"{name}: finite at {np.argwhere(np.isfinite(g) != ok)[:4].tolist()} on one side only"
    if ok.any():
        scale = max(np.abs(ref[ok]).max(), 1e-30) if scale is None else scale
        tol = 2e-5 * scale + (2.0 ** -8 * np.abs(ref[ok]) if got.dtype == BF16 else 0)
        err = np.abs(g[ok] - ref[ok])
        assert np.all(err <= tol), f"{name}: {np.max(err / scale):.3e}"


def check(d, H, terms):
    """terms: the largest sum of r . dr and dv . v of the call without the value, which dw's errors are of."""
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        fwd, bwd = ref_fwd(d, H), ref_bwd(d, H)
    for name, g, r in zip(("y", "state"), forward(d, H), fwd):
        same(g, r, name)
    for name, g, r in zip(NAMES, backward(d, H), bwd):
        same(g, r, name, terms if name == "dw" else None)


def whole(B, T, Hk, H, N, dtype):
    d = case(B, T, Hk, H, N, dtype)
    ref = ref_bwd(d, H)
    share = H // Hk
    rd = np.abs((f64(d["r"]) * ref[0]).reshape(B, T, Hk, N).sum(-1)).max() * share
    vd = np.abs((f64(d["v"]) * ref[2]).reshape(B, T, H, N).sum(-1)).max()
    return d, max(rd, vd, np.abs(ref[3]).max())


@KINDS
@pytest.mark.parametrize("at", [12, 70, 139])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("k", -INF), ("r", NAN), ("r", INF), ("dy", NAN),
                                        ("dy", INF), ("w", NAN), ("beta", NAN)])
def test_one_value(name, value, at, N, dtype):
    d, terms = whole(2, 140, 1, 2, N, dtype)
    d[name][1, at, 1 if name in ("w", "beta") else 17] = value
    check(d, 2, terms)


@KINDS
@pytest.mark.parametrize("name", ["state_in", "ds"])
def test_one_value_of_a_state(name, N, dtype):
    d, terms = whole(2, 140, 2, 2, N, dtype)
    d[name][0, 1, 3, 21] = NAN
    check(d, 2, terms)


@KINDS
@pytest.mark.parametrize("a,b", [(("v", 20), ("dy", 90)), (("v", 40), ("dy", 20)), (("v", 50), ("k", 9)), (("k", 30), ("dy", 18)),
                                 (("r", 11), ("v", 25)), (("v", 63), ("dy", 64)), (("v", 64), ("dy", 63))])
def test_two_values(a, b, N, dtype):
    """What the first leaves of the tokens on its side and the second of those on its own."""
    d, terms = whole(1, 100, 1, 1, N, dtype)
    for name, at in (a, b):
        d[name][0, at, 5] = NAN
    check(d, 1, terms)


@KINDS
def test_a_document_before_the_border(N, dtype):
    """A NaN behind a reset does not reach y of the document ahead of it."""
    d, terms = whole(1, 140, 1, 2, N, dtype)
    d["w"][:, 40] = INF
    d["v"][:, 45] = NAN
    y, s = forward(d, 2)
    ref = ref_fwd(d, 2)
    same(y, ref[0], "y")
    assert torch.isfinite(y[:, :45]).all() and not torch.isfinite(y[:, 45:]).any()
    for name, g, r in zip(NAMES, backward(d, 2), ref_bwd(d, 2)):
        same(g, r, name, terms if name == "dw" else None)


@pytest.mark.parametrize("N,dtype", [(64, BF16), (64, F32)])
def test_a_state_that_overflows(N, dtype):
    """Finite inputs of a recurrence that grows past float32: tokens before that stay."""
    d = case(1, 60, 1, 1, N, dtype, state=False)
    d["w"][:] = 0
    d["k"][:] = 0
    d["k"][..., 0] = 2.0       # beta k.k = 8: S grows by -7 a token, past 2^128 at about the 46th
    d["beta"][:] = 2.0
    y, _ = forward(d, 1)
    ref = ref_fwd(d, 1)[0][:, :44]      # 4 |v| 7^43 is 10^37
    assert torch.isfinite(y[:, :44]).all() and not torch.isfinite(y[:, 50:]).any()
    # S = y / r by tokens; each of 44 tokens rounds about four times at the largest S so far: 44 * 4 * 2^-24 = 1.1e-5
    r0 = np.abs(f64(d["r"])[:, :44, :1])
    scale = r0 * np.maximum.accumulate(np.abs(ref) / r0, axis=1)
    assert np.all(np.abs(f64(y)[:, :44] - ref) <= 2e-5 * scale + (2.0 ** -8 * np.abs(ref) if dtype == BF16 else 0))


@pytest.mark.parametrize("B,T,Hk,H,N,dtype", [(3, 700, 50, 100, 64, BF16), (5, 600, 20, 20, 128, BF16), (3, 600, 60, 60, 32, F32)])
@pytest.mark.parametrize("name,at", [("v", 300), ("k", 520), ("dy", 300), ("state_in", 0), ("ds", 0)])
def test_walks_in_parts(name, at, B, T, Hk, H, N, dtype):
    """More walks than the GPU holds: the one with the value is as in a call of its
    own, where it is walked whole, and all others keep their bits."""
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k = n(B, T, Hk, N)
    d = {"w": torch.exp(n(B, T, H) - 2), "beta": torch.sigmoid(n(B, T, H)), "r": (n(B, T, Hk * N) * N ** -0.5).to(dtype),
         "k": (k / k.norm(dim=-1, keepdim=True)).flatten(2).to(dtype), "v": n(B, T, H * N).to(dtype), "state_in": 0.3 * n(B, H, N, N),
         "dy": n(B, T, H * N).to(dtype), "ds": 0.3 * n(B, H, N, N)}
    clean = [*forward(d, H), *backward(d, H)]
    b, hk, share = B - 2, Hk - 3, H // Hk
    h = hk * share
    if name in ("state_in", "ds"):
        d[name][b, h, 4, 9] = NAN
    else:
        d[name][b, at, (h if name in ("v", "dy") else hk) * N + 9] = NAN
    got = [*forward(d, H), *backward(d, H)]
    heads = lambda x, m: x.unflatten(-1, (m, -1)) if x.dim() == 3 else x.transpose(1, 2)  # noqa: E731
    sizes = (H, H, Hk, Hk, H, H, H, H)
    # the heads of that key head by themselves
    pick = lambda x, m: x[b:b + 1].unflatten(-1, (m, -1))[..., m // Hk * hk:m // Hk * (hk + 1), :].flatten(2).contiguous()  # noqa: E731
    one = {x: pick(d[x], Hk if x in ("r", "k") else H) for x in ("w", "beta", "r", "k", "v", "dy")}
    one.update({x: d[x][b:b + 1, h:h + share].contiguous() for x in ("state_in", "ds")})
    alone = [*forward(one, share), *backward(one, share)]
    assert any(not torch.isfinite(x).all() for x in alone)
    for i, (x, y, z, m) in enumerate(zip(got, clean, alone, sizes)):
        if x.dim() == 4:      # states
            x, y, z = x.clone(), y.clone(), z[0]
            mine, x[b, h:h + share], y[b, h:h + share] = x[b, h:h + share].clone(), 0, 0
        else:
            per = m // Hk
            x, y = x.unflatten(-1, (m, -1)).clone(), y.unflatten(-1, (m, -1)).clone()
            mine = x[b, :, per * hk:per * (hk + 1)].flatten(1).clone()
            x[b, :, per * hk:per * (hk + 1)], y[b, :, per * hk:per * (hk + 1)] = 0, 0
            z = z[0]
        assert torch.equal(x, y), f"another head of output {i}"
        ok = torch.isfinite(z)
        assert torch.equal(torch.isfinite(mine), ok), f"output {i}"
        if ok.any():
            scale = z[ok].abs().max().double()
            err = (mine[ok].double() - z[ok].double()).abs()
            # both within 2e-5 of the largest (dw: of the sums it comes from, up to ten times as large), rounded once each
            assert (err <= (4e-4 if i == 5 else 4e-5) * scale + (2 * 2.0 ** -8 * z[ok].double().abs() if z.dtype == BF16 else 0)).all(), f"output {i}"

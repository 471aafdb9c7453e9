"""The group norm with an activation against the fp64 oracle.

Tolerance of the float32 arithmetic: 2e-5 of the largest magnitude of the
tensor (mean and variance round sums over a group; the exponential and the
reciprocal of the sigmoid are within 2^-22 plus |x| 2^-24 of the argument), a
bfloat16 output adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv
from oracle import delta as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, ref, name=""):
    g = f64(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g)), name
    scale = max(np.abs(ref).max(), 1e-30)
    err = np.abs(g - ref)
    assert np.all(err <= 2e-5 * scale + (2.0 ** -8 * np.abs(ref) if got.dtype == BF16 else 0)), \
        f"{name}: {np.max(err) / scale:.3e}"


def case(lead, C, dtype, affine=True, gate=True, seed=0):
    g = torch.Generator().manual_seed(seed + C)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"x": (2 * n(*lead, C) + 0.5).to(dtype), "weight": 1 + 0.3 * n(C) if affine else None,
         "bias": 0.3 * n(C) if affine else None, "gate": n(*lead, C).to(dtype) if gate else None,
         "dy": n(*lead, C).to(dtype)}
    return {k: None if x is None else x.to(DEV) for k, x in d.items()}


def check(d, G, act, eps=1e-5, **kw):
    a = (d["x"], G, d["weight"], d["bias"], d["gate"])
    r = (f64(d["x"]), G, f64(d["weight"]), f64(d["bias"]), f64(d["gate"]))
    y = wkv.wkv_group_norm(*a, act=act, eps=eps, **kw)
    close(y, D.group_norm(*r, act=act, eps=eps), "y")
    got = wkv.wkv_group_norm_backward(*a, dy=d["dy"], act=act, eps=eps, **kw)
    ref = D.group_norm_backward(*r, dy=f64(d["dy"]), act=act, eps=eps)
    given = (True, d["weight"] is not None, d["bias"] is not None, d["gate"] is not None)
    for name, g, x, want in zip(("dx", "dweight", "dbias", "dgate"), got, ref, given):
        if want:
            close(g, x, name)
        else:
            assert g is None
    return (y, *(g for g in got if g is not None))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G,size", [(1, 8), (3, 10), (2, 17), (32, 64), (5, 96), (3, 100), (1, 129), (2, 128), (4, 256),
                                    (1, 512), (2, 250), (3, 257), (1, 520), (1, 2048), (2, 1001), (7, 4), (65, 12)])
def test_group_sizes(G, size, dtype):
    check(case((2, 5), G * size, dtype), G, "silu")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_activations(act, gate, affine, dtype):
    check(case((3, 7), 192, dtype, affine, gate), 3, act)
    check(case((2,), 1200, dtype, affine, gate), 2, act)     # groups too large for registers


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 1000, 5000])
def test_rows(rows):
    check(case((rows,), 128, BF16), 2, "silu")
    check(case((rows,), 70, F32), 2, "none")


def test_many_rows_of_large_groups():
    check(case((300,), 1100, F32), 1, "silu")


def test_one_dimension_and_no_rows():
    check(case((), 64, F32), 1, "silu")
    d = case((0, 3), 64, F32)
    assert wkv.wkv_group_norm(d["x"], 2, d["weight"]).shape == (0, 3, 64)
    g = wkv.wkv_group_norm_backward(d["x"], 2, d["weight"], d["bias"], dy=d["dy"])
    assert torch.count_nonzero(g[1]) == 0 and torch.count_nonzero(g[2]) == 0


def test_groups_of_one_and_constant_groups():
    """Nothing is left of a group without variance: y is the bias."""
    d = case((4,), 8, F32, gate=False)
    assert torch.equal(wkv.wkv_group_norm(d["x"], 8, d["weight"], d["bias"]), d["bias"].expand(4, 8))
    x = torch.full((4, 128), 3.0, device=DEV)
    b = torch.randn(128, device=DEV)
    assert torch.equal(wkv.wkv_group_norm(x, 2, None, b), b.expand(4, 128))


def test_extreme_values():
    """Offsets far above the spread, and gates whose sigmoid is 0 or 1."""
    d = case((6,), 128, F32)
    d["x"] = d["x"] + 1000     # float32 holds the differences to 2^-14: the statistics are two passes
    d["gate"][0, :4] = torch.tensor([100.0, -100.0, 1e30, -1e30], device=DEV)
    y = wkv.wkv_group_norm(d["x"], 2, d["weight"], d["bias"], d["gate"], act="sigmoid")
    # the mean's own rounding, 1000 x 2^-24 over a spread of 2
    ref = D.group_norm(f64(d["x"]), 2, f64(d["weight"]), f64(d["bias"]), f64(d["gate"]), "sigmoid")
    assert np.max(np.abs(f64(y) - ref)) < 1000 * 2.0 ** -22 * np.abs(ref).max()
    d = case((3,), 64, BF16)
    d["x"] *= 1e18             # squares reach 1e37, inside float32
    close(wkv.wkv_group_norm(d["x"], 1), D.group_norm(f64(d["x"]), 1), "large")


@pytest.mark.parametrize("C,G,dtype", [(128, 2, BF16), (96, 2, F32), (1200, 1, BF16)])
def test_unaligned(C, G, dtype):
    d = case((3, 5), C, dtype)

    def odd(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    check({k: odd(x) for k, x in d.items()}, G, "silu")
    # an output alone off its alignment
    y = odd(torch.empty_like(d["x"]))
    wkv.wkv_group_norm(d["x"], G, d["weight"], d["bias"], d["gate"], act="silu", y=y)
    close(y, D.group_norm(f64(d["x"]), G, f64(d["weight"]), f64(d["bias"]), f64(d["gate"]), "silu"))


def test_same_bits_on_streams_and_in_graphs():
    d = case((700,), 256, BF16)
    want = check(d, 4, "silu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = check(d, 4, "silu", stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    run = lambda: (wkv.wkv_group_norm(d["x"], 4, d["weight"], d["bias"], d["gate"], act="silu"),  # noqa: E731
                   *wkv.wkv_group_norm_backward(d["x"], 4, d["weight"], d["bias"], d["gate"], dy=d["dy"], act="silu"))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_offsets_beyond_32_bits():
    """The last row of a call of over 2^31 values equals a call of its own."""
    rows, C = (1 << 20) + 3, 2048
    x = torch.randn((rows, C), device=DEV, dtype=BF16)
    y = wkv.wkv_group_norm(x, 32, act="silu")
    assert torch.equal(y[-2:], wkv.wkv_group_norm(x[-2:], 32, act="silu"))
    dx = wkv.wkv_group_norm_backward(x, 32, dy=y, act="silu")[0]
    assert torch.equal(dx[-2:], wkv.wkv_group_norm_backward(x[-2:], 32, dy=y[-2:], act="silu")[0])

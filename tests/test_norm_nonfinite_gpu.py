"""The group norm with values that are not finite: what the definition keeps
finite stays, at test_group_norm_gpu's tolerances, and nothing else is finite."""
import warnings

import numpy as np
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv
from oracle import delta as D
from test_group_norm_gpu import BF16, F32, case, f64

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def same(got, ref, name):
    g, ok = f64(got), np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), ok), name
    scale = np.abs(ref[ok]).max()
    assert np.all(np.abs(g[ok] - ref[ok]) <= 2e-5 * scale + (2.0 ** -8 * np.abs(ref[ok]) if got.dtype == BF16 else 0)), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C,G", [(192, 3), (65 * 3, 3), (1200, 2)])      # whole vectors, single values, groups too large for registers
@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("name,value", [("x", NAN), ("x", INF), ("gate", NAN), ("gate", INF), ("gate", -INF), ("dy", NAN), ("dy", -INF)])
def test_one_value(name, value, act, C, G, dtype):
    d = case((4, 30), C, dtype)
    d[name][2, 7, C // G + 1] = value
    a = (d["x"], G, d["weight"], d["bias"], d["gate"])
    r = [x if x is G else f64(x) for x in a]
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        y, grads = D.group_norm(*r, act=act), D.group_norm_backward(*r, dy=f64(d["dy"]), act=act)
    same(wkv.wkv_group_norm(*a, act=act), y, "y")
    for n, g, x in zip(("dx", "dweight", "dbias", "dgate"), wkv.wkv_group_norm_backward(*a, dy=d["dy"], act=act), grads):
        same(g, x, n)

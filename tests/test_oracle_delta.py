"""The fp64 oracle of the gated delta rule and of the group norm: values
worked by hand, limits, and gradients against central differences."""
import numpy as np
import pytest

from oracle import delta as D


def case(B, T, Hk, H, N, seed, state=True):
    g = np.random.default_rng(seed)
    k = g.normal(size=(B, T, Hk, N))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return {"w": np.exp(g.uniform(-3, 0.5, (B, T, H))), "beta": g.uniform(0, 1, (B, T, H)),
            "r": g.normal(size=(B, T, Hk * N)), "k": k.reshape(B, T, Hk * N), "v": g.normal(size=(B, T, H * N)),
            "state_in": g.normal(size=(B, H, N, N)) if state else None}


def test_hand_worked():
    # one head of one channel: S = a S + k b (v - a S k), y = S r
    w = np.log(np.array([2.0, 4.0])).reshape(1, 2, 1)            # a = 1/2, 1/4
    beta = np.array([0.5, 1.0]).reshape(1, 2, 1)
    k, r, v = (np.array(x).reshape(1, 2, 1) for x in ([2.0, 1.0], [3.0, 5.0], [4.0, 7.0]))
    y, S = D.delta_forward(w, beta, r, k, v, 1, np.full((1, 1, 1, 1), 8.0))
    # aS = 4, e = 4 - 8 = -4, S = 4 + 2 (0.5)(-4) = 0, y = 0; then aS = 0, e = 7, S = 7, y = 35
    assert np.allclose(y.ravel(), [0, 35], atol=1e-14) and np.allclose(S.ravel(), [7], atol=1e-14)


def test_unit_beta_stores_the_value_and_orthogonal_keys_keep_it():
    N = 4
    k = np.eye(N)[[0, 1]].reshape(1, 2, N)
    v = np.arange(8.0).reshape(1, 2, N)
    y, S = D.delta_forward(np.zeros((1, 2, 1)), np.ones((1, 2, 1)), k, k, v, 1)
    assert np.array_equal(y, v)
    assert np.array_equal(S[0, 0, 0], v[0, 0]) and np.array_equal(S[0, 0, 1], v[0, 1])
    # the same key again replaces what it stored
    k2, v2 = k[:, :1].repeat(2, 1), v
    _, S = D.delta_forward(np.zeros((1, 2, 1)), np.ones((1, 2, 1)), k2, k2, v2, 1)
    assert np.array_equal(S[0, 0, 0], v[0, 1])


def test_reset_and_padding():
    c = case(1, 6, 1, 2, 4, 3)
    c["w"][:, 3] = np.inf
    y, S = D.delta_forward(**{**c, "H": 2})
    tail = {n: c[n][:, 3:] for n in ("w", "beta", "r", "k", "v")}
    y2, S2 = D.delta_forward(**tail, H=2, state_in=None)
    assert np.allclose(y[:, 3:], y2) and np.allclose(S, S2)
    c["w"][:, 3], c["beta"][:, 3] = 0, 0
    _, S = D.delta_forward(**{**c, "H": 2})
    cut = {n: np.delete(c[n], 3, 1) for n in ("w", "beta", "r", "k", "v")}
    assert np.allclose(S, D.delta_forward(**cut, H=2, state_in=c["state_in"])[1])


@pytest.mark.parametrize("B,T,Hk,H,N,state", [(1, 1, 1, 1, 2, True), (2, 5, 2, 4, 3, True), (1, 4, 1, 2, 3, False)])
def test_delta_gradients_against_differences(B, T, Hk, H, N, state):
    c = case(B, T, Hk, H, N, B + T, state)
    g = np.random.default_rng(9)
    dy, ds = g.normal(size=c["v"].shape), g.normal(size=(B, H, N, N))

    def loss(d):
        y, S = D.delta_forward(d["w"], d["beta"], d["r"], d["k"], d["v"], H, d["state_in"])
        return (y * dy).sum() + (S * ds).sum()

    if c["state_in"] is None:
        c["state_in"] = np.zeros((B, H, N, N))
    grads = dict(zip(("r", "k", "v", "w", "beta", "state_in"),
                     D.delta_backward(c["w"], c["beta"], c["r"], c["k"], c["v"], H, c["state_in"], dy, ds)))
    for name, grad in grads.items():
        h = 1e-6
        for at in g.choice(grad.size, min(8, grad.size), replace=False):
            up, down = ({**c, name: c[name].copy()} for _ in range(2))
            up[name].flat[at] += h
            down[name].flat[at] -= h
            # central differences: h^2 of the third derivative and rounding / h
            assert abs((loss(up) - loss(down)) / (2 * h) - grad.flat[at]) < 1e-7 * (1 + abs(grad.flat[at])), name


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_against_differences(act, gated):
    g = np.random.default_rng(4)
    c = {"x": g.normal(size=(2, 3, 12)), "weight": g.normal(size=12), "bias": g.normal(size=12)}
    if gated:
        c["gate"] = g.normal(size=(2, 3, 12))
    dy = g.normal(size=(2, 3, 12))
    grads = D.group_norm_backward(**c, G=3, dy=dy, act=act)
    for name, grad in zip(("x", "weight", "bias", "gate"), grads):
        if grad is None:
            continue
        h = 1e-6
        for at in g.choice(grad.size, 6, replace=False):
            up, down = ({**c, name: c[name].copy()} for _ in range(2))
            up[name].flat[at] += h
            down[name].flat[at] -= h
            d = ((D.group_norm(**up, G=3, act=act) - D.group_norm(**down, G=3, act=act)) * dy).sum() / (2 * h)
            assert abs(d - grad.flat[at]) < 1e-7 * (1 + abs(grad.flat[at])), name


def test_norm_hand_worked():
    y = D.group_norm(np.array([[1.0, 3.0, 5.0, 5.0]]), 2, np.array([1.0, 2, 3, 4]), np.array([0.0, 1, 2, 3]), eps=0.0 + 1e-300)
    assert np.allclose(y, [[-1, 3, 2, 3]])

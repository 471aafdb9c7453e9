"""bfloat16 calls of the gated delta rule compute in float32 and round once.

Rows of zeros and ones make an output equal to one float32 number with all its
24 bits: a value of the state, of its gradient, or a learning rate.  Sums of
such rows are exact in float32 (products with 1, additions of 0), so a bfloat16
output has to be that number rounded once, and a float32 output the number
itself: no tolerance.  Half of the numbers lie one float32 step beside a border
between two bfloat16 ones, where an operand cut to 16 bits rounds the wrong way.
The numbers' eighth bit is 0, so that their leading bfloat16 piece is of their own
exponent: tensor cores cut a sum off below 24 bits of its largest term."""
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
B, H = 4, 3
SIZES = pytest.mark.parametrize("N,dtype", [(32, BF16), (64, BF16), (128, BF16), (64, F32), (128, F32)])


def numbers(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(shape, generator=g, device=DEV).view(torch.int32) & ~0x10000).view(torch.float32)
    border = (x.view(torch.int32) & -65536) | 0x8000          # halfway between two bfloat16 numbers
    side = torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.int32) * 2 - 1
    near = (border + side).view(torch.float32)                # and one float32 step off it
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, near, x)


def zeros(T, N, dtype):
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    return {"w": z(B, T, H, t=F32), "beta": z(B, T, H, t=F32), "r": z(B, T, H, N), "k": z(B, T, H, N), "v": z(B, T, H, N)}


def flat(d):
    return [x.flatten(2) if x.dim() == 4 else x for x in d.values()]


def forward(d, state=None):
    return wkv.wkv_delta_forward(*flat(d), H, state)[0].view(d["v"].shape)


def dk_of(d, dy, state=None, ds=None):
    return wkv.wkv_delta_backward(*flat(d), H, state, dy=dy.flatten(2), dstate_out=ds)[1].view(d["k"].shape)


@SIZES
def test_a_row_of_the_state(N, dtype):
    d, S = zeros(40, N, dtype), numbers(B, H, N, N, seed=N)
    at = torch.arange(40, device=DEV) * 7 % N
    d["r"][:, torch.arange(40, device=DEV), :, at] = 1
    assert torch.equal(forward(d, S), S[:, :, at].transpose(1, 2).to(dtype))


@SIZES
def test_the_learning_rate_of_a_token_before(N, dtype):
    """Token 16 c writes beta v^T, v all ones, to channel c, which the 15 after it read."""
    n = 16
    d, b = zeros(16 * n, N, dtype), numbers(B, n, H, seed=1)
    for c in range(n):
        d["k"][:, 16 * c, :, c] = 1
        d["r"][:, 16 * c:16 * c + 16, :, c] = 1
    d["v"][:, ::16] = 1
    d["beta"][:, ::16] = b
    want = b.repeat_interleave(16, 1)[..., None].expand(B, 16 * n, H, N)
    assert torch.equal(forward(d), want.to(dtype))


@SIZES
def test_an_error_read_back(N, dtype):
    """k of two channels, one of them the state's only row: y reads the other, where the update put -S."""
    d, S = zeros(1, N, dtype), torch.zeros(B, H, N, N, device=DEV)
    S[:, :, 3] = numbers(B, H, N, seed=2)
    d["beta"][:] = 1
    d["k"][..., 3] = d["k"][..., N - 2] = 1
    d["r"][..., N - 2] = 1
    assert torch.equal(forward(d, S)[:, 0], -S[:, :, 3].to(dtype))


@SIZES
def test_gradient_of_a_key_from_the_state_gradient(N, dtype):
    """dk = D u: a column of D, and the u of a diagonal D."""
    j = N - 5
    d, D = zeros(1, N, dtype), numbers(B, H, N, N, seed=3)
    d["v"][..., j] = 1
    d["beta"][:] = 1
    assert torch.equal(dk_of(d, torch.zeros_like(d["v"]), ds=D)[:, 0], D[..., j].to(dtype))
    d["v"][:] = 1
    d["beta"][:] = b = numbers(B, 1, H, seed=4)
    eye = torch.eye(N, device=DEV).expand(B, H, N, N).contiguous()
    assert torch.equal(dk_of(d, torch.zeros_like(d["v"]), ds=eye), b[..., None].expand(B, 1, H, N).to(dtype))


@SIZES
def test_gradient_of_a_key_from_the_state(N, dtype):
    """dk = -S dv where the key reads an empty row of S: a column of S, and dv."""
    j, row = 6, N - 1
    d, S, D = zeros(1, N, dtype), numbers(B, H, N, N, seed=5), torch.zeros(B, H, N, N, device=DEV)
    S[:, :, row] = 0
    D[:, :, row, j] = 1
    d["k"][..., row] = 1
    d["beta"][:] = 1
    none = torch.zeros_like(d["v"])
    assert torch.equal(dk_of(d, none, S, D)[:, 0], (0 - S[..., j]).to(dtype))
    S[:] = 1
    S[:, :, row] = 0
    d["beta"][:] = b = numbers(B, 1, H, seed=6)
    want = -b[..., None].repeat(1, 1, 1, N)
    want[..., row] = 0
    assert torch.equal(dk_of(d, none, S, D), want.to(dtype))


@SIZES
@pytest.mark.parametrize("t,s", [(0, 1), (5, 37), (17, 63), (30, 33)])
def test_gradient_of_a_key_from_a_later_output(N, dtype, t, s):
    """dk_t = (u_t.dy_s) r_s."""
    d, b = zeros(64, N, dtype), numbers(B, H, seed=7)
    dy = torch.zeros_like(d["v"])
    d["v"][:, t, :, 9] = 1
    d["beta"][:, t] = b
    dy[:, s, :, 9] = 1
    d["r"][:, s, :, 4] = 1
    want = torch.zeros_like(d["k"])
    want[:, t, :, 4] = b.to(dtype)
    assert torch.equal(dk_of(d, dy), want)


@SIZES
@pytest.mark.parametrize("s,t", [(0, 1), (5, 37), (17, 63), (30, 33)])
def test_gradient_of_a_key_from_another_token(N, dtype, s, t):
    """dk_t = -(u_s.dv_t) k_s, the state that token s left; and for the earlier one of two keys
    D u less (dv.u) k, a half of beta."""
    d, b = zeros(64, N, dtype), numbers(B, H, seed=8)
    D = torch.zeros(B, H, N, N, device=DEV)
    none = torch.zeros_like(d["v"])
    D[:, :, 2, 9] = 1
    d["k"][:, s, :, 7], d["v"][:, s, :, 9], d["beta"][:, s] = 1, 1, b
    d["k"][:, t, :, 2], d["beta"][:, t] = 1, 1
    assert torch.equal(dk_of(d, none, ds=D)[:, t, :, 7], -b.to(dtype))
    d["k"][:, s] = 0
    d["beta"][:, t] = 0.5
    assert torch.equal(dk_of(d, none, ds=D)[:, s, :, 2], (0.5 * b).to(dtype))
    # dv of 24 bits: the state of channel 7 is 1
    d["k"][:, s, :, 7], d["beta"][:, s], d["beta"][:, t] = 1, 1, b
    assert torch.equal(dk_of(d, none, ds=D)[:, t, :, 7], -b.to(dtype))

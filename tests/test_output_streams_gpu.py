"""Outputs that a call with stream= makes: no memory that the current stream is
still at work on, and none that is given away while the current stream reads it."""
import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

pytestmark = pytest.mark.gpu
B, T, H, N = 2, 2048, 8, 64
C = H * N


def run(op, stream):
    """The largest output of the operator, `stream` passed on."""
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    kw = dict(stream=stream)
    if op == "forward":
        a = z(C), z(C), z(B, T, C), z(B, T, C), z(B, T, C)
        return lambda: wkv.wkv_forward(*a, **kw)[0]
    if op == "backward":
        a, dy = (z(C), z(C), z(B, T, C), z(B, T, C), z(B, T, C)), z(B, T, C)
        return lambda: wkv.wkv_backward(*a, dy=dy, **kw)[0]
    if op == "wkv5":
        a = z(C), z(C), z(B, T, C), z(B, T, C), z(B, T, C), H
        return lambda: wkv.wkv5_forward(*a, **kw)[0]
    if op == "token_shift":
        a = z(B, T, C), z(1, C)
        return lambda: wkv.wkv_token_shift(*a, **kw)[0]
    if op == "step":
        a = z(1, C), z(1, C), z(1, B * T, C), z(1, B * T, C), z(1, 3, B * T, C)
        return lambda: wkv.wkv_step(*a, **kw)
    if op == "norm":
        a = z(B, T, C), H
        return lambda: wkv.wkv_group_norm(*a, **kw)
    if op == "norm_backward":
        a, dy = (z(B, T, C), H), z(B, T, C)
        return lambda: wkv.wkv_group_norm_backward(*a, dy=dy, **kw)[0]
    a = z(B, T, H), z(B, T, H), z(B, T, C), z(B, T, C), z(B, T, C), H
    if op == "delta_forward":
        return lambda: wkv.wkv_delta_forward(*a, **kw)[0]
    dy = z(B, T, C)
    return lambda: wkv.wkv_delta_backward(*a, dy=dy, **kw)[0]


OPS = pytest.mark.parametrize("op", ["forward", "backward", "wkv5", "token_shift", "step", "norm", "norm_backward", "delta_forward",
                                     "delta_backward"])


def busy():
    torch.cuda._sleep(200_000_000)


@OPS
def test_memory_that_the_current_stream_is_at_work_on(op):
    s = torch.cuda.Stream()
    call = run(op, s)
    torch.cuda.synchronize()
    call()                       # workspaces
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the output's size, free for the current stream behind what it is doing
    old = [torch.empty((B, T, C), device="cuda") for _ in range(12)]
    places = {t.data_ptr() for t in old}
    busy()
    del old
    out = call()
    assert out.data_ptr() not in places
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()


@OPS
def test_memory_that_the_current_stream_reads(op):
    s = torch.cuda.Stream()
    call = run(op, s)
    torch.cuda.synchronize()
    out = call()
    place = out.data_ptr()
    torch.cuda.synchronize()
    busy()                       # the current stream still reads out
    del out
    with torch.cuda.stream(s):
        again = [torch.empty((B, T, C), device="cuda") for _ in range(12)]
    assert place not in [t.data_ptr() for t in again]
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()

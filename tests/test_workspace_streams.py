"""Whose memory a Workspace hands out: of the call's device, and for as long as
the stream of the call, whichever it is, may still use it."""
import types

import pytest
import torch

import rwkv_wkv_recurrence_02_b200 as wkv

CUDA = [torch.device("cuda", i) for i in range(2)]


@pytest.mark.parametrize("take", ["get", "scratch"])
def test_a_workspace_of_another_device_is_refused(take):
    ws = wkv.Workspace(CUDA[0])
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        getattr(ws, take)(1024, device=CUDA[1])


@pytest.mark.parametrize("take,name", [("get", "buf"), ("scratch", "plain")])
def test_a_buffer_on_another_device_is_refused(take, name):
    """A Workspace of no device of its own is of its first call's."""
    ws = wkv.Workspace()
    setattr(ws, name, types.SimpleNamespace(device=CUDA[0], numel=lambda: 1 << 20, data_ptr=lambda: 1 << 40))
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        getattr(ws, take)(1024, device=CUDA[1])
    other = "scratch" if take == "get" else "get"
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        getattr(ws, other)(1024, device=CUDA[1])


def busy(stream):
    """About a fifth of a second of work, in which the test asks the allocator for memory."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)


def blocks(nbytes):
    """Places that the current stream is given now, many more than were free."""
    return [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(40)]


@pytest.mark.gpu
@pytest.mark.parametrize("take,name", [("get", "buf"), ("scratch", "plain")])
def test_a_replaced_buffer_is_not_given_to_the_current_stream(take, name):
    size = 3 << 20
    s, ws = torch.cuda.Stream(), wkv.Workspace()
    getattr(ws, take)(size, s)
    old = getattr(ws, name).data_ptr()
    torch.cuda.synchronize()
    busy(s)
    getattr(ws, take)(4 * size, s)
    assert getattr(ws, name).data_ptr() != old
    assert old not in [t.data_ptr() for t in blocks(size + 256)]
    assert not s.query()      # the stream was at work throughout
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("take,name", [("get", "buf"), ("scratch", "plain")])
def test_a_replaced_buffer_waits_for_every_stream_that_used_it(take, name):
    """Made on the current stream, used on another, replaced on the current one."""
    size = 5 << 20
    s, ws = torch.cuda.Stream(), wkv.Workspace()
    getattr(ws, take)(size)
    old = getattr(ws, name).data_ptr()
    torch.cuda.synchronize()
    getattr(ws, take)(size, s)
    assert getattr(ws, name).data_ptr() == old
    busy(s)
    getattr(ws, take)(4 * size)
    assert old not in [t.data_ptr() for t in blocks(size + 256)]
    assert not s.query()
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_calls_on_a_stream_that_grow_a_workspace():
    """Larger and larger calls on a stream of their own, while the current stream fills memory."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    cases = []
    for T in (40, 300, 900, 2100):
        d = [torch.exp(n(2, T, 3)), torch.sigmoid(n(2, T, 3)), *(0.2 * n(2, T, 96) for _ in range(4))]
        cases.append((d, wkv.wkv_delta_backward(*d[:5], 3, dy=d[5])))
    s, ws = torch.cuda.Stream(), wkv.Workspace()
    torch.cuda.synchronize()
    got = []
    for d, _ in cases:
        got.append(wkv.wkv_delta_backward(*d[:5], 3, dy=d[5], workspace=ws, stream=s))
        for _ in range(8):
            torch.empty(ws.plain.numel(), dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for (_, want), have in zip(cases, got):
        assert all(torch.equal(a, b) for a, b in zip(want, have))

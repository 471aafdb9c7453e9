"""B200 (sm_100a) RWKV WKV operators, gated delta rule and group norm: Python
binding of libwkv.so.

The binding only marshals arguments: every step of the operator runs in the
CUDA kernels behind the C ABI declared in ``include/wkv.h``.  There is no CPU
fallback; if ``libwkv.so`` is missing the import fails with instructions.

Two layers:

* ``lib()`` returns the ctypes handle; its functions carry the C names
  (``wkv_forward``, ``wkv_step``, ``wkv_forward_workspace_bytes``, ...) and take
  plain integers / pointers.
* ``wkv_forward(...)`` and ``wkv_step(...)`` below take torch CUDA tensors,
  allocate outputs and the workspace with torch when not given, pass
  ``data_ptr()`` values and the current stream, and raise ``WkvError`` on a
  non-zero status.
"""
import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwkv.so")

WKV_F32 = 0
WKV_BF16 = 1
STATUS = {
    0: "WKV_OK", -1: "WKV_ERR_NULLPTR", -2: "WKV_ERR_SHAPE", -3: "WKV_ERR_DTYPE",
    -4: "WKV_ERR_ALIGN", -5: "WKV_ERR_ALIAS", -6: "WKV_ERR_CUDA", -7: "WKV_ERR_TIMEOUT",
    -8: "WKV_ERR_WORKSPACE", -9: "WKV_ERR_SCRATCH",
}
# the functions include/wkv.h declares
EXPORTS = ("wkv_forward", "wkv_forward_ex", "wkv_forward_workspace_bytes", "wkv_workspace_init", "wkv_workspace_status",
           "wkv_step", "wkv_forward_noalloc", "wkv_forward_noalloc_scratch_bytes", "wkv_forward_noalloc_status",
           "wkv_backward", "wkv_state", "wkv_state_combine", "wkv5_forward",
           "wkv_backward_workspace_bytes", "wkv_token_shift", "wkv_delta_forward", "wkv_delta_forward_workspace_bytes",
           "wkv_delta_step",
           "wkv_delta_backward", "wkv_delta_backward_workspace_bytes", "wkv_delta_status", "wkv_group_norm", "wkv_group_norm_backward",
           "wkv_group_norm_backward_workspace_bytes", "wkv_strerror", "wkv_last_cuda_error",
           "wkv_abi_version")

_lib = None
_lock = threading.Lock()


class WkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().wkv_strerror(status).decode()
        if status == -6:
            msg += ": " + lib().wkv_last_cuda_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")


def lib():
    """ctypes handle of libwkv.so with argument types set."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'` from the repository root "
                              "(or rwkv_wkv_recurrence_02_b200/build_ext.py)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.wkv_forward.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wkv_forward.restype = i32
        L.wkv_forward_ex.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_uint, vp]
        L.wkv_forward_ex.restype = i32
        L.wkv_forward_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.wkv_forward_workspace_bytes.restype = sz
        L.wkv_workspace_init.argtypes = [vp, sz, vp]
        L.wkv_workspace_init.restype = i32
        L.wkv_workspace_status.argtypes = [vp, vp]
        L.wkv_workspace_status.restype = i32
        L.wkv_step.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.wkv_step.restype = i32
        L.wkv_token_shift.argtypes = [i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp]
        L.wkv_token_shift.restype = i32
        L.wkv_forward_noalloc.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.wkv_forward_noalloc.restype = i32
        L.wkv_forward_noalloc_scratch_bytes.argtypes = [i64, i64, i64, i32]
        L.wkv_forward_noalloc_scratch_bytes.restype = sz
        L.wkv_state.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.wkv_state.restype = i32
        L.wkv_state_combine.argtypes = [i64, i64, i32, vp, vp, vp, vp, vp, vp]
        L.wkv_state_combine.restype = i32
        L.wkv5_forward.argtypes = [i64, i64, i64, i64, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.wkv5_forward.restype = i32
        L.wkv_forward_noalloc_status.argtypes = [vp]
        L.wkv_forward_noalloc_status.restype = i32
        L.wkv_backward.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   vp, sz, vp]
        L.wkv_backward.restype = i32
        L.wkv_backward_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.wkv_backward_workspace_bytes.restype = sz
        L.wkv_delta_forward.argtypes = [i64] * 5 + [i32] + [vp] * 9 + [sz, vp]
        L.wkv_delta_forward.restype = i32
        L.wkv_delta_forward_workspace_bytes.argtypes = [i64] * 4
        L.wkv_delta_forward_workspace_bytes.restype = sz
        L.wkv_delta_step.argtypes = [i64] * 5 + [i32] + [vp] * 8
        L.wkv_delta_step.restype = i32
        L.wkv_delta_backward.argtypes = [i64] * 5 + [i32] + [vp] * 15 + [sz, vp]
        L.wkv_delta_backward.restype = i32
        L.wkv_delta_backward_workspace_bytes.argtypes = [i64] * 5
        L.wkv_delta_backward_workspace_bytes.restype = sz
        L.wkv_delta_status.argtypes = [i32, vp]
        L.wkv_delta_status.restype = i32
        L.wkv_group_norm.argtypes = [i64] * 3 + [i32, i32, ctypes.c_float] + [vp] * 6
        L.wkv_group_norm.restype = i32
        L.wkv_group_norm_backward.argtypes = [i64] * 3 + [i32, i32, ctypes.c_float] + [vp] * 10 + [sz, vp]
        L.wkv_group_norm_backward.restype = i32
        L.wkv_group_norm_backward_workspace_bytes.argtypes = [i64] * 3 + [i32]
        L.wkv_group_norm_backward_workspace_bytes.restype = sz
        L.wkv_strerror.argtypes = [i32]
        L.wkv_strerror.restype = ctypes.c_char_p
        L.wkv_last_cuda_error.argtypes = []
        L.wkv_last_cuda_error.restype = ctypes.c_char_p
        L.wkv_abi_version.argtypes = []
        L.wkv_abi_version.restype = i32
        _lib = L
        return L


# ---------------------------------------------------------------------------
# torch front end (plumbing only)
# ---------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return WKV_F32
    if t.dtype == torch.bfloat16:
        return WKV_BF16
    raise TypeError(f"k/v/r/y must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_ptr(stream, device=None):
    """cudaStream_t of `stream`, or of the current stream of `device`."""
    torch = _torch()
    if stream is not None:
        return stream.cuda_stream
    idx = device.index if device is not None and device.index is not None else torch.cuda.current_device()
    return torch._C._cuda_getCurrentRawStream(idx)


def _check(status, where):
    if status != 0:
        raise WkvError(status, where)


def _need(t, name, shape, dtype, device):
    if t is None:
        return
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _empty(shape, dtype, dev, stream):
    """A call's output: of `stream`, which writes it, and known to be used on the
    current stream; without a stream of the call's own, an ordinary tensor."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _empty_like(t, stream):
    return _torch().empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


class Workspace:
    """Device scratch for wkv_forward's cross-block exchange, grown on demand.

    Zeroed once per allocation (wkv_workspace_init); afterwards calls reuse it
    without clearing.  Calls that share one Workspace must be ordered on the
    GPU (the default: the current stream).  The delta rule's and the group
    norm's calls have a buffer of their own in it, whose contents mean nothing
    between calls.  A call that needs more than a buffer holds replaces it: a
    CUDA graph captured with the old one has to be captured again.

    A Workspace is of one device, `device` or its first call's; calls on another
    are refused.  Its memory is of the stream of the call that made it, and a
    replaced buffer is reused only when every stream of its calls is done with it."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self.plain = None
        self._owner = {}     # the raw stream that each buffer was allocated on

    def get(self, nbytes: int, stream=None, device=None):
        if nbytes == 0:
            return None, 0
        return self._take("buf", nbytes, stream, device)

    def scratch(self, nbytes: int, stream=None, device=None):
        """The other buffer: only its header (the error word) is cleared."""
        return self._take("plain", nbytes, stream, device)

    def _take(self, name, nbytes, stream, device):
        torch = _torch()
        buf = getattr(self, name)
        if device is None and buf is not None:
            device = buf.device
        if buf is None or buf.device != device or buf.numel() - 256 < nbytes:
            buf = self._make(name, nbytes, stream, device)
        elif _stream_ptr(stream, device) != self._owner[name]:
            buf.record_stream(stream if stream is not None else torch.cuda.current_stream(device))
        return self._aligned_ptr(buf), buf.numel() - 256

    def _make(self, name, nbytes, stream, device):
        torch = _torch()
        for held in (self.device, self.buf, self.plain):
            mine = getattr(held, "device", held)
            if mine is None:
                continue
            mine = torch.device(mine)
            if mine.index is not None and device is not None and mine != device:
                raise ValueError(f"the workspace is on {mine}, the call on {device}: use one for each device")
            device = device or mine
        if device is None or device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.stream(stream):   # None: the current one
            buf = torch.empty(int(nbytes) + 256, dtype=torch.uint8, device=device)
        setattr(self, name, buf)
        self._owner[name] = _stream_ptr(stream, device)
        self._init(buf, buf.numel() - 256 if name == "buf" else 256, stream)
        return buf

    def _init(self, buf, nbytes, stream):
        _launch(buf.device, "wkv_workspace_init", lib().wkv_workspace_init, self._aligned_ptr(buf), nbytes,
                _stream_ptr(stream, buf.device))

    def _aligned_ptr(self, buf=None):
        return ((self.buf if buf is None else buf).data_ptr() + 255) & ~255

    def status(self, stream=None) -> int:
        """The error word, once `stream` (that of the calls; None: the current
        one) is done with what was queued on it."""
        for buf in (self.buf, self.plain):
            if buf is not None:
                rc = lib().wkv_workspace_status(self._aligned_ptr(buf), _stream_ptr(stream, buf.device))
                if rc != 0:
                    return rc
        return 0

    def reset(self, stream=None):
        if self.buf is not None:
            self._init(self.buf, self.buf.numel() - 256, stream)
        if self.plain is not None:
            self._init(self.plain, 256, stream)


_workspaces = {}


def default_workspace(device) -> Workspace:
    key = (device.type, device.index)
    ws = _workspaces.get(key)
    if ws is None:
        ws = _workspaces[key] = Workspace(device)
    return ws


@functools.lru_cache(maxsize=1024)
def workspace_bytes(B: int, T: int, C: int, dtype_code: int) -> int:
    return int(lib().wkv_forward_workspace_bytes(B, T, C, dtype_code))


WKV_FLAG_INPUTS_READY = 1
WKV_FLAG_CHAIN_BEGIN = 2
WKV_FLAG_CHAIN_NEXT = 4


def wkv_forward(w, u, k, v, r=None, state_in=None, *, y=None, state_out=None, want_state=True,
                workspace: Workspace = None, use_workspace=True, inputs_ready=False, chain=None, stream=None):
    """Parallel mode over one chunk.  k, v, r: (B, T, C) CUDA tensors (float32
    or bfloat16); w, u: (C,) float32; state_in: (3, B, C) float32 or None.
    Returns (y, state_out) (state_out None if want_state is False and none
    was given).  state_out may be state_in for an in-place update.
    use_workspace=False passes no workspace (the scratch-free schedules).
    inputs_ready=True passes WKV_FLAG_INPUTS_READY: k, v, r, w, u are not
    written by work still running on the stream (see include/wkv.h).
    chain="begin" / "next" passes WKV_FLAG_CHAIN_BEGIN / WKV_FLAG_CHAIN_NEXT
    (a chain of chunk calls carrying one state through the workspace; see
    include/wkv.h): the first call of a chain passes "begin", every later
    one "next" with the previous call's state_out as its state_in."""
    torch = _torch()
    if k.dim() != 3:
        raise ValueError("k must be (B, T, C)")
    B, T, C = k.shape
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("wkv_forward runs on CUDA tensors only")
    code = _dtype_code(k)
    _need(v, "v", (B, T, C), k.dtype, dev)
    _need(r, "r", (B, T, C), k.dtype, dev)
    _need(w, "w", (C,), torch.float32, dev)
    _need(u, "u", (C,), torch.float32, dev)
    _need(k, "k", (B, T, C), k.dtype, dev)
    _need(state_in, "state_in", (3, B, C), torch.float32, dev)
    if y is None:
        y = _empty((B, T, C), k.dtype, dev, stream)
    _need(y, "y", (B, T, C), k.dtype, dev)
    if state_out is None and want_state:
        state_out = _empty((3, B, C), torch.float32, dev, stream)
    _need(state_out, "state_out", (3, B, C), torch.float32, dev)
    sp = _stream_ptr(stream, dev)
    if use_workspace:
        ws = workspace if workspace is not None else default_workspace(dev)
        need = workspace_bytes(B, T, C, code)
        if chain is not None:
            need = max(need, 256 + 16 * B * C)   # the chain's words follow the header
        ws_ptr, ws_bytes = ws.get(need, stream, dev)
    else:
        ws_ptr, ws_bytes = None, 0
    flags = WKV_FLAG_INPUTS_READY if inputs_ready else 0
    if chain is not None:
        if chain not in ("begin", "next"):
            raise ValueError("chain must be None, 'begin' or 'next'")
        flags |= WKV_FLAG_CHAIN_BEGIN if chain == "begin" else WKV_FLAG_CHAIN_NEXT
    if flags:
        _check(lib().wkv_forward_ex(B, T, C, code, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(state_in),
                                    _ptr(y), _ptr(state_out), ws_ptr, ws_bytes, flags, sp),
               "wkv_forward_ex")
    else:
        _check(lib().wkv_forward(B, T, C, code, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(state_in),
                                 _ptr(y), _ptr(state_out), ws_ptr, ws_bytes, sp), "wkv_forward")
    return y, state_out


def wkv_forward_noalloc(w, u, k, v, r=None, state_in=None, *, y, state_out=None, stream=None):
    """wkv_forward without a workspace, for callers that cannot allocate device
    memory: the scratch comes from a fixed array inside the library.  The
    caller supplies every output buffer (y, and state_out if wanted); this
    function allocates nothing.  Raises WkvError(WKV_ERR_SCRATCH) for problems
    larger than the built-in scratch.  Calls must be ordered on the GPU."""
    torch = _torch()
    B, T, C = k.shape
    dev = k.device
    code = _dtype_code(k)
    for t, name in ((v, "v"), (r, "r"), (y, "y")):
        _need(t, name, (B, T, C), k.dtype, dev)
    _need(w, "w", (C,), torch.float32, dev)
    _need(u, "u", (C,), torch.float32, dev)
    _need(state_in, "state_in", (3, B, C), torch.float32, dev)
    _need(state_out, "state_out", (3, B, C), torch.float32, dev)
    _check(lib().wkv_forward_noalloc(B, T, C, code, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(state_in),
                                     _ptr(y), _ptr(state_out), _stream_ptr(stream, dev)), "wkv_forward_noalloc")
    return y, state_out


def wkv_state(w, k, v, state_in=None, *, state_out=None, workspace: Workspace = None, use_workspace=True,
              stream=None):
    """State after the chunk k, v (B, T, C) entered from state_in (None: the
    empty state), without outputs; from the empty state it is the chunk's
    summary.  Returns state_out (3, B, C) float32 (may be state_in)."""
    torch = _torch()
    if k.dim() != 3:
        raise ValueError("k must be (B, T, C)")
    B, T, C = k.shape
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("wkv_state runs on CUDA tensors only")
    code = _dtype_code(k)
    _need(v, "v", (B, T, C), k.dtype, dev)
    _need(w, "w", (C,), torch.float32, dev)
    _need(k, "k", (B, T, C), k.dtype, dev)
    _need(state_in, "state_in", (3, B, C), torch.float32, dev)
    if state_out is None:
        state_out = _empty((3, B, C), torch.float32, dev, stream)
    _need(state_out, "state_out", (3, B, C), torch.float32, dev)
    sp = _stream_ptr(stream, dev)
    if use_workspace:
        ws = workspace if workspace is not None else default_workspace(dev)
        ws_ptr, ws_bytes = ws.get(workspace_bytes(B, T, C, code), stream, dev)
    else:
        ws_ptr, ws_bytes = None, 0
    _check(lib().wkv_state(B, T, C, code, _ptr(w), _ptr(k), _ptr(v), _ptr(state_in), _ptr(state_out), ws_ptr,
                           ws_bytes, sp), "wkv_state")
    return state_out


def wkv_state_combine(w, lens, states, state_in=None, *, state_out=None, stream=None):
    """Fold the summaries states (n, 3, B, C) of n consecutive chunks of
    lens[j] tokens into the state entering from state_in (None: empty).
    Returns state_out (3, B, C)."""
    torch = _torch()
    n = len(lens)
    if states.dim() != 4 or states.shape[0] < n or states.shape[1] != 3:
        raise ValueError("states must be (n, 3, B, C)")
    _, _, B, C = states.shape
    dev = states.device
    if dev.type != "cuda":
        raise ValueError("wkv_state_combine runs on CUDA tensors only")
    _need(states, "states", tuple(states.shape), torch.float32, dev)
    _need(w, "w", (C,), torch.float32, dev)
    _need(state_in, "state_in", (3, B, C), torch.float32, dev)
    if state_out is None:
        state_out = _empty((3, B, C), torch.float32, dev, stream)
    _need(state_out, "state_out", (3, B, C), torch.float32, dev)
    arr = (ctypes.c_int64 * max(1, n))(*[int(x) for x in lens])
    _check(lib().wkv_state_combine(B, C, n, _ptr(w), arr, _ptr(states), _ptr(state_in), _ptr(state_out),
                                   _stream_ptr(stream, dev)), "wkv_state_combine")
    return state_out


def wkv5_forward(w, u, r, k, v, H, state_in=None, *, y=None, state_out=None, want_state=True, stream=None):
    """Multi-head matrix-state WKV (v5 / v6).  r, k, v: (B, T, C) float32 or
    bfloat16 CUDA tensors, C = H * N with N in {32, 64}; w: (C,) decay rates
    (v5) or (B, T, C) float32 per token (v6); u: (C,) float32; state_in:
    (B, H, N, N) float32 or None (zeros).  Returns (y, state_out)."""
    torch = _torch()
    if k.dim() != 3:
        raise ValueError("k must be (B, T, C)")
    B, T, C = k.shape
    if C % H != 0:
        raise ValueError("C must be a multiple of H")
    N = C // H
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("wkv5_forward runs on CUDA tensors only")
    code = _dtype_code(k)
    for t, name in ((r, "r"), (v, "v"), (k, "k")):
        _need(t, name, (B, T, C), k.dtype, dev)
    per_token = w.dim() == 3
    _need(w, "w", (B, T, C) if per_token else (C,), torch.float32, dev)
    _need(u, "u", (C,), torch.float32, dev)
    _need(state_in, "state_in", (B, H, N, N), torch.float32, dev)
    if y is None:
        y = _empty((B, T, C), k.dtype, dev, stream)
    _need(y, "y", (B, T, C), k.dtype, dev)
    if state_out is None and want_state:
        state_out = _empty((B, H, N, N), torch.float32, dev, stream)
    _need(state_out, "state_out", (B, H, N, N), torch.float32, dev)
    _check(lib().wkv5_forward(B, T, C, H, code, _ptr(w), int(per_token), _ptr(u), _ptr(r), _ptr(k), _ptr(v),
                              _ptr(state_in), _ptr(y), _ptr(state_out), _stream_ptr(stream, dev)), "wkv5_forward")
    return y, state_out


def wkv_forward_noalloc_status(stream=None, device=None) -> int:
    """Synchronise the stream and return the error word of the library's
    built-in scratch array on the current device: 0, or WKV_ERR_TIMEOUT (-7)
    if the last wkv_forward_noalloc call that used it had a cross-block wait
    give up."""
    return int(lib().wkv_forward_noalloc_status(_stream_ptr(stream, device)))


@functools.lru_cache(maxsize=1024)
def backward_workspace_bytes(B: int, T: int, C: int, dtype_code: int) -> int:
    return int(lib().wkv_backward_workspace_bytes(B, T, C, dtype_code))


def wkv_backward(w, u, k, v, r=None, state_in=None, *, dy, dstate_out=None, dk=None, dv=None, dr=None,
                 dw=None, du=None, dstate_in=None, want_dstate_in=True, workspace: Workspace = None, stream=None):
    """Gradients of wkv_forward.  dy: (B, T, C) like k; dstate_out: (3, B, C)
    float32 dL/d(a, b) of the returned state, or None.  Returns (dk, dv, dr,
    dw, du, dstate_in); dr is None without a gate, dw and du are (C,) float32
    sums over sequences and tokens."""
    torch = _torch()
    B, T, C = k.shape
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("wkv_backward runs on CUDA tensors only")
    code = _dtype_code(k)
    for t, name in ((v, "v"), (r, "r"), (dy, "dy")):
        _need(t, name, (B, T, C), k.dtype, dev)
    _need(w, "w", (C,), torch.float32, dev)
    _need(u, "u", (C,), torch.float32, dev)
    _need(k, "k", (B, T, C), k.dtype, dev)
    _need(state_in, "state_in", (3, B, C), torch.float32, dev)
    _need(dstate_out, "dstate_out", (3, B, C), torch.float32, dev)
    if dk is None:
        dk = _empty((B, T, C), k.dtype, dev, stream)
    if dv is None:
        dv = _empty((B, T, C), k.dtype, dev, stream)
    if dr is None and r is not None:
        dr = _empty((B, T, C), k.dtype, dev, stream)
    if dw is None:
        dw = _empty((C,), torch.float32, dev, stream)
    if du is None:
        du = _empty((C,), torch.float32, dev, stream)
    if dstate_in is None and want_dstate_in:
        dstate_in = _empty((3, B, C), torch.float32, dev, stream)
    for t, name in ((dk, "dk"), (dv, "dv"), (dr, "dr")):
        _need(t, name, (B, T, C), k.dtype, dev)
    _need(dw, "dw", (C,), torch.float32, dev)
    _need(du, "du", (C,), torch.float32, dev)
    _need(dstate_in, "dstate_in", (3, B, C), torch.float32, dev)
    ws = workspace if workspace is not None else default_workspace(dev)
    sp = _stream_ptr(stream, dev)
    ws_ptr, ws_bytes = ws.get(backward_workspace_bytes(B, T, C, code), stream, dev)
    _check(lib().wkv_backward(B, T, C, code, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(state_in),
                              _ptr(dy), _ptr(dstate_out), _ptr(dk), _ptr(dv), _ptr(dr), _ptr(dw), _ptr(du),
                              _ptr(dstate_in), ws_ptr, ws_bytes, sp), "wkv_backward")
    return dk, dv, dr, dw, du, dstate_in


def wkv_token_shift(x, mu, x_prev=None, *, out=None, x_last=None, want_last=True, stream=None):
    """Token shift: x (B, T, C) float32 or bfloat16, mu (nmix, C) float32,
    x_prev (B, C) of x's dtype or None (zeros).  Returns (out, x_last) with
    out[m, b, t] = mu[m] * x[b, t] + (1 - mu[m]) * x[b, t - 1] (nmix, B, T, C)
    and x_last = x[:, T - 1] (B, C), the next call's x_prev; x_last may be
    x_prev for an in-place update."""
    torch = _torch()
    if x.dim() != 3 or mu.dim() != 2:
        raise ValueError("x must be (B, T, C) and mu (nmix, C)")
    B, T, C = x.shape
    nmix = mu.shape[0]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("wkv_token_shift runs on CUDA tensors only")
    code = _dtype_code(x)
    _need(x, "x", (B, T, C), x.dtype, dev)
    _need(mu, "mu", (nmix, C), torch.float32, dev)
    _need(x_prev, "x_prev", (B, C), x.dtype, dev)
    if out is None:
        out = _empty((nmix, B, T, C), x.dtype, dev, stream)
    _need(out, "out", (nmix, B, T, C), x.dtype, dev)
    if x_last is None and want_last:
        x_last = _empty((B, C), x.dtype, dev, stream)
    _need(x_last, "x_last", (B, C), x.dtype, dev)
    _check(lib().wkv_token_shift(B, T, C, code, nmix, _ptr(x), _ptr(mu), _ptr(x_prev), _ptr(out), _ptr(x_last),
                                 _stream_ptr(stream, dev)), "wkv_token_shift")
    return out, x_last


def wkv_step(w, u, k, v, state, r=None, *, y=None, stream=None):
    """RNN mode: one token for L layers.  w, u: (L, C) float32; k, v, r:
    (L, B, C); state: (L, 3, B, C) float32, updated in place.  Returns y."""
    torch = _torch()
    if k.dim() != 3:
        raise ValueError("k must be (L, B, C)")
    Lr, B, C = k.shape
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("wkv_step runs on CUDA tensors only")
    code = _dtype_code(k)
    _need(v, "v", (Lr, B, C), k.dtype, dev)
    _need(r, "r", (Lr, B, C), k.dtype, dev)
    _need(w, "w", (Lr, C), torch.float32, dev)
    _need(u, "u", (Lr, C), torch.float32, dev)
    _need(state, "state", (Lr, 3, B, C), torch.float32, dev)
    if y is None:
        y = _empty((Lr, B, C), k.dtype, dev, stream)
    _need(y, "y", (Lr, B, C), k.dtype, dev)
    _check(lib().wkv_step(Lr, B, C, code, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(state), _ptr(y),
                          _stream_ptr(stream, dev)), "wkv_step")
    return y


def _launch(dev, where, fn, *args):
    """fn(*args) with `dev` as the current device (the library launches on the
    current one); raises on a non-zero status."""
    torch = _torch()
    if dev.index == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != 0:
        raise WkvError(status, where)


def _delta_sizes(k, v, H, where):
    """(lead sizes, Hk, N) of k (., ., Hk * N) and v (., ., H * N)."""
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"{where}: k and v must have three dimensions")
    if H <= 0 or v.shape[2] % H != 0 or v.shape[2] == 0:
        raise ValueError(f"{where}: v's {v.shape[2]} channels are not {H} heads")
    N = v.shape[2] // H
    if k.shape[2] % N != 0 or k.shape[2] == 0 or H % (k.shape[2] // N) != 0:
        raise ValueError(f"{where}: k's {k.shape[2]} channels are not heads of {N} that {H} value heads share evenly")
    if k.device.type != "cuda":
        raise ValueError(f"{where} runs on CUDA tensors only")
    return v.shape[0], v.shape[1], k.shape[2] // N, N


def wkv_delta_forward(w, beta, r, k, v, H, state_in=None, *, y=None, state_out=None, want_state=True,
                      workspace: Workspace = None, use_workspace=True, stream=None):
    """Gated delta rule over one chunk.  r, k: (B, T, Hk * N), v: (B, T, H * N)
    float32 or bfloat16 CUDA tensors, N in {32, 64, 128} and H a multiple of
    Hk (value head h takes key head h // (H // Hk)); w (decay rates, inf
    forgets the state), beta: (B, T, H) float32; state_in: (B, H, N, N)
    float32 or None (zeros).  Per head
        e_t = v_t - exp(-w_t) S^T k_t,  S <- exp(-w_t) S + beta_t k_t e_t^T,  y_t = S^T r_t.
    Returns (y, state_out); state_out may be state_in.  use_workspace=False
    passes no workspace (one CTA a head's slice, whatever the number of heads).
    A wait on the GPU that ran out leaves NaN; wkv_delta_status() tells, and
    the workspace's status()."""
    torch = _torch()
    B, T, Hk, N = _delta_sizes(k, v, H, "wkv_delta_forward")
    dev, dt, f32 = k.device, k.dtype, torch.float32
    code = _dtype_code(k)
    keys, values, scalars, states = (B, T, Hk * N), (B, T, H * N), (B, T, H), (B, H, N, N)
    _need(r, "r", keys, dt, dev)
    _need(k, "k", keys, dt, dev)
    _need(v, "v", values, dt, dev)
    _need(w, "w", scalars, f32, dev)
    _need(beta, "beta", scalars, f32, dev)
    _need(state_in, "state_in", states, f32, dev)
    if y is None:
        y = _empty_like(v, stream)
    else:
        _need(y, "y", values, dt, dev)
    if state_out is not None:
        _need(state_out, "state_out", states, f32, dev)
    elif want_state:
        state_out = _empty(states, f32, dev, stream) if state_in is None else _empty_like(state_in, stream)
    ws_ptr, ws_bytes, owner = None, 0, None
    if use_workspace and B * H > 64:   # fewer heads never need one
        nbytes = int(lib().wkv_delta_forward_workspace_bytes(B, T, H, N))
        ws_ptr, ws_bytes, owner = _scratch(nbytes, workspace, dev, stream)
    _launch(dev, "wkv_delta_forward", lib().wkv_delta_forward, B, T, Hk, H, N, code, _ptr(w), _ptr(beta), _ptr(r), _ptr(k),
            _ptr(v), _ptr(state_in), _ptr(y), _ptr(state_out), ws_ptr, ws_bytes, _stream_ptr(stream, dev))
    return y, state_out


def wkv_delta_step(w, beta, r, k, v, state, *, y=None, stream=None):
    """Gated delta rule, one token for L layers of B sequences: r, k
    (L, B, Hk * N), v (L, B, H * N), w, beta (L, B, H) float32, state
    (L, B, H, N, N) float32 updated in place.  Returns y (L, B, H * N)."""
    torch = _torch()
    if state.dim() != 5:
        raise ValueError("state must be (L, B, H, N, N)")
    H = state.shape[2]
    Lr, B, Hk, N = _delta_sizes(k, v, H, "wkv_delta_step")
    dev, dt, f32 = k.device, k.dtype, torch.float32
    code = _dtype_code(k)
    keys, values, scalars = (Lr, B, Hk * N), (Lr, B, H * N), (Lr, B, H)
    _need(r, "r", keys, dt, dev)
    _need(k, "k", keys, dt, dev)
    _need(v, "v", values, dt, dev)
    _need(w, "w", scalars, f32, dev)
    _need(beta, "beta", scalars, f32, dev)
    _need(state, "state", (Lr, B, H, N, N), f32, dev)
    if y is None:
        y = _empty_like(v, stream)
    else:
        _need(y, "y", values, dt, dev)
    _launch(dev, "wkv_delta_step", lib().wkv_delta_step, Lr, B, Hk, H, N, code, _ptr(w), _ptr(beta), _ptr(r), _ptr(k), _ptr(v),
            _ptr(state), _ptr(y), _stream_ptr(stream, dev))
    return y


def _scratch(nbytes, workspace, dev, stream):
    """(pointer, bytes, owner) of `nbytes` of scratch that needs no clearing:
    the caller's Workspace, or memory of the current stream's pool that goes
    back to it when the call's kernels are queued."""
    if nbytes == 0:
        return None, 0, None
    if workspace is not None:
        return (*workspace.scratch(nbytes, stream, dev), None)
    torch = _torch()
    if stream is not None:
        with torch.cuda.stream(stream):
            buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return buf.data_ptr(), nbytes, buf


def wkv_delta_backward(w, beta, r, k, v, H, state_in=None, *, dy, dstate_out=None, dr=None, dk=None, dv=None, dw=None,
                       dbeta=None, dstate_in=None, want_dstate_in=True, workspace: Workspace = None, stream=None):
    """Gradients of wkv_delta_forward.  dy: (B, T, H * N) like v; dstate_out:
    (B, H, N, N) float32, the gradient of the returned state, or None.
    Returns (dr, dk, dv, dw, dbeta, dstate_in); dr and dk are summed over the
    value heads that share a key head, dw and dbeta are (B, T, H) float32."""
    torch = _torch()
    B, T, Hk, N = _delta_sizes(k, v, H, "wkv_delta_backward")
    dev, dt, f32 = k.device, k.dtype, torch.float32
    code = _dtype_code(k)
    keys, values, scalars, states = (B, T, Hk * N), (B, T, H * N), (B, T, H), (B, H, N, N)
    _need(r, "r", keys, dt, dev)
    _need(k, "k", keys, dt, dev)
    _need(v, "v", values, dt, dev)
    _need(dy, "dy", values, dt, dev)
    _need(w, "w", scalars, f32, dev)
    _need(beta, "beta", scalars, f32, dev)
    _need(state_in, "state_in", states, f32, dev)
    _need(dstate_out, "dstate_out", states, f32, dev)

    def out(t, name, shape, dtype, like):
        if t is None:
            return _empty_like(like, stream)
        _need(t, name, shape, dtype, dev)
        return t

    dr, dk, dv = out(dr, "dr", keys, dt, k), out(dk, "dk", keys, dt, k), out(dv, "dv", values, dt, v)
    dw, dbeta = out(dw, "dw", scalars, f32, w), out(dbeta, "dbeta", scalars, f32, w)
    if dstate_in is not None:
        _need(dstate_in, "dstate_in", states, f32, dev)
    elif want_dstate_in:
        dstate_in = _empty(states, f32, dev, stream) if state_in is None else _empty_like(state_in, stream)
    nbytes = int(lib().wkv_delta_backward_workspace_bytes(B, T, Hk, H, N))
    ws_ptr, ws_bytes, owner = _scratch(nbytes, workspace, dev, stream)
    _launch(dev, "wkv_delta_backward", lib().wkv_delta_backward, B, T, Hk, H, N, code, _ptr(w), _ptr(beta), _ptr(r), _ptr(k),
            _ptr(v), _ptr(state_in), _ptr(dy), _ptr(dstate_out), _ptr(dr), _ptr(dk), _ptr(dv), _ptr(dw), _ptr(dbeta),
            _ptr(dstate_in), ws_ptr, ws_bytes, _stream_ptr(stream, dev))
    return dr, dk, dv, dw, dbeta, dstate_in


def wkv_delta_status(*, clear=False, stream=None, device=None) -> int:
    """Synchronise the stream (of `device`, the current one): 0, or
    WKV_ERR_TIMEOUT (-7) if a wait of a delta rule call on the device has run
    out since the last call with clear=True, with whatever workspace or none."""
    torch = _torch()
    with torch.cuda.device(device):   # None: the current one
        return int(lib().wkv_delta_status(int(clear), _stream_ptr(stream, None)))


_ACTS = {"none": 0, "silu": 1, "sigmoid": 2}


def _norm_args(x, G, weight, bias, gate, act, where):
    if x.dim() < 1 or G <= 0 or x.shape[-1] % G != 0:
        raise ValueError(f"{where}: x's channels are not {G} groups")
    if act not in _ACTS:
        raise ValueError(f"{where}: act must be one of {sorted(_ACTS)}")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError(f"{where} runs on CUDA tensors only")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    C, f32 = x.shape[-1], _torch().float32
    _need(gate, "gate", x.shape, x.dtype, dev)
    _need(weight, "weight", (C,), f32, dev)
    _need(bias, "bias", (C,), f32, dev)
    return x.numel() // C if C else 0, C, dev, _dtype_code(x)


def wkv_group_norm(x, G, weight=None, bias=None, gate=None, *, act="none", eps=1e-5, y=None, stream=None):
    """Group norm with an activation, channels last: x (..., C) float32 or
    bfloat16, each token's channels in G groups normalised by their own mean
    and variance, z = weight * hat + bias (weight, bias (C,) float32 or None);
    y = act(z), or z * act(gate) with a gate like x.  act: "none", "silu" or
    "sigmoid".  Returns y."""
    rows, C, dev, code = _norm_args(x, G, weight, bias, gate, act, "wkv_group_norm")
    if y is None:
        y = _empty_like(x, stream)
    else:
        _need(y, "y", x.shape, x.dtype, dev)
    _launch(dev, "wkv_group_norm", lib().wkv_group_norm, rows, C, G, code, _ACTS[act], eps, _ptr(x), _ptr(weight), _ptr(bias),
            _ptr(gate), _ptr(y), _stream_ptr(stream, dev))
    return y


def wkv_group_norm_backward(x, G, weight=None, bias=None, gate=None, *, dy, act="none", eps=1e-5, dx=None, dweight=None,
                            dbias=None, dgate=None, workspace: Workspace = None, stream=None):
    """Gradients of wkv_group_norm: (dx, dweight, dbias, dgate), dweight and
    dbias (C,) float32 sums over the tokens; the gradient of an argument that
    is None is None."""
    torch = _torch()
    rows, C, dev, code = _norm_args(x, G, weight, bias, gate, act, "wkv_group_norm_backward")
    _need(dy, "dy", x.shape, x.dtype, dev)
    for t, g, name in ((weight, dweight, "dweight"), (bias, dbias, "dbias"), (gate, dgate, "dgate")):
        if t is None and g is not None:
            raise ValueError(f"{name}: there is no {name[1:]}")
    if dx is None:
        dx = _empty_like(x, stream)
    if gate is not None and dgate is None:
        dgate = _empty_like(x, stream)
    if weight is not None and dweight is None:
        dweight = _empty((C,), torch.float32, dev, stream)
    if bias is not None and dbias is None:
        dbias = _empty((C,), torch.float32, dev, stream)
    _need(dx, "dx", x.shape, x.dtype, dev)
    _need(dgate, "dgate", x.shape, x.dtype, dev)
    for t, name in ((dweight, "dweight"), (dbias, "dbias")):
        _need(t, name, (C,), torch.float32, dev)
    nbytes = 0
    if weight is not None or bias is not None:
        nbytes = int(lib().wkv_group_norm_backward_workspace_bytes(rows, C, G, code))
    ws_ptr, ws_bytes, owner = _scratch(nbytes, workspace, dev, stream)
    _launch(dev, "wkv_group_norm_backward", lib().wkv_group_norm_backward, rows, C, G, code, _ACTS[act], eps, _ptr(x),
            _ptr(weight), _ptr(bias), _ptr(gate), _ptr(dy), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(dgate), ws_ptr, ws_bytes,
            _stream_ptr(stream, dev))
    return dx, dweight, dbias, dgate

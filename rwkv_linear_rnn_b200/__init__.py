"""libwkv: the RWKV-4 WKV time-mixing operator on NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI in ``include/wkv.h`` and
``include/linattn.h`` (causal linear attention: ``linattn_forward``,
``linattn_backward``; with a decay for each head: ``linattn_decay_forward``,
``linattn_decay_backward``, ``linattn_decay_step``; rotary positions:
``linattn_rotary``).  The functions in
``abi`` carry the C names and take raw device pointers (ints) -- argument
marshalling only.  The tensor helpers below (``forward``, ``backward``,
``step``, ``WKV``, ``backward_state``, ``token_shift`` and the gated ``forward_gated``, ``backward_gated``,
``GatedWKV``) take torch CUDA tensors, allocate outputs with torch, and
call the same entry points; PyTorch provides memory and streams only, every
step of the operator runs in the library's CUDA kernels.

The library is required: importing this package fails loudly if
``libwkv.so`` is missing (build it with ``python -m rwkv_linear_rnn_b200.build``).
There is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import array
import functools
import importlib
import math

from .constants import (WKV_BF16, WKV_F32, WKV_KERNEL_AUTO, WKV_KERNEL_CHUNKED,
                        WKV_KERNEL_CLUSTER, WKV_KERNEL_SEGMENT, WKV_KERNEL_TILE, WKV_KERNEL_CHAIN,
                        WKV_KERNEL_CHUNKED_REGS, WKV_KERNEL_SEQUENTIAL, WKV_OP_BACKWARD,
                        WKV_OP_FORWARD, WKV_OP_STEP, WKV_STATIC_SCRATCH_BYTES)

__all__ = [
    "abi", "WKVError", "WKV_F32", "WKV_BF16", "WKV_OP_FORWARD", "WKV_OP_BACKWARD", "WKV_OP_STEP",
    "WKV_KERNEL_AUTO", "WKV_KERNEL_SEQUENTIAL", "WKV_KERNEL_CHUNKED", "WKV_KERNEL_CHUNKED_REGS",
    "WKV_KERNEL_SEGMENT", "WKV_KERNEL_CLUSTER", "WKV_KERNEL_TILE", "WKV_KERNEL_CHAIN", "WKV_STATIC_SCRATCH_BYTES", "Workspace", "forward", "backward", "backward_state", "step", "token_shift",
    "token_shift_backward", "TokenShift",
    "forward_gated", "backward_gated", "WKV", "wkv", "WKVState", "wkv_state", "GatedWKV", "gated_wkv", "wkv_workspace_size", "wkv_ckpt_size", "wkv_strerror", "wkv_version",
    "library_path", "LINATTN_OP_FORWARD", "LINATTN_OP_BACKWARD", "linattn_workspace_size",
    "linattn_forward", "linattn_backward",
    "linattn_decay_workspace_size", "linattn_decay_forward", "linattn_decay_backward", "linattn_decay_step",
    "linattn_decay_status", "LinattnDecay", "linattn_decay", "linattn_decay_state",
    "rotary_frequencies", "linattn_rotary", "Rotary", "rotary",
]


def __getattr__(name):
    # The ctypes layer (and with it libwkv.so) loads on first use; it raises
    # ImportError with a build hint if the library has not been built.
    if name in ("abi", "WKVError"):
        abi_mod = importlib.import_module(".abi", __name__)
        return abi_mod if name == "abi" else abi_mod.WKVError
    raise AttributeError(name)


@functools.lru_cache(maxsize=None)
def _abi():
    return importlib.import_module(".abi", __name__)


def wkv_workspace_size(op, B, T, C, dtype):
    return _abi().wkv_workspace_size(op, B, T, C, dtype)


def wkv_ckpt_size(B, T, C):
    return _abi().wkv_ckpt_size(B, T, C)


def wkv_strerror(status):
    return _abi().wkv_strerror(status)


def wkv_version():
    return _abi().wkv_version()


def library_path() -> str:
    return _abi().LIB_PATH


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return WKV_F32
    if t.dtype == torch.bfloat16:
        return WKV_BF16
    raise TypeError(f"k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


class Workspace:
    """A zero-initialised device workspace that grows on demand.

    One workspace may serve forward and backward calls of any shape, as long
    as they are ordered on one stream.
    """

    def __init__(self, device=None):
        self.device = device
        self.buf = None

    def get(self, op, B, T, C, dtype):
        return self.get_bytes(wkv_workspace_size(op, B, T, C, dtype))

    def get_bytes(self, need):
        torch = _torch()
        if need == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < need:
            # zero-filled: the library requires a zeroed workspace before first use
            self.buf = torch.zeros(need + 256, dtype=torch.uint8, device=self.device or "cuda")
        return self.buf, self.buf.numel()

    def status(self, stream=None) -> int:
        """Device-side status of earlier calls (waits for the stream); clears it."""
        if self.buf is None:
            return 0
        return _abi().wkv_get_status(self.buf.data_ptr(), _stream(stream))


_default_ws = {}


def _ws_for(device, ws):
    if ws is not None:
        return ws
    key = str(device)
    if key not in _default_ws:
        _default_ws[key] = Workspace(device)
    return _default_ws[key]


def forward(w, u, k, v, state_in=None, *, want_state=False, want_ckpt=False, y=None,
            workspace=None, stream=None, kernel=WKV_KERNEL_AUTO):
    """y = WKV(w, u, k, v) for k, v [B, T, C]; optionally the final state and
    the checkpoints for ``backward``.  Returns (y, state_out, ckpt)."""
    torch = _torch()
    _check_cuda(w, u, k, v, state_in, y)
    B, T, C = k.shape
    dt = _dtype_code(k)
    if y is None:
        y = torch.empty_like(k)
    state_out = torch.empty((3, B, C), dtype=torch.float32, device=k.device) if want_state else None
    ckpt = None
    if want_ckpt:
        n = wkv_ckpt_size(B, T, C) // 4
        ckpt = torch.empty(max(n, 1), dtype=torch.float32, device=k.device)
    ws = _ws_for(k.device, workspace)
    buf, nbytes = ws.get(WKV_OP_FORWARD, B, T, C, dt)
    abi = _abi()
    opts = abi.Options(kernel=kernel)
    abi.check(abi.wkv_forward_ex(B, T, C, dt, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(state_in),
                                 _ptr(y), _ptr(state_out), _ptr(ckpt), _ptr(buf), nbytes,
                                 _stream(stream), opts))
    return y, state_out, ckpt


def backward(w, u, k, v, grad_y, state_in=None, ckpt=None, *, grad_k=None, grad_v=None,
             workspace=None, stream=None, kernel=WKV_KERNEL_AUTO):
    """Gradients (grad_w [C], grad_u [C], grad_k, grad_v) of L given grad_y.
    ``grad_k`` / ``grad_v`` may be given as output buffers (shape and dtype of k)."""
    torch = _torch()
    _check_cuda(w, u, k, v, grad_y, state_in, ckpt, grad_k, grad_v)
    B, T, C = k.shape
    dt = _dtype_code(k)
    gw = torch.empty(C, dtype=torch.float32, device=k.device)
    gu = torch.empty(C, dtype=torch.float32, device=k.device)
    gk = torch.empty_like(k) if grad_k is None else grad_k
    gv = torch.empty_like(v) if grad_v is None else grad_v
    ws = _ws_for(k.device, workspace)
    buf, nbytes = ws.get(WKV_OP_BACKWARD, B, T, C, dt)
    abi = _abi()
    opts = abi.Options(kernel=kernel)
    abi.check(abi.wkv_backward_ex(B, T, C, dt, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(grad_y),
                                  _ptr(state_in), _ptr(ckpt), _ptr(gw), _ptr(gu), _ptr(gk),
                                  _ptr(gv), _ptr(buf), nbytes, _stream(stream), opts))
    return gw, gu, gk, gv


def backward_state(w, u, k, v, grad_y, state_in=None, ckpt=None, *, state_out=None,
                   grad_state_out=None, want_grad_state_in=True, grad_k=None, grad_v=None,
                   workspace=None, stream=None, kernel=WKV_KERNEL_AUTO):
    """``backward`` with the state terms of a sequence split across calls.
    ``grad_state_out`` is dL/d(a, b, p) of the state after the last token,
    given in the representation ``state_out`` (only its p is read).  Returns
    (grad_w, grad_u, grad_k, grad_v, grad_state_in); grad_state_in is
    dL/d(a, b, p) of ``state_in`` as given (None unless wanted)."""
    torch = _torch()
    _check_cuda(w, u, k, v, grad_y, state_in, ckpt, state_out, grad_state_out, grad_k, grad_v)
    B, T, C = k.shape
    dt = _dtype_code(k)
    gw = torch.empty(C, dtype=torch.float32, device=k.device)
    gu = torch.empty(C, dtype=torch.float32, device=k.device)
    gk = torch.empty_like(k) if grad_k is None else grad_k
    gv = torch.empty_like(v) if grad_v is None else grad_v
    gs = torch.empty((3, B, C), dtype=torch.float32, device=k.device) if want_grad_state_in else None
    ws = _ws_for(k.device, workspace)
    buf, nbytes = ws.get(WKV_OP_BACKWARD, B, T, C, dt)
    abi = _abi()
    opts = abi.Options(kernel=kernel)
    abi.check(abi.wkv_backward_state_ex(B, T, C, dt, _ptr(w), _ptr(u), _ptr(k), _ptr(v),
                                        _ptr(grad_y), _ptr(state_in), _ptr(ckpt), _ptr(state_out),
                                        _ptr(grad_state_out), _ptr(gw), _ptr(gu), _ptr(gk),
                                        _ptr(gv), _ptr(gs), _ptr(buf), nbytes, _stream(stream),
                                        opts))
    return gw, gu, gk, gv, gs


# ------------------------------------------------ causal linear attention ---

LINATTN_OP_FORWARD, LINATTN_OP_BACKWARD = 0, 1


def linattn_workspace_size(op, BH, N, D, M):
    return _abi().linattn_workspace_size(op, BH, N, D, M)


def _check_linattn(q, k, v, *more):
    torch = _torch()
    _check_cuda(q, k, v, *more)
    for t in (q, k, v) + tuple(x for x in more if x is not None):
        if t.dtype != torch.bfloat16 or t.dim() != 3:
            raise ValueError("linear attention takes bfloat16 [BH, N, D] tensors")
    BH, N, D = q.shape
    if k.shape != q.shape or v.shape[:2] != (BH, N):
        raise ValueError("q, k must be [BH, N, D] and v [BH, N, M]")
    return BH, N, D, v.shape[2]


def linattn_forward(q, k, v, *, want_state=False, out=None, workspace=None, stream=None):
    """Causal linear attention (elu + 1 feature map) for q, k [BH, N, D] and
    v [BH, N, M], bfloat16 (include/linattn.h).  Returns (out [BH, N, M],
    state or None) with state = (S [BH, D, M], Z [BH, D]) float32 after the
    last position."""
    torch = _torch()
    BH, N, D, M = _check_linattn(q, k, v, out)
    if out is None:
        out = torch.empty((BH, N, M), dtype=torch.bfloat16, device=q.device)
    st = torch.empty(BH * (D * M + D), dtype=torch.float32, device=q.device) if want_state else None
    ws = _ws_for(q.device, workspace)
    # backward-sized, so that linattn_backward(..., out=out) can reuse the
    # state this call leaves in the workspace
    buf, nbytes = ws.get_bytes(linattn_workspace_size(LINATTN_OP_BACKWARD, BH, N, D, M))
    abi = _abi()
    abi.check(abi.linattn_forward(BH, N, D, M, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(st),
                                  _ptr(buf), nbytes, _stream(stream)))
    if st is not None:
        st = (st[:BH * D * M].view(BH, D, M), st[BH * D * M:].view(BH, D))
    return out, st


def linattn_backward(q, k, v, grad_out, *, out=None, grad_q=None, grad_k=None, grad_v=None, workspace=None,
                     stream=None):
    """Gradients (grad_q, grad_k, grad_v) of L given grad_out = dL/dV'.

    With ``out`` (the output of the ``linattn_forward`` call on these q, k, v
    that used the same workspace, with no call on it since), the forward's
    saved chunk states and denominators are reused instead of recomputed
    (``linattn_backward_saved``)."""
    torch = _torch()
    BH, N, D, M = _check_linattn(q, k, v, grad_out, out, grad_q, grad_k, grad_v)
    grad_q = torch.empty_like(q) if grad_q is None else grad_q
    grad_k = torch.empty_like(k) if grad_k is None else grad_k
    grad_v = torch.empty_like(v) if grad_v is None else grad_v
    ws = _ws_for(q.device, workspace)
    buf, nbytes = ws.get_bytes(linattn_workspace_size(LINATTN_OP_BACKWARD, BH, N, D, M))
    abi = _abi()
    if out is not None:
        abi.check(abi.linattn_backward_saved(BH, N, D, M, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(grad_out),
                                             _ptr(grad_q), _ptr(grad_k), _ptr(grad_v), _ptr(buf), nbytes,
                                             _stream(stream)))
    else:
        abi.check(abi.linattn_backward(BH, N, D, M, _ptr(q), _ptr(k), _ptr(v), _ptr(grad_out), _ptr(grad_q),
                                       _ptr(grad_k), _ptr(grad_v), _ptr(buf), nbytes, _stream(stream)))
    return grad_q, grad_k, grad_v


# ------------------------- linear attention with a decay for each head ---

def linattn_decay_workspace_size(op, B, T, H, D, M, dtype):
    return _abi().linattn_decay_workspace_size(op, B, T, H, D, M, dtype)


def _scope(t, stream):
    """Context in which allocations and launches go to ``stream`` (default: the
    current stream) of the tensor's device."""
    torch = _torch()
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=t.device)
        return torch.cuda.stream(stream)
    return torch.cuda.device(t.device)


_decay_status = {}  # device index -> (the device's status word, its address)


class _Word:
    """The int32 at a device address, for torch.as_tensor."""

    def __init__(self, address):
        self.__cuda_array_interface__ = dict(shape=(1,), typestr="<i4", data=(address, False), strides=None, version=2)


def _status_ptr(dev):
    """Address of the status word of ``dev``, the current device.  It is shared by every call (kernels only
    ever store an error there), captured ones too, and belongs to the library."""
    known = _decay_status.get(dev)
    if known is None:
        torch = _torch()
        address = _abi().linattn_decay_status_word()
        if torch.cuda.is_current_stream_capturing():
            return address  # the tensor can wait
        with torch.inference_mode(False):  # cleared in place, in whatever mode it is read
            t = torch.as_tensor(_Word(address), device=f"cuda:{dev}")
        known = _decay_status.setdefault(dev, (t, address))
    return known[1]


def linattn_decay_status(device=None):
    """Device-side status of the ``linattn_decay_*`` calls made so far, replayed ones among them (0, or
    WKV_ERR_TIMEOUT if a bounded wait gave up); waits for the device and clears it."""
    torch = _torch()
    device = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if device.index is None else device.index
    with torch.cuda.device(index):
        _status_ptr(index)
        t = _decay_status[index][0]
        torch.cuda.synchronize(index)
        rc = int(t.item())
        if rc:
            t.zero_()
    return rc


# The checks below are most of a short call's time: they compare each property
# once and gather the views on the way.

def _head_view(words, name, t, dev, dtype, shape):
    """Appends the linattn_view of ``t``, which is of ``shape`` (4 or, for single tokens, 3 dimensions) and
    ``dtype`` on device ``dev`` with a contiguous last dimension."""
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors must be on one CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    words += (t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else (t.data_ptr(), s[0], 0, s[1])


def _plain_ptr(name, t, dev, dtype, shape):
    """Address of a contiguous tensor of ``shape`` and ``dtype`` on device ``dev``; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors must be on one CUDA device")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_device(q):
    """q's device index, which must be a CUDA device's, and whether it is the current one."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be on one CUDA device")
    return dev, dev == _torch().cuda.current_device()


@functools.lru_cache(maxsize=1024)
def _decay_need(dev, op, B, T, H, D, M, dt):
    # it depends on the current device's size too: callers have made dev current
    return _abi().linattn_decay_workspace_size(op, B, T, H, D, M, dt)


def _written(given):
    """Tells autograd that the library wrote into these of the caller's tensors (None: it had none to give), as
    torch's own in-place operations do: a graph that saved one refuses its backward."""
    given = [t for t in given if t is not None]
    if given:
        _torch().autograd.graph.increment_version(given)


def _scratch(ref, nbytes):
    # per call, from torch's stream-ordered allocator: calls on other streams,
    # in other threads or in captured graphs never share it
    return ref.new_empty(nbytes, dtype=_torch().uint8) if nbytes else None


def _prompt_shape(q, v):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [B, T, H, D] and v [B, T, H, M]")
    return (*q.shape, v.shape[3])


def linattn_decay_forward(q, k, v, log_decay, state=None, *, scale=1.0, lengths=None, want_state=False, out=None,
                          stream=None):
    """Linear attention with a decay for each head (include/linattn.h):
    out_t = scale * q_t^T S_t with S_t = e^{log_decay[h]} S_{t-1} + k_t v_t^T, for q, k [B, T, H, D] and
    v [B, T, H, M] (float32 or bfloat16; any strides with a contiguous last dimension), log_decay [H]
    float32 <= 0, the state before position 0 (``state`` [B, H, D, M] float32, or empty) and each row's
    number of positions (``lengths`` [B] int32, or T for all; out is zero behind them).  Keys and values that
    heads share are faster as copies than expanded (strides of 0 keep off the tensor cores).  Returns
    (out [B, T, H, M], the state after each row's last position or None)."""
    torch = _torch()
    dev, current = _on_device(q)
    if stream is not None or not current:
        with _scope(q, stream):
            return linattn_decay_forward(q, k, v, log_decay, state, scale=scale, lengths=lengths,
                                         want_state=want_state, out=out)
    B, T, H, D, M = _prompt_shape(q, v)
    dtype, f32 = q.dtype, torch.float32
    dt = _dtype_code(q)
    at = []
    _head_view(at, "q", q, dev, dtype, (B, T, H, D))
    _head_view(at, "k", k, dev, dtype, (B, T, H, D))
    _head_view(at, "v", v, dev, dtype, (B, T, H, M))
    given = out
    if out is None:
        out = q.new_empty((B, T, H, M))
    _head_view(at, "out", out, dev, dtype, (B, T, H, M))
    g = _plain_ptr("log_decay", log_decay, dev, f32, (H,))
    n = _plain_ptr("lengths", lengths, dev, torch.int32, (B,))
    s_in = _plain_ptr("state", state, dev, f32, (B, H, D, M))
    s_out = q.new_empty((B, H, D, M), dtype=f32) if want_state else None
    need = _decay_need(dev, LINATTN_OP_FORWARD, B, T, H, D, M, dt)
    ws = _scratch(q, need)
    at = array.array("q", at)
    w, abi = at.buffer_info()[0], _abi()
    rc = abi.linattn_decay_forward_at(B, T, H, D, M, dt, w, w + 32, w + 64, g, scale, n, s_in, w + 96, _ptr(s_out),
                                      _ptr(ws), need, _status_ptr(dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        abi.check(rc)
    if given is not None:
        _written((given,))
    return out, s_out


def linattn_decay_backward(q, k, v, log_decay, grad_out, state=None, *, scale=1.0, lengths=None, grad_state_out=None,
                           want_grad_state=False, grad_q=None, grad_k=None, grad_v=None, stream=None):
    """Gradients (grad_q, grad_k, grad_v, grad_state or None) of L for ``linattn_decay_forward`` with the same
    arguments, given grad_out = dL/dout and, optionally, ``grad_state_out`` = dL/d(state after the last
    position); grad_state is dL/dstate.  log_decay is a constant."""
    torch = _torch()
    dev, current = _on_device(q)
    if stream is not None or not current:
        with _scope(q, stream):
            return linattn_decay_backward(q, k, v, log_decay, grad_out, state, scale=scale, lengths=lengths,
                                          grad_state_out=grad_state_out, want_grad_state=want_grad_state,
                                          grad_q=grad_q, grad_k=grad_k, grad_v=grad_v)
    B, T, H, D, M = _prompt_shape(q, v)
    dtype, f32 = q.dtype, torch.float32
    dt = _dtype_code(q)
    wide_d, wide_m = (B, T, H, D), (B, T, H, M)
    at = []
    _head_view(at, "q", q, dev, dtype, wide_d)
    _head_view(at, "k", k, dev, dtype, wide_d)
    _head_view(at, "v", v, dev, dtype, wide_m)
    _head_view(at, "grad_out", grad_out, dev, dtype, wide_m)
    given = grad_q, grad_k, grad_v
    grad_q = q.new_empty(wide_d) if grad_q is None else grad_q
    grad_k = q.new_empty(wide_d) if grad_k is None else grad_k
    grad_v = q.new_empty(wide_m) if grad_v is None else grad_v
    _head_view(at, "grad_q", grad_q, dev, dtype, wide_d)
    _head_view(at, "grad_k", grad_k, dev, dtype, wide_d)
    _head_view(at, "grad_v", grad_v, dev, dtype, wide_m)
    g = _plain_ptr("log_decay", log_decay, dev, f32, (H,))
    n = _plain_ptr("lengths", lengths, dev, torch.int32, (B,))
    s_in = _plain_ptr("state", state, dev, f32, (B, H, D, M))
    gs_out = _plain_ptr("grad_state_out", grad_state_out, dev, f32, (B, H, D, M))
    gs = q.new_empty((B, H, D, M), dtype=f32) if want_grad_state else None
    need = _decay_need(dev, LINATTN_OP_BACKWARD, B, T, H, D, M, dt)
    ws = _scratch(q, need)
    at = array.array("q", at)
    w, abi = at.buffer_info()[0], _abi()
    rc = abi.linattn_decay_backward_at(B, T, H, D, M, dt, w, w + 32, w + 64, g, scale, n, s_in, w + 96, gs_out, w + 128,
                                       w + 160, w + 192, _ptr(gs), _ptr(ws), need, _status_ptr(dev),
                                       torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        abi.check(rc)
    _written(given)
    return grad_q, grad_k, grad_v, gs


def linattn_decay_step(q, k, v, log_decay, state, *, scale=1.0, out=None, state_out=None, stream=None):
    """One token for N sequences: q, k [N, H, D], v [N, H, M], state [N, H, D, M] float32.  ``state_out``
    defaults to updating ``state`` in place.  Returns (out [N, H, M], state_out)."""
    torch = _torch()
    dev, current = _on_device(q)
    if stream is not None or not current:
        with _scope(q, stream):
            return linattn_decay_step(q, k, v, log_decay, state, scale=scale, out=out, state_out=state_out)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k must be [N, H, D] and v [N, H, M]")
    N, H, D = q.shape
    M = v.shape[2]
    dtype, f32 = q.dtype, torch.float32
    at = []
    _head_view(at, "q", q, dev, dtype, (N, H, D))
    _head_view(at, "k", k, dev, dtype, (N, H, D))
    _head_view(at, "v", v, dev, dtype, (N, H, M))
    given = out
    if out is None:
        out = q.new_empty((N, H, M))
    _head_view(at, "out", out, dev, dtype, (N, H, M))
    g = _plain_ptr("log_decay", log_decay, dev, f32, (H,))
    s_in = _plain_ptr("state", state, dev, f32, (N, H, D, M))
    if state_out is None:
        state_out = state
    s_out = s_in if state_out is state else _plain_ptr("state_out", state_out, dev, f32, (N, H, D, M))
    at = array.array("q", at)
    w, abi = at.buffer_info()[0], _abi()
    rc = abi.linattn_decay_step_at(N, H, D, M, _dtype_code(q), w, w + 32, w + 64, g, scale, s_in, w + 96, s_out,
                                   torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        abi.check(rc)
    torch.autograd.graph.increment_version(state_out if given is None else (state_out, given))  # as _written
    return out, state_out


def _rows(t):
    """A gradient or argument as the library takes it: expanded or transposed
    ones are copied."""
    if t is None or (t.stride(-1) == 1 and all(s > 0 or n <= 1 for s, n in zip(t.stride(), t.shape))):
        return t
    return t.contiguous()


def _state(t):
    """A state or its gradient as the library takes it: slices that are not contiguous, or not 16-byte aligned
    (of odd sizes, or a gradient cut from a larger one), are copied."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class LinattnDecay:
    """torch.autograd.Function wrapper: (out, state_out) = LinattnDecay.apply(q, k, v, log_decay, state,
    lengths, scale).  Gradients reach state through both out and state_out, so a sequence split across
    calls back-propagates through the state (truncated BPTT)."""

    _fn = None

    @classmethod
    def apply(cls, q, k, v, log_decay, state=None, lengths=None, scale=1.0, want_state=True):
        if log_decay.requires_grad and _torch().is_grad_enabled():
            raise ValueError("log_decay is a constant of linattn_decay: it has no gradient (detach it)")
        if cls._fn is None:
            torch = _torch()
            from torch.autograd.function import once_differentiable

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, q, k, v, log_decay, state, lengths, scale, want_state):
                    ctx.set_materialize_grads(False)
                    q, k, v = _rows(q), _rows(k), _rows(v)
                    state = _state(state)
                    out, s_out = linattn_decay_forward(q, k, v, log_decay, state, scale=scale, lengths=lengths,
                                                       want_state=want_state)
                    ctx.save_for_backward(q, k, v, log_decay, state, lengths)
                    ctx.scale = scale
                    return out, s_out

                @staticmethod
                @once_differentiable
                def backward(ctx, go, gs):
                    q, k, v, log_decay, state, lengths = ctx.saved_tensors
                    go = torch.zeros_like(v) if go is None else go
                    gq, gk, gv, gst = linattn_decay_backward(
                        q, k, v, log_decay, _rows(go), state, scale=ctx.scale, lengths=lengths,
                        grad_state_out=_state(gs),
                        want_grad_state=state is not None and ctx.needs_input_grad[4])
                    return gq, gk, gv, None, gst, None, None, None

            cls._fn = _F
        return cls._fn.apply(q, k, v, log_decay, state, lengths, scale, want_state)


def linattn_decay(q, k, v, log_decay, state=None, *, lengths=None, scale=1.0):
    """Differentiable ``linattn_decay_forward``: out [B, T, H, M]."""
    return LinattnDecay.apply(q, k, v, log_decay, state, lengths, scale, False)[0]


def linattn_decay_state(q, k, v, log_decay, state=None, *, lengths=None, scale=1.0):
    """Differentiable ``linattn_decay_forward`` with the state: (out, state_out)."""
    return LinattnDecay.apply(q, k, v, log_decay, state, lengths, scale, True)


# ------------------------------------------------------- rotary positions ---

def rotary_frequencies(rotated, *, base=10000.0, scaling="none", factor=1.0, trained_length=None, fast_turns=32.0,
                       slow_turns=1.0, device=None):
    """The plan of ``linattn_rotary``: (inv_freq [rotated / 2] float64, mscale) with inv_freq[i] =
    base^(-2 i / rotated), stretched by ``factor`` for texts longer than those trained on:
    "linear"    every frequency divided by factor (positions compressed);
    "ntk"       base raised to base * factor^(rotated / (rotated - 2)): the slowest pair is stretched by
                factor, the fastest not at all;
    "by_parts"  pairs that turn more than ``fast_turns`` times over ``trained_length`` positions keep their
                frequency, those under ``slow_turns`` are divided by factor, linear in between; mscale =
                0.1 ln(factor) + 1."""
    torch = _torch()
    if rotated < 2 or rotated % 2:
        raise ValueError("rotated must be even and at least 2")
    if not (factor > 0 and base > 0):
        raise ValueError("factor and base must be positive")
    if scaling not in ("none", "linear", "ntk", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk" and rotated > 2:
        base = base * factor ** (rotated / (rotated - 2))
    f = float(base) ** (-torch.arange(0, rotated, 2, dtype=torch.float64) / rotated)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if not trained_length or fast_turns <= slow_turns:
            raise ValueError("by_parts needs trained_length and fast_turns > slow_turns")
        keep = ((trained_length * f / (2 * math.pi) - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return f.to("cuda" if device is None else device), mscale


def linattn_rotary(q, k, positions, inv_freq, *, mscale=1.0, interleaved=False, inverse=False, out_q=None, out_k=None,
                   stream=None):
    """Rotates the first 2 * len(inv_freq) elements of every head of q [B, T, Hq, D] and k [B, T, Hk, D] (or
    None) by ``positions`` ([B, T] or [T], int32 or int64) times ``inv_freq`` (float64, from
    ``rotary_frequencies``); pairs are (i, i + R/2), or (2i, 2i + 1) if ``interleaved``.  ``inverse``
    rotates back.  ``out_q`` / ``out_k`` may be q / k (in place).  Returns (out_q, out_k)."""
    torch = _torch()
    dev, current = _on_device(q)
    if stream is not None or not current:
        with _scope(q, stream):
            return linattn_rotary(q, k, positions, inv_freq, mscale=mscale, interleaved=interleaved, inverse=inverse,
                                  out_q=out_q, out_k=out_k)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [B, T, heads, D]")
    dtype, shape = q.dtype, q.shape
    B, T, Hq, D = shape
    if positions.dtype not in (torch.int32, torch.int64) or positions.shape not in ((T,), (B, T)):
        raise ValueError("positions must be int32 or int64, [T] or [B, T]")
    p_stride = positions.stride()
    if positions.get_device() != dev or (T > 1 and p_stride[-1] != 1):
        raise ValueError("positions must be on q's device, contiguous along T")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a float64 vector")
    pairs = inv_freq.shape[0]
    f = _plain_ptr("inv_freq", inv_freq, dev, torch.float64, (pairs,))
    given = out_q, out_k
    at = []
    _head_view(at, "q", q, dev, dtype, shape)
    if out_q is None:
        out_q = q.new_empty(shape)
    _head_view(at, "out_q", out_q, dev, dtype, shape)
    Hk = 0
    if k is not None:
        Hk = k.shape[2]
        k_shape = (B, T, Hk, D)
        _head_view(at, "k", k, dev, dtype, k_shape)
        if out_k is None:
            out_k = q.new_empty(k_shape)
        _head_view(at, "out_k", out_k, dev, dtype, k_shape)
    elif out_k is not None:
        raise ValueError("out_k without k")
    at = array.array("q", at)
    w, abi = at.buffer_info()[0], _abi()
    rc = abi.linattn_rotary_at(B, T, D, 2 * pairs, _dtype_code(q), Hq, w, Hk, w + 64 if Hk else None,
                               positions.data_ptr(), positions.element_size(),
                               p_stride[0] if len(p_stride) == 2 else 0, f, mscale, interleaved, inverse, w + 32,
                               w + 96 if Hk else None, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        abi.check(rc)
    _written(given)
    return out_q, out_k


class Rotary:
    """torch.autograd.Function wrapper: (q', k') = Rotary.apply(q, k, positions, inv_freq, mscale, interleaved);
    the gradient is the inverse rotation."""

    _fn = None

    @classmethod
    def apply(cls, q, k, positions, inv_freq, mscale=1.0, interleaved=False):
        if inv_freq.requires_grad and _torch().is_grad_enabled():
            raise ValueError("inv_freq is a constant of rotary: it has no gradient (detach it)")
        if cls._fn is None:
            torch = _torch()
            from torch.autograd.function import once_differentiable

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, q, k, positions, inv_freq, mscale, interleaved):
                    ctx.save_for_backward(positions, inv_freq)
                    ctx.how = dict(mscale=mscale, interleaved=interleaved)
                    return linattn_rotary(_rows(q), _rows(k), positions, inv_freq, **ctx.how)

                @staticmethod
                @once_differentiable
                def backward(ctx, gq, gk):
                    positions, inv_freq = ctx.saved_tensors
                    gq, gk = linattn_rotary(_rows(gq), _rows(gk), positions, inv_freq, inverse=True, **ctx.how)
                    return gq, gk, None, None, None, None

            cls._fn = _F
        return cls._fn.apply(q, k, positions, inv_freq, mscale, interleaved)


def rotary(q, k, positions, inv_freq, *, mscale=1.0, interleaved=False):
    """Differentiable ``linattn_rotary``: (q', k')."""
    return Rotary.apply(q, k, positions, inv_freq, mscale, interleaved)


def token_shift(x, mu, x_prev=None, *, out=None, stream=None):
    """out[m] = mu[m] * x[t] + (1 - mu[m]) * x[t-1] for x [B, T, C] and
    mu [n, C] (float32); x[-1] = x_prev [B, C] or 0.  Returns out [n, B, T, C]."""
    torch = _torch()
    _check_cuda(x, mu, x_prev, out)
    B, T, C = x.shape
    n = mu.shape[0]
    if out is None:
        out = torch.empty((n, B, T, C), dtype=x.dtype, device=x.device)
    abi = _abi()
    abi.check(abi.wkv_token_shift(B, T, C, _dtype_code(x), n, _ptr(mu), _ptr(x), _ptr(x_prev),
                                  _ptr(out), _stream(stream)))
    return out


def token_shift_backward(x, mu, grad_out, x_prev=None, *, want_grad_x_prev=False, stream=None):
    """Gradients (grad_x, grad_mu, grad_x_prev or None) of L given
    grad_out = dL/dout [n, B, T, C]."""
    torch = _torch()
    _check_cuda(x, mu, grad_out, x_prev)
    B, T, C = x.shape
    n = mu.shape[0]
    gx = torch.empty_like(x)
    gmu = torch.empty((n, C), dtype=torch.float32, device=x.device)
    gxp = torch.empty((B, C), dtype=x.dtype, device=x.device) if want_grad_x_prev else None
    abi = _abi()
    nws = abi.wkv_token_shift_workspace_size(B, T, C, n)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=x.device)
    abi.check(abi.wkv_token_shift_backward(B, T, C, _dtype_code(x), n, _ptr(mu), _ptr(x),
                                           _ptr(x_prev), _ptr(grad_out), _ptr(gx), _ptr(gmu),
                                           _ptr(gxp), _ptr(ws), nws, _stream(stream)))
    return gx, gmu, gxp


def forward_gated(w, u, k, v, r, state_in=None, *, want_state=False, want_ckpt=False, o=None,
                  workspace=None, stream=None, kernel=WKV_KERNEL_AUTO):
    """o = sigmoid(r) * WKV(w, u, k, v) for k, v, r [B, T, C].  Returns
    (o, state_out, ckpt) as ``forward`` does (the state and checkpoints are the
    WKV recurrence's)."""
    torch = _torch()
    _check_cuda(w, u, k, v, r, state_in, o)
    B, T, C = k.shape
    dt = _dtype_code(k)
    if o is None:
        o = torch.empty_like(k)
    state_out = torch.empty((3, B, C), dtype=torch.float32, device=k.device) if want_state else None
    ckpt = None
    if want_ckpt:
        n = wkv_ckpt_size(B, T, C) // 4
        ckpt = torch.empty(max(n, 1), dtype=torch.float32, device=k.device)
    ws = _ws_for(k.device, workspace)
    buf, nbytes = ws.get(WKV_OP_FORWARD, B, T, C, dt)
    abi = _abi()
    opts = abi.Options(kernel=kernel)
    abi.check(abi.wkv_forward_gated_ex(B, T, C, dt, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r),
                                       _ptr(state_in), _ptr(o), _ptr(state_out), _ptr(ckpt),
                                       _ptr(buf), nbytes, _stream(stream), opts))
    return o, state_out, ckpt


def backward_gated(w, u, k, v, r, grad_o, state_in=None, ckpt=None, *, grad_k=None, grad_v=None,
                   grad_r=None, workspace=None, stream=None, kernel=WKV_KERNEL_AUTO):
    """Gradients (grad_w, grad_u, grad_k, grad_v, grad_r) of L given
    grad_o = dL/do for o = sigmoid(r) * WKV(w, u, k, v)."""
    torch = _torch()
    _check_cuda(w, u, k, v, r, grad_o, state_in, ckpt, grad_k, grad_v, grad_r)
    B, T, C = k.shape
    dt = _dtype_code(k)
    gw = torch.empty(C, dtype=torch.float32, device=k.device)
    gu = torch.empty(C, dtype=torch.float32, device=k.device)
    gk = torch.empty_like(k) if grad_k is None else grad_k
    gv = torch.empty_like(v) if grad_v is None else grad_v
    gr = torch.empty_like(r) if grad_r is None else grad_r
    ws = _ws_for(k.device, workspace)
    buf, nbytes = ws.get(WKV_OP_BACKWARD, B, T, C, dt)
    abi = _abi()
    opts = abi.Options(kernel=kernel)
    abi.check(abi.wkv_backward_gated_ex(B, T, C, dt, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r),
                                        _ptr(grad_o), _ptr(state_in), _ptr(ckpt), _ptr(gw),
                                        _ptr(gu), _ptr(gk), _ptr(gv), _ptr(gr), _ptr(buf), nbytes,
                                        _stream(stream), opts))
    return gw, gu, gk, gv, gr


def step(w, u, k_t, v_t, state, *, y=None, state_out=None, stream=None):
    """One RNN-mode token for N sequences.  ``state_out`` defaults to updating
    ``state`` in place.  Returns (y_t, state_out)."""
    torch = _torch()
    _check_cuda(w, u, k_t, v_t, state, y, state_out)
    N, C = k_t.shape
    if y is None:
        y = torch.empty_like(k_t)
    if state_out is None:
        state_out = state
    abi = _abi()
    abi.check(abi.wkv_step(N, C, _ptr(w), _ptr(u), _ptr(k_t), _ptr(v_t), _ptr(state), _ptr(y),
                           _ptr(state_out), _stream(stream)))
    return y, state_out


class WKV:
    """torch.autograd.Function wrapper: y = WKV.apply(w, u, k, v)."""

    _fn = None

    @classmethod
    def apply(cls, w, u, k, v):
        if cls._fn is None:
            torch = _torch()

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, w, u, k, v):
                    w, u, k, v = (t.contiguous() for t in (w, u, k, v))
                    y, _, ck = forward(w, u, k, v, want_ckpt=True)
                    ctx.save_for_backward(w, u, k, v, ck)
                    return y

                @staticmethod
                def backward(ctx, gy):
                    w, u, k, v, ck = ctx.saved_tensors
                    gw, gu, gk, gv = backward(w, u, k, v, gy.contiguous(), ckpt=ck)
                    return gw, gu, gk, gv

            cls._fn = _F
        return cls._fn.apply(w, u, k, v)


def wkv(w, u, k, v):
    """Differentiable WKV: y [B, T, C] from w, u [C] and k, v [B, T, C]."""
    return WKV.apply(w, u, k, v)


class WKVState:
    """torch.autograd.Function wrapper with the recurrent state:
    (y, state_out) = WKVState.apply(w, u, k, v, state_in).  Gradients reach
    state_in through both y and state_out, so a sequence split across calls
    back-propagates through the state (truncated BPTT)."""

    _fn = None

    @classmethod
    def apply(cls, w, u, k, v, state_in):
        if cls._fn is None:
            torch = _torch()

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, w, u, k, v, state_in):
                    w, u, k, v, state_in = (t.contiguous() for t in (w, u, k, v, state_in))
                    y, s_out, ck = forward(w, u, k, v, state_in, want_state=True, want_ckpt=True)
                    ctx.save_for_backward(w, u, k, v, state_in, s_out, ck)
                    return y, s_out

                @staticmethod
                def backward(ctx, gy, gs):
                    w, u, k, v, state_in, s_out, ck = ctx.saved_tensors
                    gy = torch.zeros_like(k) if gy is None else gy.contiguous()
                    gs = None if gs is None else gs.contiguous()
                    return backward_state(w, u, k, v, gy, state_in, ck, state_out=s_out,
                                          grad_state_out=gs)

            cls._fn = _F
        return cls._fn.apply(w, u, k, v, state_in)


def wkv_state(w, u, k, v, state_in):
    """Differentiable WKV with the state: (y, state_out) from w, u [C],
    k, v [B, T, C] and state_in [3, B, C]."""
    return WKVState.apply(w, u, k, v, state_in)


class TokenShift:
    """torch.autograd.Function wrapper: out = TokenShift.apply(x, mu, x_prev)
    (x_prev may be None)."""

    _fn = None

    @classmethod
    def apply(cls, x, mu, x_prev=None):
        if cls._fn is None:
            torch = _torch()

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, mu, x_prev):
                    x, mu = x.contiguous(), mu.contiguous()
                    x_prev = None if x_prev is None else x_prev.contiguous()
                    ctx.save_for_backward(x, mu, x_prev)
                    return token_shift(x, mu, x_prev)

                @staticmethod
                def backward(ctx, g):
                    x, mu, x_prev = ctx.saved_tensors
                    gx, gmu, gxp = token_shift_backward(x, mu, g.contiguous(), x_prev,
                                                        want_grad_x_prev=x_prev is not None)
                    return gx, gmu, gxp

            cls._fn = _F
        return cls._fn.apply(x, mu, x_prev)


class GatedWKV:
    """torch.autograd.Function wrapper: o = GatedWKV.apply(w, u, k, v, r)."""

    _fn = None

    @classmethod
    def apply(cls, w, u, k, v, r):
        if cls._fn is None:
            torch = _torch()

            class _F(torch.autograd.Function):
                @staticmethod
                def forward(ctx, w, u, k, v, r):
                    w, u, k, v, r = (t.contiguous() for t in (w, u, k, v, r))
                    o, _, ck = forward_gated(w, u, k, v, r, want_ckpt=True)
                    ctx.save_for_backward(w, u, k, v, r, ck)
                    return o

                @staticmethod
                def backward(ctx, go):
                    w, u, k, v, r, ck = ctx.saved_tensors
                    return backward_gated(w, u, k, v, r, go.contiguous(), ckpt=ck)

            cls._fn = _F
        return cls._fn.apply(w, u, k, v, r)


def gated_wkv(w, u, k, v, r):
    """Differentiable gated WKV: sigmoid(r) * WKV(w, u, k, v)."""
    return GatedWKV.apply(w, u, k, v, r)

"""Short causal convolution and selective state space scan: Python binding.

Like the gated delta rule's calls these only marshal arguments for the C ABI
(``gdr_short_conv_*`` and ``gdr_ssm_scan_*`` in ``include/gdr.h``, which states
the formulas).  Differences in manner:

* Inputs may be strided views as long as their last dimension is dense
  (``Bm`` and ``Cm``: the last two), so slices of one projection and
  ``[B,T,H,d]`` rows seen as ``[B,H,T,d]`` need no copy.
* ``lengths`` (int32 ``[B]``) ends rows before T.  Behind a row's end inputs
  are not read and ``y`` is left as it is; a ``y`` made by the call is zero
  there.
* Outputs and workspaces are made on the stream that the call runs on.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _DTYPES, _check, _need, _to_device, _to_host, lib

_ACTIVATIONS = {None: 0, "silu": 1}
_I64x3 = ctypes.c_longlong * 3
_I64x5 = ctypes.c_longlong * 5
_I64x10 = ctypes.c_longlong * 10
_I64x12 = ctypes.c_longlong * 12


def _scoped(dev: torch.device, stream, body):
    """body(stream handle) with the device and the stream current that the call runs on."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return body(torch.cuda.current_stream().cuda_stream)
        with torch.cuda.device(dev):
            return body(torch.cuda.current_stream().cuda_stream)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _device(x: torch.Tensor) -> torch.device:
    return x.device if x.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, dtype, dev, dense: int = 1):
    """A tensor of the given shape whose last `dense` dimensions are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        step = 1
        for k in range(1, dense + 1):
            if t.shape[-k] != 1 and t.stride(-k) != step and t.numel():
                raise ValueError(f"the last dimension{'s' if dense > 1 else ''} of {name} must be contiguous")
            step *= t.shape[-k]


def _vector(t: Optional[torch.Tensor], name: str, shape, dev, dtype=torch.float32):
    if t is not None:
        _need(t, name, dtype, dev)
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _type_of(x: torch.Tensor):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    if x.dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16")
    return x.dtype


def _workspace(ws: Optional[torch.Tensor], size: int, dev):
    if not size:
        return None
    if ws is None or ws.numel() * ws.element_size() < size:
        return torch.empty(size, dtype=torch.uint8, device=dev)
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    return ws


# ------------------------------------------------------------- short convolution

def _conv_shape(x):
    """(B, H, T, d) of [B,H,T,d] or [B,T,D] (one head)."""
    if x.dim() == 4:
        return tuple(x.shape)
    if x.dim() == 3:
        B, T, D = x.shape
        return B, 1, T, D
    raise ValueError("x must be [B,H,T,d] or [B,T,D]")


def _conv_strides(x):
    s = x.stride()
    return _I64x3(s[0], s[1], s[2]) if len(s) == 4 else _I64x3(s[0], 0, s[1])


def _conv_params(weight, bias, activation, D, dev):
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu'")
    _need(weight, "weight", torch.float32, dev)
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be [{D},W], got {list(weight.shape)}")
    _vector(bias, "bias", (D,), dev)
    return weight.shape[1]


def short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   state: Optional[torch.Tensor] = None, activation: Optional[str] = "silu",
                   lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   state_out: Optional[torch.Tensor] = None, final_state: bool = True,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Short causal depthwise convolution over a prompt (``gdr_short_conv_fwd``).

    x [B,H,T,d] or [B,T,D] (D = H*d; fp32 or bf16, strided); weight fp32 [D,W], W in 2..4;
    bias fp32 [D]; state [B,W-1,D] in x's type: the rows before x, oldest first (None: zeros);
    activation "silu" or None; lengths int32 [B].  Returns (y, contiguous in x's shape and
    type, and the state after the prompt or None); ``state_out`` may be ``state``.
    """
    dt = _type_of(x)
    dev, host = _device(x), not x.is_cuda
    B, H, T, d = _conv_shape(x)
    D = H * d

    def body(handle, x=x, weight=weight, bias=bias, state=state, lengths=lengths, y=y, state_out=state_out):
        if host:
            x, weight, bias, state, lengths = (_to_device(t, dev) for t in (x, weight, bias, state, lengths))
        _rows(x, "x", x.shape, dt, dev)
        W = _conv_params(weight, bias, activation, D, dev)
        _vector(state, "state", (B, W - 1, D), dev, dt)
        _vector(lengths, "lengths", (B,), dev, torch.int32)
        if y is None:
            y = (torch.empty if lengths is None else torch.zeros)(x.shape, dtype=dt, device=dev)
        else:
            _vector(y, "y", x.shape, dev, dt)
        if state_out is not None:
            _vector(state_out, "state_out", (B, W - 1, D), dev, dt)
        elif final_state:
            state_out = torch.empty(B, max(W - 1, 0), D, dtype=dt, device=dev)
        _check(lib().gdr_short_conv_fwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(y), _ptr(state_out),
            _conv_strides(x), B, H, T, d, W, _ACTIVATIONS[activation], _DTYPES[dt], handle), "gdr_short_conv_fwd")
        return y, state_out

    out = _scoped(dev, stream, body)
    return tuple(_to_host(t) for t in out) if host else out


def short_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    activation: Optional[str] = "silu", y: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The convolution for one token per row (``gdr_short_conv_step``).

    x [B,D] (rows may be strided); state [B,W-1,D] in x's type is shifted IN PLACE; weight, bias
    and activation as ``short_conv_fwd``.  Returns y [B,D].
    """
    dt = _type_of(x)
    dev = x.device
    if not x.is_cuda:
        raise ValueError("short_conv_step works on CUDA tensors: the state is updated in place")
    if x.dim() != 2:
        raise ValueError("x must be [B,D]")
    B, D = x.shape
    _rows(x, "x", x.shape, dt, dev)
    W = _conv_params(weight, bias, activation, D, dev)
    _vector(state, "state", (B, W - 1, D), dev, dt)

    def body(handle, y=y):
        if y is None:
            y = torch.empty(B, D, dtype=dt, device=dev)
        else:
            _vector(y, "y", (B, D), dev, dt)
        _check(lib().gdr_short_conv_step(_ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), x.stride(0), B, D,
                                         W, _ACTIVATIONS[activation], _DTYPES[dt], handle), "gdr_short_conv_step")
        return y

    return _scoped(dev, stream, body)


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   state: Optional[torch.Tensor] = None, dstate_out: Optional[torch.Tensor] = None,
                   activation: Optional[str] = "silu", lengths: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of ``short_conv_fwd`` (``gdr_short_conv_bwd``): the gradients of
    <dy, y> + <dstate_out, state_out>.

    dy has x's shape and type (strided); dstate_out [B,W-1,D] or None (zeros).  Returns
    (dx, dweight fp32 [D,W], dbias fp32 [D] or None without a bias, dstate or None without a
    state).  dx has x's shape and its order in memory (token rows stay token rows); it is
    zero behind a row's end.
    """
    dt = _type_of(x)
    dev, host = _device(x), not x.is_cuda
    B, H, T, d = _conv_shape(x)
    D = H * d

    def body(handle, x=x, weight=weight, dy=dy, bias=bias, state=state, dstate_out=dstate_out, lengths=lengths):
        if host:
            x, weight, dy, bias, state, dstate_out, lengths = (
                _to_device(t, dev) for t in (x, weight, dy, bias, state, dstate_out, lengths))
        _rows(x, "x", x.shape, dt, dev)
        _rows(dy, "dy", x.shape, dt, dev)
        W = _conv_params(weight, bias, activation, D, dev)
        _vector(state, "state", (B, W - 1, D), dev, dt)
        _vector(dstate_out, "dstate_out", (B, W - 1, D), dev, dt)
        _vector(lengths, "lengths", (B,), dev, torch.int32)
        if x.dim() == 4 and x.stride(1) < x.stride(2):
            dx = torch.empty(B, T, H, d, dtype=dt, device=dev).transpose(1, 2)
        else:
            dx = torch.empty(x.shape, dtype=dt, device=dev)
        dweight = torch.empty(D, W, dtype=torch.float32, device=dev)
        dbias = None if bias is None else torch.empty(D, dtype=torch.float32, device=dev)
        dstate = None if state is None else torch.empty(B, W - 1, D, dtype=dt, device=dev)
        L = lib()
        size = L.gdr_short_conv_bwd_workspace_size(B, H, T, d, W, _DTYPES[dt])
        ws = _workspace(workspace, size, dev)
        _check(L.gdr_short_conv_bwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(dy), _ptr(dstate_out), _ptr(dx),
            _ptr(dweight), _ptr(dbias), _ptr(dstate), _conv_strides(x), _conv_strides(dy), _conv_strides(dx),
            B, H, T, d, W, _ACTIVATIONS[activation], _DTYPES[dt], _ptr(ws), size, handle), "gdr_short_conv_bwd")
        return dx, dweight, dbias, dstate

    out = _scoped(dev, stream, body)
    return tuple(_to_host(t) for t in out) if host else out


# ------------------------------------------------------------ state space scan

def _scan_inputs(x, dt_, A, Bm, Cm, D_skip, z, dt_bias, lead, dev):
    """Checks what the three scan calls share; returns (G, N)."""
    dt, D = x.dtype, x.shape[-1]
    _rows(x, "x", x.shape, dt, dev)
    _rows(dt_, "dt", x.shape, dt, dev)
    if z is not None:
        _rows(z, "z", x.shape, dt, dev)
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != len(lead) + 2:
        raise ValueError(f"Bm and Cm must be [{'B,T' if len(lead) == 2 else 'B'},G,N]")
    G, N = Bm.shape[-2:]
    _rows(Bm, "Bm", lead + (G, N), dt, dev, 2)
    _rows(Cm, "Cm", lead + (G, N), dt, dev, 2)
    if G < 1 or D % G:
        raise ValueError(f"{G} groups do not divide {D} channels")
    _vector(A, "A", (D, N), dev)
    if A is None:
        raise TypeError("A must be a tensor")
    _vector(D_skip, "D_skip", (D,), dev)
    _vector(dt_bias, "dt_bias", (D,), dev)
    return G, N


def _scan_strides(*tensors):
    out = []
    for t in tensors:
        out += (0, 0) if t is None else t.stride()[:2]
    return out


def ssm_scan_fwd_workspace_size(B, T, D, G=1, N=16, dtype=torch.bfloat16) -> int:
    return int(lib().gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N, _DTYPES[dtype]))


def ssm_scan_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                 D_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                 h0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, h_T: Optional[torch.Tensor] = None, final_state: bool = True,
                 workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan over a prompt (``gdr_ssm_scan_fwd``).

    x, dt and z (output gate, or None) [B,T,D], Bm and Cm [B,T,G,N] in fp32 or bf16, strided;
    A [D,N], D_skip [D], dt_bias [D], h0 [B,D,N] fp32; N in 8, 16, 32, 64; lengths int32 [B].
    Returns (y [B,T,D] in x's type, h_T [B,D,N] fp32 or None); ``h_T`` may be ``h0``.
    """
    ty = _type_of(x)
    dev, host = _device(x), not x.is_cuda
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    B, T, D = x.shape

    def body(handle, x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D_skip=D_skip, z=z, dt_bias=dt_bias, h0=h0, lengths=lengths, y=y,
             h_T=h_T):
        if host:
            x, dt, A, Bm, Cm, D_skip, z, dt_bias, h0, lengths = (
                _to_device(t, dev) for t in (x, dt, A, Bm, Cm, D_skip, z, dt_bias, h0, lengths))
        G, N = _scan_inputs(x, dt, A, Bm, Cm, D_skip, z, dt_bias, (B, T), dev)
        _vector(h0, "h0", (B, D, N), dev)
        _vector(lengths, "lengths", (B,), dev, torch.int32)
        if y is None:
            y = (torch.empty if lengths is None else torch.zeros)(x.shape, dtype=ty, device=dev)
        else:
            _vector(y, "y", x.shape, dev, ty)
        if h_T is not None:
            _vector(h_T, "h_T", (B, D, N), dev)
        elif final_state:
            h_T = torch.empty(B, D, N, dtype=torch.float32, device=dev)
        L = lib()
        size = L.gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N, _DTYPES[ty])
        ws = _workspace(workspace, size, dev)
        _check(L.gdr_ssm_scan_fwd(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D_skip), _ptr(z), _ptr(dt_bias), _ptr(h0),
            _ptr(lengths), _ptr(y), _ptr(h_T), _I64x10(*_scan_strides(x, dt, Bm, Cm, z)), B, T, D, G, N,
            1 if dt_softplus else 0, _DTYPES[ty], _ptr(ws), size, handle), "gdr_ssm_scan_fwd")
        return y, h_T

    out = _scoped(dev, stream, body)
    return tuple(_to_host(t) for t in out) if host else out


def ssm_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                  h: torch.Tensor, D_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                  y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The scan for one token per row (``gdr_ssm_scan_step``); h [B,D,N] fp32 is updated IN PLACE.

    x, dt, z [B,D] and Bm, Cm [B,G,N] (rows may be strided), the rest as ``ssm_scan_fwd``.
    Returns y [B,D].
    """
    ty = _type_of(x)
    dev = x.device
    if not x.is_cuda:
        raise ValueError("ssm_scan_step works on CUDA tensors: the state is updated in place")
    if x.dim() != 2:
        raise ValueError("x must be [B,D]")
    B, D = x.shape
    G, N = _scan_inputs(x, dt, A, Bm, Cm, D_skip, z, dt_bias, (B,), dev)
    if h is None:
        raise TypeError("h must be a tensor")
    _vector(h, "h", (B, D, N), dev)

    def body(handle, y=y):
        if y is None:
            y = torch.empty(B, D, dtype=ty, device=dev)
        else:
            _vector(y, "y", (B, D), dev, ty)
        strides = _I64x5(x.stride(0), dt.stride(0), Bm.stride(0), Cm.stride(0), 0 if z is None else z.stride(0))
        _check(lib().gdr_ssm_scan_step(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D_skip), _ptr(z), _ptr(dt_bias), _ptr(h), _ptr(y),
            strides, B, D, G, N, 1 if dt_softplus else 0, _DTYPES[ty], handle), "gdr_ssm_scan_step")
        return y

    return _scoped(dev, stream, body)


def ssm_scan_bwd_workspace_size(B, T, D, G=1, N=16, dtype=torch.bfloat16) -> int:
    return int(lib().gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N, _DTYPES[dtype]))


def ssm_scan_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                 dy: torch.Tensor, D_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                 h0: Optional[torch.Tensor] = None, dh_T: Optional[torch.Tensor] = None,
                 lengths: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of ``ssm_scan_fwd`` (``gdr_ssm_scan_bwd``): the gradients of <dy, y> + <dh_T, h_T>.

    Inputs as ``ssm_scan_fwd``, dy [B,T,D] in x's type (strided), dh_T [B,D,N] fp32 or None.
    Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0), each in its input's shape and type
    (contiguous) and None where that input is; dx, ddt, dB, dC and dz are zero behind a row's end.
    """
    ty = _type_of(x)
    dev, host = _device(x), not x.is_cuda
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    B, T, D = x.shape

    def body(handle, x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, dy=dy, D_skip=D_skip, z=z, dt_bias=dt_bias, h0=h0, dh_T=dh_T,
             lengths=lengths):
        if host:
            x, dt, A, Bm, Cm, dy, D_skip, z, dt_bias, h0, dh_T, lengths = (
                _to_device(t, dev) for t in (x, dt, A, Bm, Cm, dy, D_skip, z, dt_bias, h0, dh_T, lengths))
        G, N = _scan_inputs(x, dt, A, Bm, Cm, D_skip, z, dt_bias, (B, T), dev)
        _rows(dy, "dy", x.shape, ty, dev)
        _vector(h0, "h0", (B, D, N), dev)
        _vector(dh_T, "dh_T", (B, D, N), dev)
        _vector(lengths, "lengths", (B,), dev, torch.int32)

        def like(t, *shape, dtype=torch.float32):
            return None if t is None else torch.empty(shape, dtype=dtype, device=dev)
        dx, ddt, dz = (like(t, B, T, D, dtype=ty) for t in (x, dt, z))
        dB, dC = (like(t, B, T, G, N, dtype=ty) for t in (Bm, Cm))
        dA, dD, db, dh0 = like(A, D, N), like(D_skip, D), like(dt_bias, D), like(h0, B, D, N)
        L = lib()
        size = L.gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N, _DTYPES[ty])
        ws = _workspace(workspace, size, dev)
        _check(L.gdr_ssm_scan_bwd(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D_skip), _ptr(z), _ptr(dt_bias), _ptr(h0),
            _ptr(lengths), _ptr(dy), _ptr(dh_T), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz),
            _ptr(db), _ptr(dh0), _I64x12(*_scan_strides(x, dt, Bm, Cm, z, dy)), B, T, D, G, N,
            1 if dt_softplus else 0, _DTYPES[ty], _ptr(ws), size, handle), "gdr_ssm_scan_bwd")
        return dx, ddt, dA, dB, dC, dD, dz, db, dh0

    out = _scoped(dev, stream, body)
    return tuple(_to_host(t) for t in out) if host else out

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
* Outputs and workspaces are made on the stream that the call runs on (see the package about `stream`).
* With a host ``x`` the inputs are copied to the current device and the results
  come back as new host tensors; an output that the caller gives has to lie on
  the device (a host one is refused), and the step calls, which update a state
  in place, take device tensors only.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _DTYPES, _check, _record, _stream_on, _to_device, _to_host, lib

_ACTIVATIONS = {None: 0, "silu": 1}
_F32, _I32 = torch.float32, torch.int32
_I64x3 = ctypes.c_longlong * 3
_I64x5 = ctypes.c_longlong * 5
_I64x10 = ctypes.c_longlong * 10
_I64x12 = ctypes.c_longlong * 12

# A decode step takes a few microseconds on the device, so the host's share counts: these two are
# what torch.cuda.current_device() and current_stream() come to, without the objects around them.
# They are looked up by the first call: a build of torch without CUDA does not have them, and can
# still import this package (and build the library).
def _current_device():
    global _current_device
    _current_device = torch._C._cuda_getDevice
    return _current_device()


def _current_stream(index):
    global _current_stream
    _current_stream = torch._C._cuda_getCurrentRawStream
    return _current_stream(index)


def _here(x, stream):
    """x's device if that is the current one and the call runs on its current stream, else None:
    the case in which nothing has to be switched or copied."""
    try:
        index = x.get_device()
    except AttributeError:
        raise TypeError("x must be a tensor") from None
    return index if stream is None and index >= 0 and index == _current_device() else None


def _elsewhere(call, x, stream, *args, outputs=()):
    """call(stream handle, device index, x, *args, *outputs) with the device and the stream current
    that it runs on, so that what it allocates belongs to that stream.  A host x: every tensor of
    `args` is copied to the current device first and the results back afterwards.  `outputs` (name
    and tensor or None) are not copied, as the call would write the copies: they have to lie on the
    device."""
    index = x.get_device()
    host = index < 0
    if host:
        _type_of(x)
        for name, t in outputs:
            if isinstance(t, torch.Tensor) and t.get_device() < 0:
                raise ValueError(f"{name} is a host tensor: a call with host inputs returns its results in new ones")
        index = torch.cuda.current_device()
    dev = torch.device("cuda", index)
    caller = torch.cuda.current_stream(dev)
    given = stream
    stream = caller if stream is None else _stream_on(stream, dev)
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        if host:
            x = _to_device(x, dev)
            args = [_to_device(t, dev) if isinstance(t, torch.Tensor) else t for t in args]
        out = call(stream.cuda_stream, index, x, *args, **dict(outputs))
        if host:
            return tuple(_to_host(t) for t in out)
    if given is not None:
        _record(given, (x, *args, *(t for _, t in outputs)))
        _record(caller, out if isinstance(out, tuple) else (out,))
    return out


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _refuse(t, name, shape, index, dtype):
    """Says what is wrong with a tensor that _dense or _rows did not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dense(t, name, shape, index, dtype=_F32):
    """A contiguous tensor of the given shape."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _refuse(t, name, shape, index, dtype)


def _rows(t, name, shape, index, dtype, dense=1):
    """A tensor of the given shape whose last `dense` dimensions are contiguous."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape:
            if t.is_contiguous() or not t.numel():
                return
            step, strides = 1, t.stride()
            for k in range(1, dense + 1):
                if shape[-k] != 1 and strides[-k] != step:
                    raise ValueError(f"the last dimension{'s' if dense > 1 else ''} of {name} must be contiguous")
                step *= shape[-k]
            return
    except AttributeError:
        pass
    _refuse(t, name, shape, index, dtype)


def _type_of(x):
    if x.dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16")
    return x.dtype


def _new(shape, dtype, index):
    return torch.empty(shape, dtype=dtype, device=index)


def _workspace(ws, size, index):
    if not size:
        return None
    if ws is None or ws.numel() * ws.element_size() < size:
        return torch.empty(size, dtype=torch.uint8, device=index)
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index}")
    return ws


# ------------------------------------------------------------- short convolution

def _conv_shape(x):
    """(B, H, T, d) of [B,H,T,d] or [B,T,D] (one head)."""
    n = x.dim()
    if n == 4:
        return x.shape
    if n == 3:
        B, T, D = x.shape
        return B, 1, T, D
    raise ValueError("x must be [B,H,T,d] or [B,T,D]")


def _conv_strides(x):
    s = x.stride()
    return _I64x3(s[0], s[1], s[2]) if len(s) == 4 else _I64x3(s[0], 0, s[1])


def _conv_params(weight, bias, activation, D, index):
    """Checks weight and bias; returns (taps, the activation's number)."""
    try:
        act = _ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError("activation must be None or 'silu'") from None
    try:
        rows, W = weight.shape
        if rows != D or weight.dtype is not _F32 or weight.get_device() != index or not weight.is_contiguous():
            raise ValueError
    except (AttributeError, ValueError):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise ValueError(f"weight must be a tensor [{D},W]") from None
        _refuse(weight, "weight", (D, weight.shape[1]), index, _F32)
    if bias is not None:
        _dense(bias, "bias", (D,), index)
    return W, act


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
    index = _here(x, stream)
    if index is None:
        return _elsewhere(_conv_fwd, x, stream, weight, bias, state, activation, lengths, final_state,
                          outputs=(("y", y), ("state_out", state_out)))
    return _conv_fwd(_current_stream(index), index, x, weight, bias, state, activation, lengths, final_state, y,
                     state_out)


def _conv_fwd(handle, index, x, weight, bias, state, activation, lengths, final_state, y, state_out):
    dt = _type_of(x)
    B, H, T, d = _conv_shape(x)
    shape, D = x.shape, H * d
    _rows(x, "x", shape, index, dt)
    W, act = _conv_params(weight, bias, activation, D, index)
    if state is not None:
        _dense(state, "state", (B, W - 1, D), index, dt)
    if lengths is not None:
        _dense(lengths, "lengths", (B,), index, _I32)
    zero_tail = y is None
    if zero_tail:
        y = _new(shape, dt, index)
    else:
        _dense(y, "y", shape, index, dt)
    if state_out is not None:
        _dense(state_out, "state_out", (B, W - 1, D), index, dt)
    elif final_state:
        state_out = _new((B, max(W - 1, 0), D), dt, index)
    status = lib().gdr_short_conv_fwd(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths), y.data_ptr(), _ptr(state_out),
        _conv_strides(x), zero_tail, B, H, T, d, W, act, _DTYPES[dt], handle)
    if status:
        _check(status, "gdr_short_conv_fwd")
    return y, state_out


def short_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    activation: Optional[str] = "silu", y: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The convolution for one token per row (``gdr_short_conv_step``).

    x [B,D] (rows may be strided); state [B,W-1,D] in x's type is shifted IN PLACE; weight, bias
    and activation as ``short_conv_fwd``.  Returns y [B,D].
    """
    index = _here(x, stream)
    if index is None:
        if x.get_device() < 0:
            raise ValueError("short_conv_step works on CUDA tensors: the state is updated in place")
        return _elsewhere(_conv_step, x, stream, state, weight, bias, activation, y)
    return _conv_step(_current_stream(index), index, x, state, weight, bias, activation, y)


def _conv_step(handle, index, x, state, weight, bias, activation, y):
    dt, shape = x.dtype, x.shape
    if len(shape) != 2:
        raise ValueError("x must be [B,D]")
    code = _DTYPES.get(dt)
    if code is None:
        _type_of(x)
    B, D = shape
    xs = D
    if not x.is_contiguous():
        _rows(x, "x", shape, index, dt)
        xs = x.stride()[0]
    W, act = _conv_params(weight, bias, activation, D, index)
    _dense(state, "state", (B, W - 1, D), index, dt)
    if y is None:
        y = torch.empty(shape, dtype=dt, device=index)
    else:
        _dense(y, "y", shape, index, dt)
    status = lib().gdr_short_conv_step(x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(),
                                       state.data_ptr(), y.data_ptr(), xs, B, D, W, act, code, handle)
    if status:
        _check(status, "gdr_short_conv_step")
    return y


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
    index = _here(x, stream)
    if index is None:
        return _elsewhere(_conv_bwd, x, stream, weight, dy, bias, state, dstate_out, activation, lengths, workspace)
    return _conv_bwd(_current_stream(index), index, x, weight, dy, bias, state, dstate_out, activation, lengths,
                     workspace)


def _conv_bwd(handle, index, x, weight, dy, bias, state, dstate_out, activation, lengths, workspace):
    dt = _type_of(x)
    B, H, T, d = _conv_shape(x)
    shape, D = x.shape, H * d
    _rows(x, "x", shape, index, dt)
    _rows(dy, "dy", shape, index, dt)
    W, act = _conv_params(weight, bias, activation, D, index)
    if state is not None:
        _dense(state, "state", (B, W - 1, D), index, dt)
    if dstate_out is not None:
        _dense(dstate_out, "dstate_out", (B, W - 1, D), index, dt)
    if lengths is not None:
        _dense(lengths, "lengths", (B,), index, _I32)
    if len(shape) == 4 and x.stride(1) < x.stride(2):
        dx = _new((B, T, H, d), dt, index).transpose(1, 2)
    else:
        dx = _new(shape, dt, index)
    dweight = _new((D, W), _F32, index)
    dbias = None if bias is None else _new((D,), _F32, index)
    dstate = None if state is None else _new((B, W - 1, D), dt, index)
    L = lib()
    size = L.gdr_short_conv_bwd_workspace_size(B, H, T, d, W, _DTYPES[dt])
    ws = _workspace(workspace, size, index)
    status = L.gdr_short_conv_bwd(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths), dy.data_ptr(), _ptr(dstate_out),
        dx.data_ptr(), dweight.data_ptr(), _ptr(dbias), _ptr(dstate), _conv_strides(x), _conv_strides(dy),
        _conv_strides(dx), B, H, T, d, W, act, _DTYPES[dt], _ptr(ws), size, handle)
    if status:
        _check(status, "gdr_short_conv_bwd")
    return dx, dweight, dbias, dstate


# ------------------------------------------------------------ state space scan

def _scan_inputs(index, x, dt, A, Bm, Cm, D_skip, z, dt_bias):
    """Checks what the three scan calls share; returns (G, N)."""
    ty, shape = _type_of(x), x.shape
    if not x.is_contiguous():
        _rows(x, "x", shape, index, ty)
    _rows(dt, "dt", shape, index, ty)
    if z is not None:
        _rows(z, "z", shape, index, ty)
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != len(shape) + 1:
        raise ValueError(f"Bm and Cm must be [{'B,T' if len(shape) == 3 else 'B'},G,N]")
    lead = Bm.shape
    *rows, G, N = lead
    D = shape[-1]
    if tuple(rows) != shape[:-1] or G < 1 or D % G:
        raise ValueError(f"Bm {list(lead)} does not fit x {list(shape)}: [..., G, N] with G dividing {D}")
    _rows(Bm, "Bm", lead, index, ty, 2)
    _rows(Cm, "Cm", lead, index, ty, 2)
    _dense(A, "A", (D, N), index)
    if D_skip is not None:
        _dense(D_skip, "D_skip", (D,), index)
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", (D,), index)
    return G, N


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
    index = _here(x, stream)
    if index is None:
        return _elsewhere(_scan_fwd, x, stream, dt, A, Bm, Cm, D_skip, z, dt_bias, dt_softplus, h0, lengths,
                          final_state, workspace, outputs=(("y", y), ("h_T", h_T)))
    return _scan_fwd(_current_stream(index), index, x, dt, A, Bm, Cm, D_skip, z, dt_bias, dt_softplus, h0, lengths,
                     final_state, workspace, y, h_T)


def _scan_fwd(handle, index, x, dt, A, Bm, Cm, D_skip, z, dt_bias, dt_softplus, h0, lengths, final_state, workspace,
              y, h_T):
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    shape, ty = x.shape, x.dtype
    B, T, D = shape
    G, N = _scan_inputs(index, x, dt, A, Bm, Cm, D_skip, z, dt_bias)
    if h0 is not None:
        _dense(h0, "h0", (B, D, N), index)
    if lengths is not None:
        _dense(lengths, "lengths", (B,), index, _I32)
    zero_tail = y is None
    if zero_tail:
        y = _new(shape, ty, index)
    else:
        _dense(y, "y", shape, index, ty)
    if h_T is not None:
        _dense(h_T, "h_T", (B, D, N), index)
    elif final_state:
        h_T = _new((B, D, N), _F32, index)
    L = lib()
    size = L.gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N, _DTYPES[ty])
    ws = _workspace(workspace, size, index)
    strides = _I64x10(*x.stride()[:2], *dt.stride()[:2], *Bm.stride()[:2], *Cm.stride()[:2],
                      *(z if z is not None else x).stride()[:2])
    status = L.gdr_ssm_scan_fwd(
        x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _ptr(D_skip), _ptr(z), _ptr(dt_bias),
        _ptr(h0), _ptr(lengths), y.data_ptr(), _ptr(h_T), strides, zero_tail, B, T, D, G, N,
        1 if dt_softplus else 0, _DTYPES[ty], _ptr(ws), size, handle)
    if status:
        _check(status, "gdr_ssm_scan_fwd")
    return y, h_T


def ssm_scan_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                  h: torch.Tensor, D_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                  y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The scan for one token per row (``gdr_ssm_scan_step``); h [B,D,N] fp32 is updated IN PLACE.

    x, dt, z [B,D] and Bm, Cm [B,G,N] (rows may be strided), the rest as ``ssm_scan_fwd``.
    Returns y [B,D].
    """
    index = _here(x, stream)
    if index is None:
        if x.get_device() < 0:
            raise ValueError("ssm_scan_step works on CUDA tensors: the state is updated in place")
        return _elsewhere(_scan_step, x, stream, dt, A, Bm, Cm, h, D_skip, z, dt_bias, dt_softplus, y)
    return _scan_step(_current_stream(index), index, x, dt, A, Bm, Cm, h, D_skip, z, dt_bias, dt_softplus, y)


def _scan_step(handle, index, x, dt, A, Bm, Cm, h, D_skip, z, dt_bias, dt_softplus, y):
    if x.dim() != 2:
        raise ValueError("x must be [B,D]")
    shape, ty = x.shape, x.dtype
    B, D = shape
    G, N = _scan_inputs(index, x, dt, A, Bm, Cm, D_skip, z, dt_bias)
    _dense(h, "h", (B, D, N), index)
    if y is None:
        y = torch.empty(shape, dtype=ty, device=index)
    else:
        _dense(y, "y", shape, index, ty)
    strides = _I64x5(x.stride()[0], dt.stride()[0], Bm.stride()[0], Cm.stride()[0],
                     0 if z is None else z.stride()[0])
    status = lib().gdr_ssm_scan_step(
        x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _ptr(D_skip), _ptr(z), _ptr(dt_bias),
        h.data_ptr(), y.data_ptr(), strides, B, D, G, N, 1 if dt_softplus else 0, _DTYPES[ty], handle)
    if status:
        _check(status, "gdr_ssm_scan_step")
    return y


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
    index = _here(x, stream)
    if index is None:
        return _elsewhere(_scan_bwd, x, stream, dt, A, Bm, Cm, dy, D_skip, z, dt_bias, dt_softplus, h0, dh_T, lengths,
                          workspace)
    return _scan_bwd(_current_stream(index), index, x, dt, A, Bm, Cm, dy, D_skip, z, dt_bias, dt_softplus, h0, dh_T,
                     lengths, workspace)


def _scan_bwd(handle, index, x, dt, A, Bm, Cm, dy, D_skip, z, dt_bias, dt_softplus, h0, dh_T, lengths, workspace):
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    shape, ty = x.shape, x.dtype
    B, T, D = shape
    G, N = _scan_inputs(index, x, dt, A, Bm, Cm, D_skip, z, dt_bias)
    _rows(dy, "dy", shape, index, ty)
    if h0 is not None:
        _dense(h0, "h0", (B, D, N), index)
    if dh_T is not None:
        _dense(dh_T, "dh_T", (B, D, N), index)
    if lengths is not None:
        _dense(lengths, "lengths", (B,), index, _I32)
    dx, ddt, dz = _new(shape, ty, index), _new(shape, ty, index), None if z is None else _new(shape, ty, index)
    dB, dC, dA = _new(Bm.shape, ty, index), _new(Bm.shape, ty, index), _new((D, N), _F32, index)
    if D == 0:      # the library has nothing to do: sums over no channels
        dB.zero_()
        dC.zero_()
    dD = None if D_skip is None else _new((D,), _F32, index)
    db = None if dt_bias is None else _new((D,), _F32, index)
    dh0 = None if h0 is None else _new((B, D, N), _F32, index)
    L = lib()
    size = L.gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N, _DTYPES[ty])
    ws = _workspace(workspace, size, index)
    strides = _I64x12(*x.stride()[:2], *dt.stride()[:2], *Bm.stride()[:2], *Cm.stride()[:2],
                      *(z if z is not None else x).stride()[:2], *dy.stride()[:2])
    status = L.gdr_ssm_scan_bwd(
        x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _ptr(D_skip), _ptr(z), _ptr(dt_bias),
        _ptr(h0), _ptr(lengths), dy.data_ptr(), _ptr(dh_T), dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(),
        dB.data_ptr(), dC.data_ptr(), _ptr(dD), _ptr(dz), _ptr(db), _ptr(dh0), strides, B, T, D, G, N,
        1 if dt_softplus else 0, _DTYPES[ty], _ptr(ws), size, handle)
    if status:
        _check(status, "gdr_ssm_scan_bwd")
    return dx, ddt, dA, dB, dC, dD, dz, db, dh0

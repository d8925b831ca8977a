"""The operators around the SSD: conv1d, selective_scan and norm.

Same manner as the rest of the package: ``mamba2_*`` functions keep the C
names and arguments and check every tensor against ``dims`` first; the short
names (``conv1d_forward`` ...) make the dims, allocate outputs and workspace
with torch and call them.  Where ``dims`` has a stride, the tensor may be a
column range of a wider one (the last axis without gaps, equal steps between
tokens); every other tensor is contiguous.

Calls run on the device of their tensors, whichever is current, on that
device's current stream unless ``stream`` is given (a ``torch.cuda.Stream`` or
a raw handle); what a call allocates then belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (MAMBA2_DTYPE_BF16, MAMBA2_DTYPE_F32, MAMBA2_ERR_DTYPE, MAMBA2_ERR_NULL,
               MAMBA2_ERR_SHAPE, MAMBA2_ERR_UNSUPPORTED, Mamba2ConvDims, Mamba2Error,
               Mamba2NormDims, Mamba2ScanDims, _check, _lib, _ptr, _req_bytes, _same_device)

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_ACTIVATIONS = {"none": 0, "silu": 1}
_KINDS = {"rms": 0, "layer": 1}


def _dtype_code(where, name, t):
    if t.dtype is _BF16:
        return MAMBA2_DTYPE_BF16
    if t.dtype is _F32:
        return MAMBA2_DTYPE_F32
    raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"{name} is {t.dtype}, needs float32 or bfloat16")


def _io(dims):
    return _F32 if dims.dtype == MAMBA2_DTYPE_F32 else _BF16


def _stride(where, name, t, lead):
    """Elements between the tokens of ``t``, whose first ``lead`` axes are tokens
    in order; the axes after them have to be without gaps."""
    shape, st = t.shape, t.stride()
    row = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != row:
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name} has gaps inside a token (strides {st})")
        row *= shape[i]
    step, count = 0, 1  # the innermost token axis that has more than one entry sets the step
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if step == 0:
            step = st[i]
        elif st[i] != step * count:
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name}'s tokens are not at equal steps (strides {st})")
        count *= shape[i]
    if count == 1:
        return row
    if step < row:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"{name}'s tokens overlap (strides {st})")
    return step


def _want(where, name, t, shape, dtype, optional=False, stride=None, lead=0):
    """Checks one argument, as ``_req`` does for the SSD's roles; with ``stride``
    the tokens (the first ``lead`` axes) are that many elements apart."""
    if t is None:
        if optional:
            return
        raise Mamba2Error(MAMBA2_ERR_NULL, where, f"{name} is None")
    if isinstance(t, int):
        return
    if not isinstance(t, torch.Tensor):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"{name} is a {type(t).__name__}, not a tensor")
    if t.dtype is not dtype:
        raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"{name} is {t.dtype}, needs {dtype}")
    if t.shape != shape:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"{name} has shape {tuple(t.shape)}, needs {shape}")
    if stride is None:
        if not t.is_contiguous():
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name} is not contiguous (strides {t.stride()})")
        return
    row = 1
    for n in shape[lead:]:
        row *= n
    tokens = 1
    for n in shape[:lead]:
        tokens *= n
    got = _stride(where, name, t, lead)
    if tokens > 1 and got != (stride or row):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"{name}'s tokens are {got} elements apart, dims says {stride or row}")


def _call(where, stream, tensors, *args):
    """The C call on the tensors' device and stream."""
    _same_device(where, *tensors)
    fn = getattr(_lib, where)
    dev = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
    index = torch.cuda.current_device() if dev is None else dev.index
    if stream is None:
        stream = torch.cuda.current_stream(index).cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    _check(status, where)


def _owner(stream, t):
    """Allocations inside belong to ``stream``."""
    if stream is None or not t.is_cuda:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, t.device)
    return torch.cuda.stream(stream)


def _workspace(need, workspace, t):
    """The caller's workspace, or one of ``need`` bytes (where the sizes are refused, need
    is 0 and the C call says why), and its size."""
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=t.device)
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------- conv1d


def make_conv_dims(batch, seqlen, channels, width, parts, dtype, *, activation="silu", x_stride=0,
                   dx_stride=0) -> Mamba2ConvDims:
    """dtype: torch.float32 / torch.bfloat16; parts: the outputs' channels (None: one output)."""
    parts = (channels,) if parts is None else tuple(parts)
    if not 1 <= len(parts) <= 3:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, "make_conv_dims", f"{len(parts)} parts: 1 to 3 are possible")
    if activation not in _ACTIVATIONS:
        raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, "make_conv_dims", f"unknown activation {activation!r}")
    code = MAMBA2_DTYPE_BF16 if dtype is _BF16 else MAMBA2_DTYPE_F32 if dtype is _F32 else int(dtype)
    d = Mamba2ConvDims(batch, seqlen, channels, width)
    for i, p in enumerate(parts):
        d.part[i] = p
    d.x_stride, d.dx_stride, d.dtype, d.activation = x_stride, dx_stride, code, _ACTIVATIONS[activation]
    return d


def mamba2_conv1d_backward_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_conv1d_backward_workspace_bytes(ctypes.byref(dims)))


def _conv_args(w, dims, x, weight, bias, states, ys, names, step=False):
    b, L, C, W, io = dims.batch, dims.seqlen, dims.channels, dims.width, _io(dims)
    lead = (b,) if step else (b, L)
    _want(w, "x", x, lead + (C,), io, stride=dims.x_stride, lead=len(lead))
    _want(w, "weight", weight, (C, W), _F32)
    _want(w, "bias", bias, (C,), _F32, optional=True)
    for name, t in states:
        _want(w, name, t, (b, W - 1, C), io, optional=name != "state")
    for i, (name, y) in enumerate(zip(names, ys)):
        if dims.part[i]:
            _want(w, name, y, lead + (dims.part[i],), io)


def mamba2_conv1d_forward(dims, x, weight, bias, init_state, lengths, y0, y1, y2, final_state,
                          stream=None):
    w = "mamba2_conv1d_forward"
    _conv_args(w, dims, x, weight, bias,
               (("init_state", init_state), ("final_state", final_state)), (y0, y1, y2),
               ("y0", "y1", "y2"))
    _want(w, "lengths", lengths, (dims.batch,), _I32, optional=True)
    _call(w, stream, (x, weight, bias, init_state, lengths, y0, y1, y2, final_state),
          ctypes.byref(dims), _ptr(x), _ptr(weight), _ptr(bias), _ptr(init_state), _ptr(lengths),
          _ptr(y0), _ptr(y1), _ptr(y2), _ptr(final_state))


def mamba2_conv1d_backward(dims, x, weight, bias, init_state, lengths, dy0, dy1, dy2, dfinal, dx,
                           dweight, dbias, dinit, workspace, workspace_bytes, stream=None):
    w = "mamba2_conv1d_backward"
    _conv_args(w, dims, x, weight, bias,
               (("init_state", init_state), ("dfinal", dfinal), ("dinit", dinit)),
               (dy0, dy1, dy2), ("dy0", "dy1", "dy2"))
    _want(w, "lengths", lengths, (dims.batch,), _I32, optional=True)
    _want(w, "dx", dx, (dims.batch, dims.seqlen, dims.channels), _io(dims), stride=dims.dx_stride,
          lead=2)
    _want(w, "dweight", dweight, (dims.channels, dims.width), _F32)
    _want(w, "dbias", dbias, (dims.channels,), _F32, optional=True)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (x, weight, bias, init_state, lengths, dy0, dy1, dy2, dfinal, dx, dweight,
                      dbias, dinit, workspace),
          ctypes.byref(dims), _ptr(x), _ptr(weight), _ptr(bias), _ptr(init_state), _ptr(lengths),
          _ptr(dy0), _ptr(dy1), _ptr(dy2), _ptr(dfinal), _ptr(dx), _ptr(dweight), _ptr(dbias),
          _ptr(dinit), _ptr(workspace), int(workspace_bytes))


def mamba2_conv1d_step(dims, x, weight, bias, state, y0, y1, y2, stream=None):
    w = "mamba2_conv1d_step"
    _conv_args(w, dims, x, weight, bias, (("state", state),), (y0, y1, y2), ("y0", "y1", "y2"),
               step=True)
    _call(w, stream, (x, weight, bias, state, y0, y1, y2), ctypes.byref(dims), _ptr(x),
          _ptr(weight), _ptr(bias), _ptr(state), _ptr(y0), _ptr(y1), _ptr(y2))


def _conv_dims(where, x, weight, parts, activation, step=False):
    lead = 1 if step else 2
    if x.dim() != lead + 1 or weight.dim() != 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"x {tuple(x.shape)} must be {lead + 1}-d and weight "
                          f"{tuple(weight.shape)} 2-d")
    _dtype_code(where, "x", x)
    if parts is not None and sum(parts) != x.shape[-1]:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"parts {tuple(parts)} do not add up to x's {x.shape[-1]} channels")
    return make_conv_dims(x.shape[0], 1 if step else x.shape[1], x.shape[-1], weight.shape[1],
                          parts, x.dtype, activation=activation,
                          x_stride=_stride(where, "x", x, lead))


def conv1d_forward(x, weight, bias=None, init_state=None, *, parts=None, activation="silu",
                   lengths=None, stream=None):
    """The causal depthwise convolution of x[B,L,C] (a column range of wider rows is
    taken as it is) with weight[C,W], W = 2, 3 or 4.  ``parts``: up to three channel
    counts that add up to C; the output then comes as that many contiguous tensors,
    e.g. (H*P, G*N, G*N) for the x, B and C of an SSD call.  ``activation``: "silu"
    or "none".  Returns (y or tuple of parts, final_state[B,W-1,C])."""
    where = "conv1d_forward"
    dims = _conv_dims(where, x, weight, parts, activation)
    b, L, C = x.shape
    with _owner(stream, x):
        ys = [torch.empty((b, L, p), dtype=x.dtype, device=x.device)
              for p in ((C,) if parts is None else parts)]
        final = torch.empty((b, dims.width - 1, C), dtype=x.dtype, device=x.device)
    mamba2_conv1d_forward(dims, x, weight, bias, init_state, lengths,
                          *(ys + [None] * (3 - len(ys))), final, stream)
    return (ys[0] if parts is None else tuple(ys)), final


def conv1d_backward(x, weight, bias, init_state, dys, dfinal=None, *, activation="silu",
                    lengths=None, workspace=None, stream=None):
    """Gradients of conv1d_forward: ``dys`` is the gradient of y, or a tuple of the
    parts' gradients.  Returns a dict with dx, dweight, dbias (None without bias)
    and dinit."""
    where = "conv1d_backward"
    dys = (dys,) if isinstance(dys, torch.Tensor) else tuple(dys)
    dims = _conv_dims(where, x, weight, tuple(d.shape[-1] for d in dys), activation)
    with _owner(stream, x):
        workspace, n = _workspace(mamba2_conv1d_backward_workspace_bytes(dims), workspace, x)
        g = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device),
             "dweight": torch.empty_like(weight),
             "dbias": None if bias is None else torch.empty_like(bias),
             "dinit": torch.empty((x.shape[0], dims.width - 1, x.shape[2]), dtype=x.dtype,
                                  device=x.device)}
    mamba2_conv1d_backward(dims, x, weight, bias, init_state, lengths,
                           *(dys + (None,) * (3 - len(dys))), dfinal, g["dx"], g["dweight"],
                           g["dbias"], g["dinit"], workspace, n, stream)
    return g


def conv1d_step(x, weight, bias, state, *, parts=None, activation="silu", stream=None):
    """One token of every sequence: x[B,C], ``state``[B,W-1,C] moved on in place.
    Returns y[B,C] or the tuple of its parts."""
    where = "conv1d_step"
    dims = _conv_dims(where, x, weight, parts, activation, step=True)
    with _owner(stream, x):
        ys = [torch.empty((x.shape[0], p), dtype=x.dtype, device=x.device)
              for p in ((x.shape[1],) if parts is None else parts)]
    mamba2_conv1d_step(dims, x, weight, bias, state, *(ys + [None] * (3 - len(ys))), stream)
    return ys[0] if parts is None else tuple(ys)


# --------------------------------------------------------------- selective scan


def make_scan_dims(batch, seqlen, channels, dstate, ngroups, dtype, *, softplus=True, z_stride=0,
                   b_stride=0, c_stride=0, dz_stride=0) -> Mamba2ScanDims:
    code = MAMBA2_DTYPE_BF16 if dtype is _BF16 else MAMBA2_DTYPE_F32 if dtype is _F32 else int(dtype)
    return Mamba2ScanDims(batch, seqlen, channels, dstate, ngroups, z_stride, b_stride, c_stride,
                          dz_stride, code, int(softplus))


def mamba2_selective_scan_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_selective_scan_workspace_bytes(ctypes.byref(dims)))


def _scan_args(w, dims, u, dt, A, B, C, D, z, dt_bias, step=False):
    b, L, ch, n, g, io = (dims.batch, dims.seqlen, dims.channels, dims.dstate, dims.ngroups,
                          _io(dims))
    lead = (b,) if step else (b, L)
    k = len(lead)
    _want(w, "u", u, lead + (ch,), io)
    _want(w, "dt", dt, lead + (ch,), io)
    _want(w, "A", A, (ch, n), _F32)
    _want(w, "B", B, lead + (g, n), io, stride=dims.b_stride, lead=k)
    _want(w, "C", C, lead + (g, n), io, stride=dims.c_stride, lead=k)
    _want(w, "D", D, (ch,), _F32, optional=True)
    _want(w, "z", z, lead + (ch,), io, optional=True, stride=dims.z_stride, lead=k)
    _want(w, "dt_bias", dt_bias, (ch,), _F32, optional=True)


def mamba2_selective_scan_forward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, y,
                                  final_state, workspace, workspace_bytes, stream=None):
    w = "mamba2_selective_scan_forward"
    _scan_args(w, dims, u, dt, A, B, C, D, z, dt_bias)
    state = (dims.batch, dims.channels, dims.dstate)
    _want(w, "init_state", init_state, state, _F32, optional=True)
    _want(w, "lengths", lengths, (dims.batch,), _I32, optional=True)
    _want(w, "y", y, (dims.batch, dims.seqlen, dims.channels), _io(dims))
    _want(w, "final_state", final_state, state, _F32, optional=True)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (u, dt, A, B, C, D, z, dt_bias, init_state, lengths, y, final_state, workspace),
          ctypes.byref(dims), _ptr(u), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
          _ptr(dt_bias), _ptr(init_state), _ptr(lengths), _ptr(y), _ptr(final_state),
          _ptr(workspace), int(workspace_bytes))


def mamba2_selective_scan_backward_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_selective_scan_backward_workspace_bytes(ctypes.byref(dims)))


def mamba2_selective_scan_backward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, dy,
                                   dfinal, du, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit, workspace,
                                   workspace_bytes, stream=None):
    w = "mamba2_selective_scan_backward"
    _scan_args(w, dims, u, dt, A, B, C, D, z, dt_bias)
    io, full = _io(dims), (dims.batch, dims.seqlen, dims.channels)
    state, ch = (dims.batch, dims.channels, dims.dstate), (dims.channels,)
    bc = (dims.batch, dims.seqlen, dims.ngroups, dims.dstate)
    for name, t in (("init_state", init_state), ("dfinal", dfinal), ("dinit", dinit)):
        _want(w, name, t, state, _F32, optional=True)
    _want(w, "lengths", lengths, (dims.batch,), _I32, optional=True)
    for name, t in (("dy", dy), ("du", du), ("ddt", ddt)):
        _want(w, name, t, full, io)
    _want(w, "dA", dA, (dims.channels, dims.dstate), _F32)
    _want(w, "dB", dB, bc, io)
    _want(w, "dC", dC, bc, io)
    _want(w, "dD", dD, ch, _F32, optional=True)
    _want(w, "dz", dz, full, io, optional=z is None, stride=dims.dz_stride, lead=2)
    _want(w, "ddt_bias", ddt_bias, ch, _F32, optional=True)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (u, dt, A, B, C, D, z, dt_bias, init_state, lengths, dy, dfinal, du, ddt, dA,
                      dB, dC, dD, dz, ddt_bias, dinit, workspace),
          ctypes.byref(dims), _ptr(u), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
          _ptr(dt_bias), _ptr(init_state), _ptr(lengths), _ptr(dy), _ptr(dfinal), _ptr(du),
          _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz), _ptr(ddt_bias),
          _ptr(dinit), _ptr(workspace), int(workspace_bytes))


def mamba2_selective_scan_step(dims, u, dt, A, B, C, D, z, dt_bias, state, y, stream=None):
    w = "mamba2_selective_scan_step"
    _scan_args(w, dims, u, dt, A, B, C, D, z, dt_bias, step=True)
    _want(w, "state", state, (dims.batch, dims.channels, dims.dstate), _F32)
    _want(w, "y", y, (dims.batch, dims.channels), _io(dims))
    _call(w, stream, (u, dt, A, B, C, D, z, dt_bias, state, y), ctypes.byref(dims), _ptr(u),
          _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(state),
          _ptr(y))


def _scan_dims(where, u, A, B, C, z, softplus, step=False):
    lead = 1 if step else 2
    if u.dim() != lead + 1 or B.dim() != lead + 2 or C.dim() != lead + 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"u {tuple(u.shape)} must be {lead + 1}-d, B {tuple(B.shape)} and C "
                          f"{tuple(C.shape)} {lead + 2}-d")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise Mamba2Error(MAMBA2_ERR_NULL if A is None else MAMBA2_ERR_SHAPE, where,
                          "A must be a tensor [D, N]")
    _dtype_code(where, "u", u)
    return make_scan_dims(u.shape[0], 1 if step else u.shape[1], u.shape[-1], A.shape[1],
                          B.shape[-2], u.dtype, softplus=softplus,
                          z_stride=0 if z is None else _stride(where, "z", z, lead),
                          b_stride=_stride(where, "B", B, lead),
                          c_stride=_stride(where, "C", C, lead))


def selective_scan_forward(u, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *,
                           softplus=True, lengths=None, workspace=None, stream=None):
    """The selective scan of u[B,L,D] with time steps softplus(dt + dt_bias) (dt + dt_bias
    with softplus=False), decays A[D,N], B and C [B,L,G,N], skip D[D] and gate z[B,L,D]
    (z, B and C may be column ranges of wider rows).  Returns (y[B,L,D],
    final_state[B,D,N])."""
    where = "selective_scan_forward"
    dims = _scan_dims(where, u, A, B, C, z, softplus)
    with _owner(stream, u):
        workspace, n = _workspace(mamba2_selective_scan_workspace_bytes(dims), workspace, u)
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        final = torch.empty((dims.batch, dims.channels, dims.dstate), dtype=_F32, device=u.device)
    mamba2_selective_scan_forward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, y,
                                  final, workspace, n, stream)
    return y, final


def selective_scan_backward(u, dt, A, B, C, D, z, dt_bias, init_state, dy, dfinal=None, *,
                            softplus=True, lengths=None, workspace=None, stream=None):
    """Gradients of selective_scan_forward: a dict with du, ddt, dA, dB, dC, dD (None
    without D), dz (None without z), ddt_bias (None without dt_bias) and dinit."""
    where = "selective_scan_backward"
    dims = _scan_dims(where, u, A, B, C, z, softplus)
    dev = u.device
    with _owner(stream, u):
        workspace, n = _workspace(mamba2_selective_scan_backward_workspace_bytes(dims), workspace,
                                  u)
        g = {"du": torch.empty(u.shape, dtype=u.dtype, device=dev),
             "ddt": torch.empty(u.shape, dtype=u.dtype, device=dev),
             "dA": torch.empty_like(A),
             "dB": torch.empty(B.shape, dtype=u.dtype, device=dev),
             "dC": torch.empty(C.shape, dtype=u.dtype, device=dev),
             "dD": None if D is None else torch.empty_like(D),
             "dz": None if z is None else torch.empty(u.shape, dtype=u.dtype, device=dev),
             "ddt_bias": None if dt_bias is None else torch.empty_like(dt_bias),
             "dinit": torch.empty((dims.batch, dims.channels, dims.dstate), dtype=_F32,
                                  device=dev)}
    mamba2_selective_scan_backward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, dy,
                                   dfinal, g["du"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"],
                                   g["dz"], g["ddt_bias"], g["dinit"], workspace, n, stream)
    return g


def selective_scan_step(u, dt, A, B, C, D, z, dt_bias, state, *, softplus=True, stream=None):
    """One token of every sequence: u, dt, z [B,D], B, C [B,G,N]; ``state``[B,D,N] is
    updated in place.  Returns y[B,D]."""
    where = "selective_scan_step"
    dims = _scan_dims(where, u, A, B, C, z, softplus, step=True)
    with _owner(stream, u):
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    mamba2_selective_scan_step(dims, u, dt, A, B, C, D, z, dt_bias, state, y, stream)
    return y


# ------------------------------------------------------------------------ norm


def make_norm_dims(rows, channels, ngroups, dtype, *, kind="rms", eps=1e-5, x_stride=0, z_stride=0,
                   dz_stride=0) -> Mamba2NormDims:
    if kind not in _KINDS:
        raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, "make_norm_dims", f"unknown norm {kind!r}")
    code = MAMBA2_DTYPE_BF16 if dtype is _BF16 else MAMBA2_DTYPE_F32 if dtype is _F32 else int(dtype)
    return Mamba2NormDims(rows, channels, ngroups, x_stride, z_stride, dz_stride, eps, _KINDS[kind],
                          code, 0)


def mamba2_norm_backward_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_norm_backward_workspace_bytes(ctypes.byref(dims)))


def _norm_args(w, dims, x, z, weight):
    _want(w, "x", x, (dims.rows, dims.channels), _io(dims), stride=dims.x_stride, lead=1)
    _want(w, "z", z, (dims.rows, dims.channels), _io(dims), optional=True, stride=dims.z_stride,
          lead=1)
    _want(w, "weight", weight, (dims.channels,), _F32)


def mamba2_norm_forward(dims, x, z, weight, bias, y, stream=None):
    w = "mamba2_norm_forward"
    _norm_args(w, dims, x, z, weight)
    _want(w, "bias", bias, (dims.channels,), _F32, optional=True)
    _want(w, "y", y, (dims.rows, dims.channels), _io(dims))
    _call(w, stream, (x, z, weight, bias, y), ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(weight),
          _ptr(bias), _ptr(y))


def mamba2_norm_backward(dims, x, z, weight, dy, dx, dz, dweight, dbias, workspace,
                         workspace_bytes, stream=None):
    w = "mamba2_norm_backward"
    _norm_args(w, dims, x, z, weight)
    full, io = (dims.rows, dims.channels), _io(dims)
    _want(w, "dy", dy, full, io)
    _want(w, "dx", dx, full, io)
    _want(w, "dz", dz, full, io, optional=z is None, stride=dims.dz_stride, lead=1)
    _want(w, "dweight", dweight, (dims.channels,), _F32)
    _want(w, "dbias", dbias, (dims.channels,), _F32, optional=True)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (x, z, weight, dy, dx, dz, dweight, dbias, workspace), ctypes.byref(dims),
          _ptr(x), _ptr(z), _ptr(weight), _ptr(dy), _ptr(dx), _ptr(dz), _ptr(dweight),
          _ptr(dbias), _ptr(workspace), int(workspace_bytes))


def _norm_dims(where, x, z, ngroups, kind, eps):
    """Dims, and x and z as rows (views: leading axes that are tokens in order)."""
    if x.dim() < 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"x {tuple(x.shape)} must be at least 2-d")
    _dtype_code(where, "x", x)
    if z is not None and z.shape != x.shape:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"z has shape {tuple(z.shape)}, needs {tuple(x.shape)}")
    lead = x.dim() - 1
    dims = make_norm_dims(x.numel() // max(1, x.shape[-1]), x.shape[-1], ngroups, x.dtype,
                          kind=kind, eps=eps, x_stride=_stride(where, "x", x, lead),
                          z_stride=0 if z is None else _stride(where, "z", z, lead))
    if x.dim() > 2:
        x = x.view(dims.rows, dims.channels)
        z = None if z is None else z.view(dims.rows, dims.channels)
    return dims, x, z


def norm_forward(x, weight, bias=None, z=None, *, ngroups=1, kind="rms", eps=1e-5, stream=None):
    """RMS norm (kind="rms") or layer norm ("layer") of x, or of x * silu(z), over
    ``ngroups`` groups of the last axis; weight and bias [D] float32.  Returns y."""
    shape = x.shape
    dims, x, z = _norm_dims("norm_forward", x, z, ngroups, kind, eps)
    with _owner(stream, x):
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
    mamba2_norm_forward(dims, x, z, weight, bias, y.view(dims.rows, dims.channels), stream)
    return y


def norm_backward(x, weight, bias, z, dy, *, ngroups=1, kind="rms", eps=1e-5, workspace=None,
                  stream=None):
    """Gradients of norm_forward: a dict with dx, dweight, dbias (None without bias)
    and dz (None without z)."""
    where = "norm_backward"
    shape = x.shape
    dims, x, z = _norm_dims(where, x, z, ngroups, kind, eps)
    if dy.shape != shape or not dy.is_contiguous():
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"dy {tuple(dy.shape)} must be contiguous and of x's shape {tuple(shape)}")
    rows = (dims.rows, dims.channels)
    with _owner(stream, x):
        workspace, n = _workspace(mamba2_norm_backward_workspace_bytes(dims), workspace, x)
        g = {"dx": torch.empty(shape, dtype=x.dtype, device=x.device),
             "dweight": torch.empty_like(weight),
             "dbias": None if bias is None else torch.empty_like(bias),
             "dz": None if z is None else torch.empty(shape, dtype=x.dtype, device=x.device)}
    mamba2_norm_backward(dims, x, z, weight, dy.view(rows), g["dx"].view(rows),
                         None if z is None else g["dz"].view(rows), g["dweight"], g["dbias"],
                         workspace, n, stream)
    return g

"""The operators around the SSD: conv1d, selective_scan and norm.

Same manner as the rest of the package: ``mamba2_*`` functions keep the C
names and arguments and check every tensor against ``dims`` first; the short
names (``conv1d_forward`` ...) make the dims, allocate outputs and workspace
with torch and call them.  Where ``dims`` has a stride, the tensor may be a
column range of a wider one (the last axis without gaps, equal steps between
tokens); every other tensor is contiguous.  A tensor broadcast over tokens or
sequences (``expand``) is refused: its rows have to be there (``contiguous``).

Calls run on the device of their tensors, whichever is current, on that
device's current stream unless ``stream`` is given (a ``torch.cuda.Stream`` or
a raw handle); what a call allocates then belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import (MAMBA2_DTYPE_BF16, MAMBA2_DTYPE_F32, MAMBA2_ERR_DTYPE, MAMBA2_ERR_NULL,
               MAMBA2_ERR_SHAPE, MAMBA2_ERR_UNSUPPORTED, MAMBA2_ERR_WORKSPACE, Mamba2ConvDims,
               Mamba2Error, Mamba2NormDims, Mamba2ScanDims, _check, _lib, _ptr, _req_bytes,
               _same_device)

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_Tensor = torch.Tensor
_ACTIVATIONS = {"none": 0, "silu": 1}
_KINDS = {"rms": 0, "layer": 1}


def _known(name, names):
    return isinstance(name, str) and name in names


def _io(dims):
    return _F32 if dims.dtype == MAMBA2_DTYPE_F32 else _BF16


def _stride(where, name, shape, st, lead):
    """Elements between the tokens of a tensor of this shape and strides, whose first
    ``lead`` axes are tokens in order; the axes after them have to be without gaps."""
    row = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != row:
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name} has gaps inside a token (strides {st})")
        row *= shape[i]
    # the innermost token axis with more than one entry sets the step; a step of 0 is one too
    # (a row for all tokens, which the kernels would read past)
    step, count = None, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if step is None:
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
    got = _stride(where, name, t.shape, t.stride(), lead)
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


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _launch(fn, where, index, stream, *args):
    """The C call for tensors that are known to be right, on device ``index``."""
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _raw_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status:
        raise Mamba2Error(status, where)


def _plain(t, dtype, shape, index):
    """Whether t is a contiguous tensor of this type and shape on device ``index``.  The
    short functions ask this first and launch at once where it holds for all inputs; else
    the mamba2_* function looks closer and says what is wrong."""
    try:
        return (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == index)
    except AttributeError:
        return False


def _tensors(where, **tensors):
    """Raises the error for what is no tensor among what a short function looks into before
    the call."""
    for name, t in tensors.items():
        if t is None:
            raise Mamba2Error(MAMBA2_ERR_NULL, where, f"{name} is None")
        if not isinstance(t, _Tensor):
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name} is a {type(t).__name__}, not a tensor")


def _given(where, **tensors):
    """The same for optional tensors, in the branch that hands on to a mamba2_* function: those
    take whole numbers as addresses, the short functions do not."""
    _tensors(where, **{name: t for name, t in tensors.items() if t is not None})


def _like(t):
    """The gradient's tensor of an optional input (the call refuses what is no tensor)."""
    return torch.empty_like(t) if isinstance(t, _Tensor) else None


_CURRENT = contextlib.nullcontext()


def _owner(stream, t):
    """Allocations inside belong to ``stream``."""
    if stream is None or not t.is_cuda:
        return _CURRENT
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, t.device) if stream
                  else torch.cuda.default_stream(t.device))
    return torch.cuda.stream(stream)


def _workspace(where, need, workspace, t):
    """The caller's workspace, or one of ``need`` bytes (where the sizes are refused, need
    is 0 and the C call says why), and its size."""
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=t.device)
    elif not isinstance(workspace, _Tensor):
        raise Mamba2Error(MAMBA2_ERR_WORKSPACE, where,
                          f"workspace is a {type(workspace).__name__}, not a tensor")
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------- conv1d


def make_conv_dims(batch, seqlen, channels, width, parts, dtype, *, activation="silu", x_stride=0,
                   dx_stride=0) -> Mamba2ConvDims:
    """dtype: torch.float32 / torch.bfloat16; parts: the outputs' channels (None: one output)."""
    parts = (channels,) if parts is None else tuple(parts)
    if not 1 <= len(parts) <= 3:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, "make_conv_dims", f"{len(parts)} parts: 1 to 3 are possible")
    if not _known(activation, _ACTIVATIONS):
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


@functools.lru_cache(maxsize=256)
def _conv_plan(where, shape, strides, wshape, parts, activation, dtype, step):
    """dims, the states' shape and the outputs' shapes of a call with these sizes."""
    lead = 1 if step else 2
    if len(shape) != lead + 1 or len(wshape) != 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"x {tuple(shape)} must be {lead + 1}-d and weight {tuple(wshape)} 2-d")
    if dtype is not _F32 and dtype is not _BF16:
        raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"x is {dtype}, needs float32 or bfloat16")
    C = shape[-1]
    if parts is not None and sum(parts) != C:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"parts {parts} do not add up to x's {C} channels")
    dims = make_conv_dims(shape[0], 1 if step else shape[1], C, wshape[1], parts, dtype,
                          activation=activation, x_stride=_stride(where, "x", shape, strides, lead))
    return (dims, ctypes.byref(dims), torch.Size((shape[0], wshape[1] - 1, C)),
            [torch.Size(tuple(shape[:-1]) + (p,)) for p in (parts or (C,))],
            torch.Size((C, wshape[1])), torch.Size((C,)),
            mamba2_conv1d_backward_workspace_bytes(dims))


def _conv_plan_of(where, x, weight, parts, activation, step=False):
    try:
        if parts is not None and type(parts) is not tuple:
            parts = tuple(parts)
        return _conv_plan(where, x.shape, x.stride(), weight.shape, parts, activation, x.dtype,
                          step)
    except (AttributeError, TypeError, Mamba2Error) as e:  # what is of another kind, if anything
        _tensors(where, x=x, weight=weight)
        if isinstance(e, Mamba2Error):
            raise
        if not _known(activation, _ACTIVATIONS):
            raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, where,
                              f"unknown activation {activation!r}") from None
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"parts is {parts!r}, not up to three channel counts") from None


def _optional(t, dtype, shape, index):
    return t is None or _plain(t, dtype, shape, index)


def conv1d_forward(x, weight, bias=None, init_state=None, *, parts=None, activation="silu",
                   lengths=None, stream=None):
    """The causal depthwise convolution of x[B,L,C] (a column range of wider rows is
    taken as it is) with weight[C,W], W = 2, 3 or 4.  ``parts``: up to three channel
    counts that add up to C; the output then comes as that many contiguous tensors,
    e.g. (H*P, G*N, G*N) for the x, B and C of an SSD call.  ``activation``: "silu"
    or "none".  Returns (y or tuple of parts, final_state[B,W-1,C])."""
    dims, ref, state, shapes, wshape, bshape, _ = _conv_plan_of(
        "conv1d_forward", x, weight, parts, activation)
    with _owner(stream, x):
        ys = [x.new_empty(p) for p in shapes]
        final = x.new_empty(state)
    out = ys + [None] * (3 - len(ys))
    i = x.get_device()
    if (i >= 0 and _plain(weight, _F32, wshape, i) and _optional(bias, _F32, bshape, i)
            and _optional(init_state, x.dtype, state, i)
            and _optional(lengths, _I32, x.shape[:1], i)):
        _launch(_lib.mamba2_conv1d_forward, "conv1d_forward", i, stream, ref, x.data_ptr(),
                weight.data_ptr(), _ptr(bias), _ptr(init_state), _ptr(lengths), *map(_ptr, out),
                final.data_ptr())
    else:
        _given("conv1d_forward", weight=weight, bias=bias, init_state=init_state, lengths=lengths)
        mamba2_conv1d_forward(dims, x, weight, bias, init_state, lengths, *out, final, stream)
    return (ys[0] if parts is None else tuple(ys)), final


def conv1d_backward(x, weight, bias, init_state, dys, dfinal=None, *, activation="silu",
                    lengths=None, workspace=None, stream=None):
    """Gradients of conv1d_forward: ``dys`` is the gradient of y, or a tuple of the
    parts' gradients.  Returns a dict with dx, dweight, dbias (None without bias)
    and dinit."""
    try:
        dys = (dys,) if isinstance(dys, _Tensor) else tuple(dys)
        widths = tuple([d.size(-1) for d in dys])
    except (AttributeError, IndexError, TypeError):
        dys = dys if isinstance(dys, tuple) else (dys,)
        _tensors("conv1d_backward", **{f"dy{i}": d for i, d in enumerate(dys)})
        raise Mamba2Error(MAMBA2_ERR_SHAPE, "conv1d_backward", "a dy has no channels") from None
    dims, ref, state, shapes, wshape, bshape, need = _conv_plan_of(
        "conv1d_backward", x, weight, widths, activation)
    with _owner(stream, x):
        workspace, n = _workspace("conv1d_backward", need, workspace, x)
        g = {"dx": x.new_empty(x.shape), "dweight": _like(weight), "dbias": _like(bias),
             "dinit": x.new_empty(state)}
    dy3 = dys + (None,) * (3 - len(dys))
    i = x.get_device()
    if (i >= 0 and n >= need > 0 and _plain(weight, _F32, wshape, i)
            and _optional(bias, _F32, bshape, i) and _optional(init_state, x.dtype, state, i)
            and _optional(dfinal, x.dtype, state, i) and _optional(lengths, _I32, x.shape[:1], i)
            and all(_plain(d, x.dtype, p, i) for d, p in zip(dys, shapes))
            and workspace.is_contiguous() and workspace.get_device() == i):
        _launch(_lib.mamba2_conv1d_backward, "conv1d_backward", i, stream, ref, x.data_ptr(),
                weight.data_ptr(), _ptr(bias), _ptr(init_state), _ptr(lengths), *map(_ptr, dy3),
                _ptr(dfinal), g["dx"].data_ptr(), g["dweight"].data_ptr(), _ptr(g["dbias"]),
                g["dinit"].data_ptr(), workspace.data_ptr(), n)
    else:
        _given("conv1d_backward", weight=weight, bias=bias, init_state=init_state, dfinal=dfinal,
               lengths=lengths)
        mamba2_conv1d_backward(dims, x, weight, bias, init_state, lengths, *dy3, dfinal, g["dx"],
                               g["dweight"], g["dbias"], g["dinit"], workspace, n, stream)
    return g


def conv1d_step(x, weight, bias, state, *, parts=None, activation="silu", stream=None):
    """One token of every sequence: x[B,C], ``state``[B,W-1,C] moved on in place.
    Returns y[B,C] or the tuple of its parts."""
    dims, ref, sshape, shapes, wshape, bshape, _ = _conv_plan_of(
        "conv1d_step", x, weight, parts, activation, True)
    with _owner(stream, x):
        ys = [x.new_empty(p) for p in shapes]
    out = ys + [None] * (3 - len(ys))
    i = x.get_device()
    if (i >= 0 and _plain(state, x.dtype, sshape, i)
            and _plain(weight, _F32, wshape, i) and _optional(bias, _F32, bshape, i)):
        _launch(_lib.mamba2_conv1d_step, "conv1d_step", i, stream, ref, x.data_ptr(),
                weight.data_ptr(), _ptr(bias), state.data_ptr(), *map(_ptr, out))
    else:
        _given("conv1d_step", weight=weight, bias=bias, state=state)
        mamba2_conv1d_step(dims, x, weight, bias, state, *out, stream)
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


@functools.lru_cache(maxsize=256)
def _scan_plan(where, shape, ashape, bshape, bstrides, cshape, cstrides, zstrides, dtype, softplus,
               step):
    """dims, the states' shape and the workspaces of a call with these sizes."""
    lead = 1 if step else 2
    if len(shape) != lead + 1 or len(bshape) != lead + 2 or len(cshape) != lead + 2 or \
            len(ashape) != 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"u {tuple(shape)} must be {lead + 1}-d, A {tuple(ashape)} 2-d, B "
                          f"{tuple(bshape)} and C {tuple(cshape)} {lead + 2}-d")
    if dtype is not _F32 and dtype is not _BF16:
        raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"u is {dtype}, needs float32 or bfloat16")
    if zstrides is not None and len(zstrides) != len(shape):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"z is {len(zstrides)}-d, u {len(shape)}-d")
    ch, n, g = shape[-1], ashape[1], bshape[-2]
    dims = make_scan_dims(
        shape[0], 1 if step else shape[1], ch, n, g, dtype, softplus=softplus,
        z_stride=0 if zstrides is None else _stride(where, "z", shape, zstrides, lead),
        b_stride=_stride(where, "B", bshape, bstrides, lead),
        c_stride=_stride(where, "C", cshape, cstrides, lead))
    return (dims, ctypes.byref(dims), torch.Size((shape[0], ch, n)), torch.Size((ch, n)),
            torch.Size((ch,)), torch.Size(tuple(shape[:-1]) + (g, n)),
            mamba2_selective_scan_workspace_bytes(dims),
            mamba2_selective_scan_backward_workspace_bytes(dims))


def _scan_plan_of(where, u, A, B, C, z, softplus, step=False):
    try:
        return _scan_plan(where, u.shape, A.shape, B.shape, B.stride(), C.shape, C.stride(),
                          None if z is None else z.stride(), u.dtype, bool(softplus), step)
    except (AttributeError, TypeError, Mamba2Error):
        _tensors(where, u=u, A=A, B=B, C=C)
        if z is not None:
            _tensors(where, z=z)
        raise


def _scan_plain(i, u, dt, A, B, C, D, z, dt_bias, ashape, cshape, bcshape):
    io = u.dtype
    return (i >= 0 and u.is_contiguous() and _plain(dt, io, u.shape, i)
            and _plain(A, _F32, ashape, i) and B.dtype is io and B.shape == bcshape
            and B.get_device() == i and C.dtype is io and C.shape == bcshape
            and C.get_device() == i and _optional(D, _F32, cshape, i)
            and (z is None or (z.dtype is io and z.shape == u.shape and z.get_device() == i))
            and _optional(dt_bias, _F32, cshape, i))


def selective_scan_forward(u, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *,
                           softplus=True, lengths=None, workspace=None, stream=None):
    """The selective scan of u[B,L,D] with time steps softplus(dt + dt_bias) (dt + dt_bias
    with softplus=False), decays A[D,N], B and C [B,L,G,N], skip D[D] and gate z[B,L,D]
    (z, B and C may be column ranges of wider rows).  Returns (y[B,L,D],
    final_state[B,D,N])."""
    dims, ref, state, ashape, cshape, bc, need, _ = _scan_plan_of(
        "selective_scan_forward", u, A, B, C, z, softplus)
    with _owner(stream, u):
        workspace, n = _workspace("selective_scan_forward", need, workspace, u)
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
        final = u.new_empty(state, dtype=_F32)
    i = u.get_device()
    if (n >= need > 0 and _scan_plain(i, u, dt, A, B, C, D, z, dt_bias, ashape, cshape, bc)
            and _optional(init_state, _F32, state, i) and _optional(lengths, _I32, u.shape[:1], i)
            and workspace.is_contiguous() and workspace.get_device() == i):
        _launch(_lib.mamba2_selective_scan_forward, "selective_scan_forward", i, stream, ref,
                u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D),
                _ptr(z), _ptr(dt_bias), _ptr(init_state), _ptr(lengths), y.data_ptr(),
                final.data_ptr(), workspace.data_ptr(), n)
    else:
        _given("selective_scan_forward", dt=dt, D=D, dt_bias=dt_bias, init_state=init_state,
               lengths=lengths)
        mamba2_selective_scan_forward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths, y,
                                      final, workspace, n, stream)
    return y, final


def selective_scan_backward(u, dt, A, B, C, D, z, dt_bias, init_state, dy, dfinal=None, *,
                            softplus=True, lengths=None, workspace=None, stream=None):
    """Gradients of selective_scan_forward: a dict with du, ddt, dA, dB, dC, dD (None
    without D), dz (None without z), ddt_bias (None without dt_bias) and dinit."""
    dims, ref, state, ashape, cshape, bc, _, need = _scan_plan_of(
        "selective_scan_backward", u, A, B, C, z, softplus)
    with _owner(stream, u):
        workspace, n = _workspace("selective_scan_backward", need, workspace, u)
        du, ddt = u.new_empty(u.shape), u.new_empty(u.shape)
        dA, dB, dC = _like(A), u.new_empty(B.shape), u.new_empty(C.shape)
        dD = _like(D)
        dz = None if z is None else u.new_empty(u.shape)
        dbias = _like(dt_bias)
        dinit = u.new_empty(state, dtype=_F32)
    i = u.get_device()
    if (n >= need > 0 and _scan_plain(i, u, dt, A, B, C, D, z, dt_bias, ashape, cshape, bc)
            and _plain(dy, u.dtype, u.shape, i)
            and _optional(init_state, _F32, state, i) and _optional(dfinal, _F32, state, i)
            and _optional(lengths, _I32, u.shape[:1], i)
            and workspace.is_contiguous() and workspace.get_device() == i):
        _launch(_lib.mamba2_selective_scan_backward, "selective_scan_backward", i, stream, ref,
                u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D),
                _ptr(z), _ptr(dt_bias), _ptr(init_state), _ptr(lengths), dy.data_ptr(),
                _ptr(dfinal), du.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(),
                dC.data_ptr(), _ptr(dD), _ptr(dz), _ptr(dbias), dinit.data_ptr(),
                workspace.data_ptr(), n)
    else:
        _given("selective_scan_backward", dt=dt, D=D, dt_bias=dt_bias, init_state=init_state, dy=dy,
               dfinal=dfinal, lengths=lengths)
        mamba2_selective_scan_backward(dims, u, dt, A, B, C, D, z, dt_bias, init_state, lengths,
                                       dy, dfinal, du, ddt, dA, dB, dC, dD, dz, dbias, dinit,
                                       workspace, n, stream)
    return {"du": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "dz": dz,
            "ddt_bias": dbias, "dinit": dinit}


def selective_scan_step(u, dt, A, B, C, D, z, dt_bias, state, *, softplus=True, stream=None):
    """One token of every sequence: u, dt, z [B,D], B, C [B,G,N]; ``state``[B,D,N] is
    updated in place.  Returns y[B,D]."""
    dims, ref, sshape, ashape, cshape, bc, _, _ = _scan_plan_of(
        "selective_scan_step", u, A, B, C, z, softplus, True)
    with _owner(stream, u):
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    i = u.get_device()
    if (_plain(state, _F32, sshape, i)
            and _scan_plain(i, u, dt, A, B, C, D, z, dt_bias, ashape, cshape, bc)):
        _launch(_lib.mamba2_selective_scan_step, "selective_scan_step", i, stream, ref,
                u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D),
                _ptr(z), _ptr(dt_bias), state.data_ptr(), y.data_ptr())
    else:
        _given("selective_scan_step", dt=dt, D=D, dt_bias=dt_bias, state=state)
        mamba2_selective_scan_step(dims, u, dt, A, B, C, D, z, dt_bias, state, y, stream)
    return y


# ------------------------------------------------------------------------ norm


def make_norm_dims(rows, channels, ngroups, dtype, *, kind="rms", eps=1e-5, x_stride=0, z_stride=0,
                   dz_stride=0) -> Mamba2NormDims:
    if not _known(kind, _KINDS):
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


@functools.lru_cache(maxsize=256)
def _norm_plan(where, shape, strides, zshape, zstrides, ngroups, kind, eps, dtype):
    """dims, the weight's shape and the backward's workspace of a call with these sizes."""
    if len(shape) < 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"x {tuple(shape)} must be at least 2-d")
    if dtype is not _F32 and dtype is not _BF16:
        raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"x is {dtype}, needs float32 or bfloat16")
    if zshape is not None and zshape != shape:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"z has shape {tuple(zshape)}, needs {tuple(shape)}")
    lead = len(shape) - 1
    dims = make_norm_dims(
        shape[:-1].numel(), shape[-1], ngroups, dtype, kind=kind, eps=eps,
        x_stride=_stride(where, "x", shape, strides, lead),
        z_stride=0 if zshape is None else _stride(where, "z", shape, zstrides, lead))
    return (dims, ctypes.byref(dims), shape[-1:], mamba2_norm_backward_workspace_bytes(dims))


def _norm_plan_of(where, x, z, ngroups, kind, eps):
    try:
        return _norm_plan(where, x.shape, x.stride(), None if z is None else z.shape,
                          None if z is None else z.stride(), ngroups, kind, float(eps), x.dtype)
    except (AttributeError, TypeError, Mamba2Error) as e:
        _tensors(where, x=x)
        if z is not None:
            _tensors(where, z=z)
        if isinstance(e, Mamba2Error):
            raise
        if not _known(kind, _KINDS):
            raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, where, f"unknown norm {kind!r}") from None
        raise


def _rows(t, dims):
    return None if t is None else t.view(dims.rows, dims.channels)


def norm_forward(x, weight, bias=None, z=None, *, ngroups=1, kind="rms", eps=1e-5, stream=None):
    """RMS norm (kind="rms") or layer norm ("layer") of x, or of x * silu(z), over
    ``ngroups`` groups of the last axis; weight and bias [D] float32.  Returns y."""
    dims, ref, wshape, _ = _norm_plan_of("norm_forward", x, z, ngroups, kind, eps)
    with _owner(stream, x):
        y = x.new_empty(x.shape)
    i = x.get_device()
    if (i >= 0 and _plain(weight, _F32, wshape, i) and _optional(bias, _F32, wshape, i)
            and (z is None or (z.dtype is x.dtype and z.get_device() == i))):
        _launch(_lib.mamba2_norm_forward, "norm_forward", i, stream, ref, x.data_ptr(), _ptr(z),
                weight.data_ptr(), _ptr(bias), y.data_ptr())
    else:
        _given("norm_forward", weight=weight, bias=bias)
        mamba2_norm_forward(dims, _rows(x, dims), _rows(z, dims), weight, bias, _rows(y, dims),
                            stream)
    return y


def norm_backward(x, weight, bias, z, dy, *, ngroups=1, kind="rms", eps=1e-5, workspace=None,
                  stream=None):
    """Gradients of norm_forward: a dict with dx, dweight, dbias (None without bias)
    and dz (None without z)."""
    dims, ref, wshape, need = _norm_plan_of("norm_backward", x, z, ngroups, kind, eps)
    if not isinstance(dy, _Tensor):
        _tensors("norm_backward", dy=dy)
    if not (bias is None or isinstance(bias, _Tensor)):
        _tensors("norm_backward", bias=bias)
    if dy.shape != x.shape or not dy.is_contiguous():
        raise Mamba2Error(MAMBA2_ERR_SHAPE, "norm_backward",
                          f"dy {tuple(dy.shape)} must be contiguous and of x's shape "
                          f"{tuple(x.shape)}")
    with _owner(stream, x):
        workspace, n = _workspace("norm_backward", need, workspace, x)
        g = {"dx": x.new_empty(x.shape), "dweight": _like(weight), "dbias": _like(bias),
             "dz": None if z is None else x.new_empty(x.shape)}
    i = x.get_device()
    if (i >= 0 and n >= need > 0 and _plain(weight, _F32, wshape, i)
            and _optional(bias, _F32, wshape, i) and dy.dtype is x.dtype and dy.get_device() == i
            and (z is None or (z.dtype is x.dtype and z.get_device() == i))
            and workspace.is_contiguous() and workspace.get_device() == i):
        _launch(_lib.mamba2_norm_backward, "norm_backward", i, stream, ref, x.data_ptr(), _ptr(z),
                weight.data_ptr(), dy.data_ptr(), g["dx"].data_ptr(), _ptr(g["dz"]),
                g["dweight"].data_ptr(), _ptr(g["dbias"]), workspace.data_ptr(), n)
    else:
        _given("norm_backward", weight=weight, bias=bias)
        mamba2_norm_backward(dims, _rows(x, dims), _rows(z, dims), weight, _rows(dy, dims),
                             _rows(g["dx"], dims), _rows(g["dz"], dims), g["dweight"], g["dbias"],
                             workspace, n, stream)
    return g

"""The operators of an attention layer between SSD layers: rotary, attention
and attention_step.

Same manner as ``layer.py``: ``mamba2_*`` functions keep the C names and
arguments and check every tensor against ``dims`` first; the short names
(``rotary_forward`` ...) make the dims, allocate outputs and workspace with
torch and call them.  q, k and v may be column ranges of wider rows (one
projection's output); every other tensor is contiguous.  Calls run on the
device of their tensors, on that device's current stream unless ``stream`` is
given.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import (MAMBA2_DTYPE_BF16, MAMBA2_DTYPE_F32, MAMBA2_ERR_DTYPE, MAMBA2_ERR_SHAPE,
               MAMBA2_ERR_UNSUPPORTED, Mamba2AttentionDims, Mamba2AttentionStepDims, Mamba2Error,
               Mamba2RotaryDims, _lib, _ptr, _req_bytes)
from .layer import (_BF16, _F32, _I32, _Tensor, _call, _given, _io, _known, _launch, _optional,
                    _owner, _plain, _stride, _tensors, _want, _workspace)

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = ("none", "linear", "base", "parts")


def _code(dtype):
    return MAMBA2_DTYPE_BF16 if dtype is _BF16 else MAMBA2_DTYPE_F32 if dtype is _F32 else int(dtype)


def _number(where, name, v):
    try:
        return float(v)
    except (TypeError, ValueError, OverflowError):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"{name} is {v!r}, not a number") from None


def _known_dtype(where, dtype):
    if dtype is not _F32 and dtype is not _BF16:
        raise Mamba2Error(MAMBA2_ERR_DTYPE, where, f"q is {dtype}, needs float32 or bfloat16")


# ---------------------------------------------------------------------- rotary


def rotary_frequencies(rotary, base=10000.0, *, scaling="none", factor=1.0, original_length=None,
                       fast=32.0, slow=1.0, device=None):
    """(inv_freq[rotary/2] float32, scale) for rotary_forward: base^(-2i/rotary), stretched for
    contexts ``factor`` times as long.  ``scaling``: "none"; "linear": every frequency divided
    by factor; "base" (published as the NTK-aware change of base): the base raised by
    factor^(rotary/(rotary-2)), so that the lowest frequency is divided by factor and the highest
    stays (rotary = 2 has but the highest, and no effect); "parts" (published as YaRN): frequencies
    that turn more than ``fast`` times within ``original_length`` tokens stay, those under ``slow``
    times are divided by factor, a ramp between, with scale = 0.1 ln(factor) + 1 on q and k.  Formed
    in float64."""
    w = "rotary_frequencies"
    if scaling not in _SCALINGS:
        raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, w, f"unknown scaling {scaling!r}")
    if not isinstance(rotary, int) or rotary < 2 or rotary % 2:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, w, f"rotary must be even and at least 2 (got {rotary!r})")
    base, factor = _number(w, "base", base), _number(w, "factor", factor)
    if not (1 < base < math.inf and 1 <= factor < math.inf):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, w,
                          f"base must be above 1 and factor at least 1 (got {base}, {factor})")
    if scaling == "base" and rotary > 2:
        try:
            base *= factor ** (rotary / (rotary - 2))
        except OverflowError:
            base = math.inf
        if base == math.inf:
            raise Mamba2Error(MAMBA2_ERR_SHAPE, w, f"factor {factor} takes the base beyond float64")
    f = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        fast, slow = _number(w, "fast", fast), _number(w, "slow", slow)
        if original_length is not None:
            original_length = _number(w, "original_length", original_length)
        try:
            if original_length is None or not (original_length >= 1 and 0 < slow < fast):
                raise ValueError
            # the ramp is linear in i between the frequencies with `fast` and `slow` turns
            turns_at = [rotary * math.log(original_length / (t * 2 * math.pi)) / (2 * math.log(base))
                        for t in (fast, slow)]
            lo, hi = max(math.floor(turns_at[0]), 0), min(math.ceil(turns_at[1]), rotary - 1)
        except (ValueError, OverflowError):  # the logarithm of 0 or infinity among them
            raise Mamba2Error(MAMBA2_ERR_SHAPE, w,
                              "parts needs original_length >= 1 and 0 < slow < fast, all finite (got "
                              f"{original_length}, {slow}, {fast})") from None
        # no room between the ends: the context is shorter than `slow` turns of the first frequency
        # (hi <= 0, all are divided) or all frequencies turn more than `fast` times (none is)
        i = torch.arange(rotary // 2, dtype=torch.float64)
        ramp = ((i - lo) / (hi - lo)).clamp(0, 1) if hi > lo else (i >= hi).to(i.dtype)
        f = f / factor * ramp + f * (1 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(_F32).to(device), scale


def make_rotary_dims(batch, seqlen, nheads, ngroups, headdim, rotary, dtype, *, layout="half",
                     scale=1.0, q_stride=0, k_stride=0, yq_stride=0,
                     yk_stride=0) -> Mamba2RotaryDims:
    if not _known(layout, _LAYOUTS):
        raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, "make_rotary_dims", f"unknown layout {layout!r}")
    return Mamba2RotaryDims(batch, seqlen, nheads, ngroups, headdim, rotary, q_stride, k_stride,
                            yq_stride, yk_stride, scale, _LAYOUTS[layout], _code(dtype), 0)


def _rotary(w, names, dims, q, k, inv_freq, positions, yq, yk, stream):
    b, L, d, io = dims.batch, dims.seqlen, dims.headdim, _io(dims)
    _want(w, names[0], q, (b, L, dims.nheads, d), io, stride=dims.q_stride, lead=2)
    _want(w, names[2], yq, (b, L, dims.nheads, d), io, stride=dims.yq_stride, lead=2)
    none = dims.ngroups == 0
    if not none:
        _want(w, names[1], k, (b, L, dims.ngroups, d), io, stride=dims.k_stride, lead=2)
        _want(w, names[3], yk, (b, L, dims.ngroups, d), io, stride=dims.yk_stride, lead=2)
    _want(w, "inv_freq", inv_freq, (dims.rotary // 2,), _F32)
    _want(w, "positions", positions, (b, L), _I32, optional=True)
    ts = (q, inv_freq, positions, yq) if none else (q, k, inv_freq, positions, yq, yk)
    _call(w, stream, ts, ctypes.byref(dims), _ptr(q), None if none else _ptr(k), _ptr(inv_freq),
          _ptr(positions), _ptr(yq), None if none else _ptr(yk))


def mamba2_rotary_forward(dims, q, k, inv_freq, positions, yq, yk, stream=None):
    _rotary("mamba2_rotary_forward", ("q", "k", "yq", "yk"), dims, q, k, inv_freq, positions, yq,
            yk, stream)


def mamba2_rotary_backward(dims, dyq, dyk, inv_freq, positions, dq, dk, stream=None):
    _rotary("mamba2_rotary_backward", ("dyq", "dyk", "dq", "dk"), dims, dyq, dyk, inv_freq,
            positions, dq, dk, stream)


@functools.lru_cache(maxsize=256)
def _rotary_plan(where, shape, strides, kshape, kstrides, pairs, layout, scale, dtype):
    """dims and the shape of the tokens."""
    _known_dtype(where, dtype)
    if len(shape) < 3 or (kshape is not None and len(kshape) != len(shape)):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"q {tuple(shape)} and k must be [..., heads, headdim] with as many axes")
    lead = shape[:-2]
    if kshape is not None and (kshape[:-2] != lead or kshape[-1] != shape[-1]):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"k {tuple(kshape)} does not match q {tuple(shape)}")
    n = len(lead)
    dims = make_rotary_dims(
        lead[:-1].numel(), lead[-1], shape[-2], 0 if kshape is None else kshape[-2], shape[-1],
        2 * pairs, dtype, layout=layout, scale=scale,
        q_stride=_stride(where, "q", shape, strides, n),
        k_stride=0 if kshape is None else _stride(where, "k", kshape, kstrides, n))
    return dims, ctypes.byref(dims), lead


def _rotary_short(where, full, fn, names, q, k, inv_freq, positions, layout, scale, stream):
    try:
        dims, ref, lead = _rotary_plan(
            where, q.shape, q.stride(), None if k is None else k.shape,
            None if k is None else k.stride(), inv_freq.shape[0], layout, float(scale), q.dtype)
    except (AttributeError, IndexError, TypeError, ValueError, Mamba2Error) as e:
        _tensors(where, **{names[0]: q, "inv_freq": inv_freq})
        if k is not None:
            _tensors(where, **{names[1]: k})
        if isinstance(e, Mamba2Error):
            raise
        if not _known(layout, _LAYOUTS):
            raise Mamba2Error(MAMBA2_ERR_UNSUPPORTED, where, f"unknown layout {layout!r}") from None
        _number(where, "scale", scale)
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"inv_freq {tuple(inv_freq.shape)} must be 1-d") from None
    with _owner(stream, q):
        yq = q.new_empty(q.shape)
        yk = None if k is None else q.new_empty(k.shape)
    i = q.get_device()
    if (i >= 0 and _plain(inv_freq, _F32, inv_freq.shape[:1], i)
            and _optional(positions, _I32, lead, i)
            and (k is None or (k.dtype is q.dtype and k.get_device() == i))):
        _launch(fn, where, i, stream, ref, q.data_ptr(), _ptr(k), inv_freq.data_ptr(),
                _ptr(positions), yq.data_ptr(), _ptr(yk))
    else:
        if positions is not None:
            _tensors(where, positions=positions)
            if positions.shape != lead:
                raise Mamba2Error(MAMBA2_ERR_SHAPE, where, f"positions has shape "
                                  f"{tuple(positions.shape)}, needs {tuple(lead)}")
            if not positions.is_contiguous():
                raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                                  f"positions is not contiguous (strides {positions.stride()})")
            positions = positions.view(dims.batch, dims.seqlen)

        def rows(t, heads):
            # the tokens are at equal steps (dims was made), so they have a 2-d form
            if t is None:
                return None
            return t.as_strided((dims.batch, dims.seqlen, heads, dims.headdim),
                                (dims.seqlen * t_stride(t), t_stride(t), dims.headdim, 1))

        def t_stride(t):
            return _stride(where, "q", t.shape, t.stride(), len(lead))

        full(dims, rows(q, dims.nheads), rows(k, dims.ngroups), inv_freq, positions,
             rows(yq, dims.nheads), rows(yk, dims.ngroups), stream)
    return yq if k is None else (yq, yk)


def rotary_forward(q, k, inv_freq, positions=None, *, layout="half", scale=1.0, stream=None):
    """q[..., H, D] and k[..., G, D] (or None) of the same tokens with the first 2 *
    len(inv_freq) elements of every head turned by position * inv_freq.  ``positions``: int32 of
    the tokens' shape; None: a token's index along the last token axis.  ``layout``: "half"
    (pairs i, i + R/2) or "interleaved" (2i, 2i + 1).  Returns yq, or (yq, yk)."""
    return _rotary_short("rotary_forward", mamba2_rotary_forward, _lib.mamba2_rotary_forward,
                         ("q", "k"), q, k, inv_freq, positions, layout, scale, stream)


def rotary_backward(dyq, dyk, inv_freq, positions=None, *, layout="half", scale=1.0, stream=None):
    """Gradients of rotary_forward's q and k from those of its outputs: dq, or (dq, dk)."""
    return _rotary_short("rotary_backward", mamba2_rotary_backward, _lib.mamba2_rotary_backward,
                         ("dyq", "dyk"), dyq, dyk, inv_freq, positions, layout, scale, stream)


# ------------------------------------------------------------------- attention


def make_attention_dims(batch, q_len, k_len, nheads, ngroups, headdim, dtype, *, causal=True,
                        scale=None, q_packed=False, k_packed=False, q_stride=0, k_stride=0,
                        v_stride=0, dq_stride=0, dk_stride=0, dv_stride=0) -> Mamba2AttentionDims:
    if scale is None:
        scale = 1 / math.sqrt(headdim) if headdim > 0 else 1.0
    return Mamba2AttentionDims(batch, q_len, k_len, nheads, ngroups, headdim, q_stride, k_stride,
                               v_stride, dq_stride, dk_stride, dv_stride, scale, int(causal),
                               int(q_packed), int(k_packed), _code(dtype), 0)


def mamba2_attention_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_attention_workspace_bytes(ctypes.byref(dims)))


def mamba2_attention_backward_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_attention_backward_workspace_bytes(ctypes.byref(dims)))


def _attention_leads(dims):
    return ((dims.q_len,) if dims.q_packed else (dims.batch, dims.q_len),
            (dims.k_len,) if dims.k_packed else (dims.batch, dims.k_len))


def _attention_args(w, dims, q, k, v, q_seqs, k_seqs, o, lse):
    lq, lk = _attention_leads(dims)
    io, d = _io(dims), dims.headdim
    _want(w, "q", q, lq + (dims.nheads, d), io, stride=dims.q_stride, lead=len(lq))
    _want(w, "k", k, lk + (dims.ngroups, d), io, stride=dims.k_stride, lead=len(lk))
    _want(w, "v", v, lk + (dims.ngroups, d), io, stride=dims.v_stride, lead=len(lk))
    for name, t, packed in (("q_seqs", q_seqs, dims.q_packed), ("k_seqs", k_seqs, dims.k_packed)):
        _want(w, name, t, (dims.batch + (1 if packed else 0),), _I32, optional=not packed)
    _want(w, "o", o, lq + (dims.nheads, d), io)
    _want(w, "lse", lse, lq + (dims.nheads,), _F32)


def mamba2_attention_forward(dims, q, k, v, q_seqs, k_seqs, o, lse, workspace, workspace_bytes,
                             stream=None):
    w = "mamba2_attention_forward"
    _attention_args(w, dims, q, k, v, q_seqs, k_seqs, o, lse)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (q, k, v, q_seqs, k_seqs, o, lse, workspace), ctypes.byref(dims), _ptr(q),
          _ptr(k), _ptr(v), _ptr(q_seqs), _ptr(k_seqs), _ptr(o), _ptr(lse), _ptr(workspace),
          int(workspace_bytes))


def mamba2_attention_backward(dims, q, k, v, q_seqs, k_seqs, o, lse, dout, dq, dk, dv, workspace,
                              workspace_bytes, stream=None):
    w = "mamba2_attention_backward"
    _attention_args(w, dims, q, k, v, q_seqs, k_seqs, o, lse)
    lq, lk = _attention_leads(dims)
    io, d = _io(dims), dims.headdim
    _want(w, "dout", dout, lq + (dims.nheads, d), io)
    _want(w, "dq", dq, lq + (dims.nheads, d), io, stride=dims.dq_stride, lead=len(lq))
    _want(w, "dk", dk, lk + (dims.ngroups, d), io, stride=dims.dk_stride, lead=len(lk))
    _want(w, "dv", dv, lk + (dims.ngroups, d), io, stride=dims.dv_stride, lead=len(lk))
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (q, k, v, q_seqs, k_seqs, o, lse, dout, dq, dk, dv, workspace),
          ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(q_seqs), _ptr(k_seqs), _ptr(o),
          _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
          int(workspace_bytes))


@functools.lru_cache(maxsize=256)
def _attention_plan(where, qshape, qstrides, kshape, kstrides, vshape, vstrides, qstarts, kstarts,
                    causal, scale, dtype):
    """dims, the shapes of lse and of the lengths or starts, and the workspaces.  qstarts and
    kstarts: the starts' shapes where a side is packed, else None."""
    _known_dtype(where, dtype)
    nq, nk = (3 if s is not None else 4 for s in (qstarts, kstarts))
    if len(qshape) != nq or len(kshape) != nk or kshape != vshape:
        raise Mamba2Error(
            MAMBA2_ERR_SHAPE, where,
            f"q {tuple(qshape)}, k {tuple(kshape)}, v {tuple(vshape)}: padded sequences are "
            "[batch, len, heads, headdim], packed ones (with starts) [rows, heads, headdim]; k "
            "and v alike")
    for name, s in (("q_starts", qstarts), ("k_starts", kstarts)):
        if s is not None and (len(s) != 1 or s[0] < 2):
            raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                              f"{name} {tuple(s)} must be 1-d, one more than the sequences")
    batch = qshape[0] if qstarts is None else qstarts[0] - 1
    other = kshape[0] if kstarts is None else kstarts[0] - 1
    if batch != other or qshape[-1] != kshape[-1]:
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"q {tuple(qshape)} and k {tuple(kshape)}: {batch} and {other} "
                          "sequences, or another headdim")
    dims = make_attention_dims(
        batch, qshape[-3], kshape[-3], qshape[-2], kshape[-2], qshape[-1], dtype, causal=causal,
        scale=scale, q_packed=qstarts is not None, k_packed=kstarts is not None,
        q_stride=_stride(where, "q", qshape, qstrides, nq - 2),
        k_stride=_stride(where, "k", kshape, kstrides, nk - 2),
        v_stride=_stride(where, "v", vshape, vstrides, nk - 2))
    return (dims, ctypes.byref(dims), torch.Size(qshape[:-1]),
            torch.Size((batch + (qstarts is not None),)),
            torch.Size((batch + (kstarts is not None),)), mamba2_attention_workspace_bytes(dims),
            mamba2_attention_backward_workspace_bytes(dims))


def _attention_plan_of(where, q, k, v, q_lengths, k_lengths, q_starts, k_starts, causal, scale):
    try:
        plan = _attention_plan(where, q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(),
                               None if q_starts is None else q_starts.shape,
                               None if k_starts is None else k_starts.shape, bool(causal),
                               None if scale is None else float(scale), q.dtype)
    except (AttributeError, TypeError, ValueError, Mamba2Error) as e:
        _tensors(where, q=q, k=k, v=v)
        if q_starts is not None:
            _tensors(where, q_starts=q_starts)
        if k_starts is not None:
            _tensors(where, k_starts=k_starts)
        if isinstance(e, Mamba2Error):
            raise
        _number(where, "scale", scale)
        raise
    if (q_starts is not None and q_lengths is not None) or (
            k_starts is not None and k_lengths is not None):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where, "a side has lengths (padded) or starts (packed)")
    return (plan, q_lengths if q_starts is None else q_starts,
            k_lengths if k_starts is None else k_starts)


def _qkv_plain(i, q, k, v):
    return (i >= 0 and k.dtype is q.dtype and v.dtype is q.dtype and k.get_device() == i
            and v.get_device() == i)


def attention_forward(q, k, v, *, causal=True, scale=None, q_lengths=None, k_lengths=None,
                      q_starts=None, k_starts=None, workspace=None, stream=None):
    """Softmax attention of q[B,Lq,H,D] to k, v [B,Lk,G,D] (padded; ``q_lengths`` and
    ``k_lengths`` int32 [B], None: full), or of q[T,H,D] and k, v [T,G,D] with ``q_starts`` and
    ``k_starts`` int32 [B+1] (packed; each side by itself).  Causal: a sequence's last query sees
    all of its keys.  ``scale``: 1/sqrt(D) if None.  Returns (o like q, lse [..., H] float32)."""
    w = "attention_forward"
    (dims, ref, lshape, qn, kn, need, _), qs, ks = _attention_plan_of(
        w, q, k, v, q_lengths, k_lengths, q_starts, k_starts, causal, scale)
    with _owner(stream, q):
        workspace, n = _workspace(w, need, workspace, q)
        o = q.new_empty(q.shape)
        lse = q.new_empty(lshape, dtype=_F32)
    i = q.get_device()
    if (n >= need > 0 and _qkv_plain(i, q, k, v) and _optional(qs, _I32, qn, i)
            and _optional(ks, _I32, kn, i) and workspace.is_contiguous()
            and workspace.get_device() == i):
        _launch(_lib.mamba2_attention_forward, w, i, stream, ref, q.data_ptr(), k.data_ptr(),
                v.data_ptr(), _ptr(qs), _ptr(ks), o.data_ptr(), lse.data_ptr(),
                workspace.data_ptr(), n)
    else:
        _given(w, q_lengths=q_lengths, k_lengths=k_lengths)
        mamba2_attention_forward(dims, q, k, v, qs, ks, o, lse, workspace, n, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dout, *, causal=True, scale=None, q_lengths=None,
                       k_lengths=None, q_starts=None, k_starts=None, workspace=None, stream=None):
    """Gradients of attention_forward from o and lse, its outputs for the same arguments, and
    dout, the gradient of o: a dict with dq, dk and dv."""
    w = "attention_backward"
    (dims, ref, lshape, qn, kn, _, need), qs, ks = _attention_plan_of(
        w, q, k, v, q_lengths, k_lengths, q_starts, k_starts, causal, scale)
    with _owner(stream, q):
        workspace, n = _workspace(w, need, workspace, q)
        g = {"dq": q.new_empty(q.shape), "dk": q.new_empty(k.shape), "dv": q.new_empty(v.shape)}
    i = q.get_device()
    if (n >= need > 0 and _qkv_plain(i, q, k, v) and _optional(qs, _I32, qn, i)
            and _optional(ks, _I32, kn, i) and _plain(o, q.dtype, q.shape, i)
            and _plain(dout, q.dtype, q.shape, i) and _plain(lse, _F32, lshape, i)
            and workspace.is_contiguous() and workspace.get_device() == i):
        _launch(_lib.mamba2_attention_backward, w, i, stream, ref, q.data_ptr(), k.data_ptr(),
                v.data_ptr(), _ptr(qs), _ptr(ks), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(), workspace.data_ptr(),
                n)
    else:
        _given(w, q_lengths=q_lengths, k_lengths=k_lengths, o=o, lse=lse, dout=dout)
        mamba2_attention_backward(dims, q, k, v, qs, ks, o, lse, dout, g["dq"], g["dk"], g["dv"],
                                  workspace, n, stream)
    return g


# ------------------------------------------------------------------- one token


def make_attention_step_dims(batch, rows, nheads, ngroups, headdim, dtype, *, prefix=0, scale=None,
                             q_stride=0, k_stride=0, v_stride=0) -> Mamba2AttentionStepDims:
    if scale is None:
        scale = 1 / math.sqrt(headdim) if headdim > 0 else 1.0
    return Mamba2AttentionStepDims(batch, rows, prefix, nheads, ngroups, headdim, q_stride,
                                   k_stride, v_stride, scale, _code(dtype))


def mamba2_attention_step_workspace_bytes(dims) -> int:
    return int(_lib.mamba2_attention_step_workspace_bytes(ctypes.byref(dims)))


def mamba2_attention_step(dims, q, k, v, k_cache, v_cache, lengths, k_prefix, v_prefix, o,
                          workspace, workspace_bytes, stream=None):
    w = "mamba2_attention_step"
    b, g, d, io = dims.batch, dims.ngroups, dims.headdim, _io(dims)
    _want(w, "q", q, (b, dims.nheads, d), io, stride=dims.q_stride, lead=1)
    _want(w, "k", k, (b, g, d), io, stride=dims.k_stride, lead=1)
    _want(w, "v", v, (b, g, d), io, stride=dims.v_stride, lead=1)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _want(w, name, t, (b, dims.rows, g, d), io)
    _want(w, "lengths", lengths, (b,), _I32)
    if dims.prefix:
        for name, t in (("k_prefix", k_prefix), ("v_prefix", v_prefix)):
            _want(w, name, t, (dims.prefix, g, d), io)
    else:
        k_prefix = v_prefix = None
    _want(w, "o", o, (b, dims.nheads, d), io)
    _req_bytes(w, "workspace", workspace, workspace_bytes)
    _call(w, stream, (q, k, v, k_cache, v_cache, lengths, k_prefix, v_prefix, o, workspace),
          ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
          _ptr(lengths), _ptr(k_prefix), _ptr(v_prefix), _ptr(o), _ptr(workspace),
          int(workspace_bytes))


@functools.lru_cache(maxsize=256)
def _step_plan(where, qshape, qstrides, kshape, kstrides, vshape, vstrides, cshape, pshape, scale,
               dtype):
    """dims, the prefix's shape and the workspace."""
    _known_dtype(where, dtype)
    if len(qshape) != 3 or len(kshape) != 3 or kshape != vshape or len(cshape) != 4 or (
            pshape is not None and len(pshape) != 3):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, where,
                          f"q {tuple(qshape)}, k {tuple(kshape)} and v {tuple(vshape)} must be "
                          f"3-d, k and v alike, the caches {tuple(cshape)} 4-d, a prefix 3-d")
    dims = make_attention_step_dims(
        qshape[0], cshape[1], qshape[1], kshape[1], qshape[2], dtype, scale=scale,
        prefix=0 if pshape is None else pshape[0],
        q_stride=_stride(where, "q", qshape, qstrides, 1),
        k_stride=_stride(where, "k", kshape, kstrides, 1),
        v_stride=_stride(where, "v", vshape, vstrides, 1))
    b, g, d = qshape[0], kshape[1], qshape[2]
    return (dims, ctypes.byref(dims), torch.Size((b, g, d)), torch.Size((b, cshape[1], g, d)),
            torch.Size((dims.prefix, g, d)), mamba2_attention_step_workspace_bytes(dims))


def attention_step(q, k, v, k_cache, v_cache, lengths, k_prefix=None, v_prefix=None, *, scale=None,
                   workspace=None, stream=None):
    """One token of every sequence: q[B,H,D], k, v [B,G,D] against the caches [B,rows,G,D], of
    which sequence b holds ``lengths``[b] (int32) rows, and a prefix [P,G,D] that comes before
    all of them (or None).  k and v are written to row lengths[b] of the caches (a full cache
    keeps its rows); lengths is left to the caller, who adds one once all layers are done.
    Returns o[B,H,D]."""
    w = "attention_step"
    try:
        dims, ref, kshape, cshape, pshape, need = _step_plan(
            w, q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(), k_cache.shape,
            None if k_prefix is None else k_prefix.shape, None if scale is None else float(scale),
            q.dtype)
    except (AttributeError, TypeError, ValueError, Mamba2Error) as e:
        _tensors(w, q=q, k=k, v=v, k_cache=k_cache)
        if k_prefix is not None:
            _tensors(w, k_prefix=k_prefix)
        if isinstance(e, Mamba2Error):
            raise
        _number(w, "scale", scale)
        raise
    if (k_prefix is None) != (v_prefix is None):
        raise Mamba2Error(MAMBA2_ERR_SHAPE, w, "k_prefix and v_prefix come together")
    if k_prefix is not None and dims.prefix == 0:
        k_prefix = v_prefix = None
    with _owner(stream, q):
        workspace, n = _workspace(w, need, workspace, q)
        o = q.new_empty(q.shape)
    i = q.get_device()
    io = q.dtype
    if (n >= need > 0 and _qkv_plain(i, q, k, v) and k.shape == kshape
            and _plain(k_cache, io, cshape, i) and _plain(v_cache, io, cshape, i)
            and _plain(lengths, _I32, kshape[:1], i) and _optional(k_prefix, io, pshape, i)
            and _optional(v_prefix, io, pshape, i) and workspace.is_contiguous()
            and workspace.get_device() == i):
        _launch(_lib.mamba2_attention_step, w, i, stream, ref, q.data_ptr(), k.data_ptr(),
                v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), lengths.data_ptr(),
                _ptr(k_prefix), _ptr(v_prefix), o.data_ptr(), workspace.data_ptr(), n)
    else:
        _given(w, v_cache=v_cache, lengths=lengths, v_prefix=v_prefix)
        mamba2_attention_step(dims, q, k, v, k_cache, v_cache, lengths, k_prefix, v_prefix, o,
                              workspace, n, stream)
    return o

"""Host-only checks of the operators around the SSD: their structs, refusals
of the C interface before anything touches a device, and the wrappers' checks
of tensors.  None of these calls launches a kernel."""
import ctypes

import pytest
import torch

import state_space_sequence_02_amd as m2

OK = 1 << 20  # a 16-byte aligned address that is never read: checks fail first
BIG = 1 << 40


def test_struct_layouts():
    assert ctypes.sizeof(m2.Mamba2ConvDims) == 9 * 8 + 2 * 4
    assert m2.Mamba2ConvDims.part.offset == 32 and m2.Mamba2ConvDims.dtype.offset == 72
    assert ctypes.sizeof(m2.Mamba2ScanDims) == 9 * 8 + 2 * 4
    assert m2.Mamba2ScanDims.dtype.offset == 72
    assert ctypes.sizeof(m2.Mamba2NormDims) == 6 * 8 + 4 * 4
    assert m2.Mamba2NormDims.eps.offset == 48 and m2.Mamba2NormDims.reserved.offset == 60


def _conv(**kw):
    a = dict(batch=2, seqlen=100, channels=96, width=4, parts=(64, 16, 16), dtype=torch.bfloat16)
    a.update(kw)
    return m2.make_conv_dims(**a)


def _scan(**kw):
    a = dict(batch=2, seqlen=100, channels=96, dstate=16, ngroups=2, dtype=torch.bfloat16)
    a.update(kw)
    return m2.make_scan_dims(**a)


def _norm(**kw):
    a = dict(rows=10, channels=96, ngroups=2, dtype=torch.bfloat16)
    a.update(kw)
    return m2.make_norm_dims(**a)


def conv_forward(d, **over):
    a = dict(x=OK, w=OK, b=None, init=None, lens=None, y0=OK, y1=OK, y2=OK, fin=None)
    a.update(over)
    return m2._lib.mamba2_conv1d_forward(ctypes.byref(d), *a.values(), 0)


def conv_backward(d, **over):
    a = dict(x=OK, w=OK, b=None, init=None, lens=None, dy0=OK, dy1=OK, dy2=OK, dfin=None, dx=OK,
             dw=OK, db=None, dinit=None, ws=OK, n=BIG)
    a.update(over)
    return m2._lib.mamba2_conv1d_backward(ctypes.byref(d), *a.values(), 0)


def conv_step(d, **over):
    a = dict(x=OK, w=OK, b=None, state=OK, y0=OK, y1=OK, y2=OK)
    a.update(over)
    return m2._lib.mamba2_conv1d_step(ctypes.byref(d), *a.values(), 0)


def scan_forward(d, **over):
    a = dict(u=OK, dt=OK, A=OK, B=OK, C=OK, D=None, z=None, bias=None, init=None, lens=None, y=OK,
             fin=None, ws=OK, n=BIG)
    a.update(over)
    return m2._lib.mamba2_selective_scan_forward(ctypes.byref(d), *a.values(), 0)


def scan_backward(d, **over):
    a = dict(u=OK, dt=OK, A=OK, B=OK, C=OK, D=None, z=None, bias=None, init=None, lens=None, dy=OK,
             dfin=None, du=OK, ddt=OK, dA=OK, dB=OK, dC=OK, dD=None, dz=None, dbias=None,
             dinit=None, ws=OK, n=BIG)
    a.update(over)
    return m2._lib.mamba2_selective_scan_backward(ctypes.byref(d), *a.values(), 0)


def scan_step(d, **over):
    a = dict(u=OK, dt=OK, A=OK, B=OK, C=OK, D=None, z=None, bias=None, state=OK, y=OK)
    a.update(over)
    return m2._lib.mamba2_selective_scan_step(ctypes.byref(d), *a.values(), 0)


def norm_forward(d, **over):
    a = dict(x=OK, z=None, w=OK, b=None, y=OK)
    a.update(over)
    return m2._lib.mamba2_norm_forward(ctypes.byref(d), *a.values(), 0)


def norm_backward(d, **over):
    a = dict(x=OK, z=None, w=OK, dy=OK, dx=OK, dz=None, dw=OK, db=None, ws=OK, n=BIG)
    a.update(over)
    return m2._lib.mamba2_norm_backward(ctypes.byref(d), *a.values(), 0)


def _refused(rc, status, word):
    assert rc == status, (rc, m2.mamba2_last_error())
    assert word in m2.mamba2_last_error()


@pytest.mark.parametrize("call,make,bytes_of", [
    (conv_forward, _conv, None), (conv_backward, _conv, "mamba2_conv1d_backward_workspace_bytes"),
    (scan_forward, _scan, "mamba2_selective_scan_workspace_bytes"),
    (scan_backward, _scan, "mamba2_selective_scan_backward_workspace_bytes"),
    (norm_forward, _norm, None),
    (norm_backward, _norm, "mamba2_norm_backward_workspace_bytes")])
def test_sizes_refused(call, make, bytes_of):
    def no(status, word, **kw):
        d = make(**kw)
        _refused(call(d, **({"x": None} if "x" in kw else {})), status, word)
        if bytes_of:
            assert getattr(m2, bytes_of)(d) == 0

    no(m2.MAMBA2_ERR_DTYPE, "dtype", dtype=7)
    no(m2.MAMBA2_ERR_SHAPE, "sizes", channels=0, **({"parts": (0,)} if make is _conv else {}))
    no(m2.MAMBA2_ERR_SHAPE, "sizes", **({"rows": 0} if make is _norm else {"seqlen": 0}))
    no(m2.MAMBA2_ERR_UNSUPPORTED, "", **({"rows": 1 << 31} if make is _norm else {"batch": 65536}))
    if make is not _conv:
        no(m2.MAMBA2_ERR_SHAPE, "multiple", ngroups=5)
        no(m2.MAMBA2_ERR_SHAPE, "sizes", ngroups=0)
        no(m2.MAMBA2_ERR_SHAPE, "z_stride", z_stride=95)
    if bytes_of:
        assert getattr(m2, bytes_of)(make()) >= 256
    assert call.__name__ and m2.mamba2_status_string(m2.MAMBA2_ERR_SHAPE)


def test_conv_sizes():
    no = _refused
    no(conv_forward(_conv(width=1)), m2.MAMBA2_ERR_UNSUPPORTED, "width")
    no(conv_forward(_conv(width=5)), m2.MAMBA2_ERR_UNSUPPORTED, "width")
    no(conv_forward(_conv(parts=(64, 16))), m2.MAMBA2_ERR_SHAPE, "parts")
    no(conv_forward(_conv(parts=(64, 0, 32))), m2.MAMBA2_ERR_SHAPE, "part[2]")
    no(conv_forward(_conv(parts=(64, 48, -16))), m2.MAMBA2_ERR_SHAPE, "part[2]")
    no(conv_forward(_conv(x_stride=95)), m2.MAMBA2_ERR_SHAPE, "x_stride")
    no(conv_backward(_conv(dx_stride=-1)), m2.MAMBA2_ERR_SHAPE, "dx_stride")
    no(conv_forward(_conv(x_stride=1 << 25)), m2.MAMBA2_ERR_UNSUPPORTED, "x_stride")
    no(conv_forward(_conv(batch=1, seqlen=1 << 30)), m2.MAMBA2_ERR_UNSUPPORTED, "large")
    no(conv_forward(_conv(batch=1, seqlen=(1 << 30) + 1)), m2.MAMBA2_ERR_UNSUPPORTED, "range")
    d = _conv()
    d.activation = 2
    no(conv_forward(d), m2.MAMBA2_ERR_UNSUPPORTED, "activation")
    with pytest.raises(m2.Mamba2Error, match="activation"):
        _conv(activation="relu")
    with pytest.raises(m2.Mamba2Error, match="parts"):
        _conv(parts=(24, 24, 24, 24))
    no(m2._lib.mamba2_conv1d_forward(None, *[OK] * 9, 0), m2.MAMBA2_ERR_NULL, "dims")


def test_scan_sizes():
    no = _refused
    no(scan_forward(_scan(dstate=0)), m2.MAMBA2_ERR_SHAPE, "dstate")
    no(scan_forward(_scan(dstate=65)), m2.MAMBA2_ERR_UNSUPPORTED, "dstate")
    no(scan_forward(_scan(b_stride=31)), m2.MAMBA2_ERR_SHAPE, "b_stride")
    no(scan_forward(_scan(c_stride=31)), m2.MAMBA2_ERR_SHAPE, "c_stride")
    for kw in (dict(batch=60000, seqlen=1, channels=1 << 20, ngroups=1),
               dict(batch=1, seqlen=1 << 29, channels=128, ngroups=1),
               dict(batch=1, seqlen=1 << 27, channels=4, ngroups=4)):
        no(scan_forward(_scan(**kw)), m2.MAMBA2_ERR_UNSUPPORTED, "large")
        no(scan_backward(_scan(**kw)), m2.MAMBA2_ERR_UNSUPPORTED, "large")
    no(scan_backward(_scan(dz_stride=95)), m2.MAMBA2_ERR_SHAPE, "dz_stride")
    d = _scan()
    d.softplus = 2
    no(scan_forward(d), m2.MAMBA2_ERR_SHAPE, "softplus")
    no(m2._lib.mamba2_selective_scan_forward(None, *[OK] * 13, BIG, 0), m2.MAMBA2_ERR_NULL, "dims")


def test_norm_sizes():
    no = _refused
    no(norm_forward(_norm(channels=8193, ngroups=1)), m2.MAMBA2_ERR_UNSUPPORTED, "8192")
    no(norm_forward(_norm(eps=-1e-5)), m2.MAMBA2_ERR_SHAPE, "eps")
    no(norm_forward(_norm(eps=float("nan"))), m2.MAMBA2_ERR_SHAPE, "eps")
    no(norm_forward(_norm(eps=float("inf"))), m2.MAMBA2_ERR_SHAPE, "eps")
    no(norm_forward(_norm(x_stride=95)), m2.MAMBA2_ERR_SHAPE, "x_stride")
    no(norm_backward(_norm(dz_stride=95)), m2.MAMBA2_ERR_SHAPE, "dz_stride")
    d = _norm()
    d.kind = 2
    no(norm_forward(d), m2.MAMBA2_ERR_UNSUPPORTED, "norm")
    d = _norm()
    d.reserved = 1
    no(norm_forward(d), m2.MAMBA2_ERR_SHAPE, "reserved")
    with pytest.raises(m2.Mamba2Error, match="norm"):
        _norm(kind="batch")


@pytest.mark.parametrize("call,dims,needed,optional", [
    (conv_forward, _conv(), "x w y0 y1 y2", "b init lens fin"),
    (conv_backward, _conv(), "x w dy0 dy1 dy2 dx dw", "b init lens dfin db dinit"),
    (conv_step, _conv(seqlen=1), "x w state y0 y1 y2", "b"),
    (scan_forward, _scan(), "u dt A B C y", "D z bias init lens fin"),
    (scan_backward, _scan(), "u dt A B C dy du ddt dA dB dC",
     "D z bias init lens dfin dD dbias dinit"),
    (scan_step, _scan(seqlen=1), "u dt A B C state y", "D z bias"),
    (norm_forward, _norm(), "x w y", "z b"),
    (norm_backward, _norm(), "x w dy dx dw", "db"),
])
def test_pointers_refused(call, dims, needed, optional):
    for name in needed.split():
        assert call(dims, **{name: None}) == m2.MAMBA2_ERR_NULL, name
        assert call(dims, **{name: OK + 4}) == m2.MAMBA2_ERR_ALIGN, name
    for name in optional.split():
        assert call(dims, **{name: OK + 8}) == m2.MAMBA2_ERR_ALIGN, name


def test_gate_gradient_is_required_with_a_gate():
    _refused(norm_backward(_norm(), z=OK), m2.MAMBA2_ERR_NULL, "dz")
    _refused(norm_backward(_norm(), z=OK, dz=OK + 2), m2.MAMBA2_ERR_ALIGN, "dz")
    _refused(scan_backward(_scan(), z=OK), m2.MAMBA2_ERR_NULL, "dz")
    _refused(scan_backward(_scan(), z=OK, dz=OK + 2), m2.MAMBA2_ERR_ALIGN, "dz")


@pytest.mark.parametrize("call,dims,bytes_of", [
    (conv_backward, _conv(), "mamba2_conv1d_backward_workspace_bytes"),
    (scan_forward, _scan(seqlen=4096), "mamba2_selective_scan_workspace_bytes"),
    (scan_backward, _scan(seqlen=4096), "mamba2_selective_scan_backward_workspace_bytes"),
    (norm_backward, _norm(), "mamba2_norm_backward_workspace_bytes")])
def test_workspace_refused(call, dims, bytes_of):
    n = getattr(m2, bytes_of)(dims)
    assert call(dims, ws=None) == m2.MAMBA2_ERR_WORKSPACE
    assert call(dims, ws=OK + 16) == m2.MAMBA2_ERR_WORKSPACE
    _refused(call(dims, n=n - 1), m2.MAMBA2_ERR_WORKSPACE, "needed")


def test_steps_take_one_token():
    _refused(conv_step(_conv(seqlen=2)), m2.MAMBA2_ERR_SHAPE, "seqlen")
    _refused(scan_step(_scan(seqlen=2)), m2.MAMBA2_ERR_SHAPE, "seqlen")


# ------------------------------------------------------------ tensors' checks


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _raises(status, word, fn, *a, **kw):
    with pytest.raises(m2.Mamba2Error) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value
    assert word in str(e.value)


def test_conv_tensors():
    x, w = _t(2, 10, 96), _t(96, 4, dtype=torch.float32)
    f = m2.conv1d_forward
    _raises(m2.MAMBA2_ERR_NULL, "GPU", f, x, w)
    _raises(m2.MAMBA2_ERR_DTYPE, "x", f, x.half(), w)
    _raises(m2.MAMBA2_ERR_DTYPE, "weight", f, x, w.bfloat16())
    _raises(m2.MAMBA2_ERR_SHAPE, "x", f, x[0], w)
    _raises(m2.MAMBA2_ERR_SHAPE, "weight", f, x, w[:95])
    _raises(m2.MAMBA2_ERR_SHAPE, "parts", f, x, w, parts=(64, 16))
    _raises(m2.MAMBA2_ERR_SHAPE, "gaps", f, x.transpose(1, 2).contiguous().transpose(1, 2), w)
    _raises(m2.MAMBA2_ERR_SHAPE, "steps", f, _t(2, 20, 96)[:, :10], w)
    _raises(m2.MAMBA2_ERR_SHAPE, "overlap", f, _t(1, 1, 96).expand(1, 10, 96), w)
    _raises(m2.MAMBA2_ERR_SHAPE, "init_state", f, x, w, None, _t(2, 4, 96))
    _raises(m2.MAMBA2_ERR_DTYPE, "init_state", f, x, w, None, _t(2, 3, 96, dtype=torch.float32))
    _raises(m2.MAMBA2_ERR_DTYPE, "lengths", f, x, w, lengths=torch.zeros(2, dtype=torch.int64))
    _raises(m2.MAMBA2_ERR_SHAPE, "lengths", f, x, w, lengths=torch.zeros(3, dtype=torch.int32))
    # a column range of wider rows passes the checks of strides
    _raises(m2.MAMBA2_ERR_NULL, "GPU", f, _t(2, 10, 200)[..., 8:104], w)
    b = m2.conv1d_backward
    _raises(m2.MAMBA2_ERR_SHAPE, "dy1", b, x, w, None, None, (_t(2, 10, 64), _t(2, 9, 32)))
    _raises(m2.MAMBA2_ERR_SHAPE, "parts", b, x, w, None, None, _t(2, 10, 64))
    _raises(m2.MAMBA2_ERR_DTYPE, "dfinal", b, x, w, None, None, x, _t(2, 3, 96).float())
    s = m2.conv1d_step
    _raises(m2.MAMBA2_ERR_NULL, "state", s, x[:, 0], w, None, None)
    _raises(m2.MAMBA2_ERR_SHAPE, "state", s, x[:, 0], w, None, _t(2, 2, 96))
    _raises(m2.MAMBA2_ERR_NULL, "GPU", s, x[:, 0], w, None, _t(2, 3, 96))


def _scan_tensors():
    f = torch.float32
    return dict(u=_t(2, 10, 96), dt=_t(2, 10, 96), A=_t(96, 16, dtype=f), B=_t(2, 10, 2, 16),
                C=_t(2, 10, 2, 16), D=_t(96, dtype=f), z=_t(2, 10, 96), dt_bias=_t(96, dtype=f),
                init_state=_t(2, 96, 16, dtype=f))


@pytest.mark.parametrize("name,value,status", [
    ("dt", _t(2, 10, 95), m2.MAMBA2_ERR_SHAPE), ("A", _t(96, 16), m2.MAMBA2_ERR_DTYPE),
    ("B", _t(2, 10, 2, 15), m2.MAMBA2_ERR_SHAPE), ("C", _t(2, 10, 4, 16), m2.MAMBA2_ERR_SHAPE),
    ("C", _t(2, 10, 2, 16).float(), m2.MAMBA2_ERR_DTYPE), ("D", _t(96), m2.MAMBA2_ERR_DTYPE),
    ("z", _t(2, 10, 96).float(), m2.MAMBA2_ERR_DTYPE), ("z", _t(2, 96, 10).mT, m2.MAMBA2_ERR_SHAPE),
    ("dt_bias", _t(95).float(), m2.MAMBA2_ERR_SHAPE), ("A", None, m2.MAMBA2_ERR_NULL),
    ("init_state", _t(2, 96, 16), m2.MAMBA2_ERR_DTYPE),
    ("u", _t(2, 10, 192)[..., :96], m2.MAMBA2_ERR_SHAPE)])
def test_scan_tensors(name, value, status):
    _raises(status, name, m2.selective_scan_forward, **(_scan_tensors() | {name: value}))


def test_scan_on_host_tensors():
    t = _scan_tensors()
    _raises(m2.MAMBA2_ERR_NULL, "GPU", m2.selective_scan_forward, **t)
    bc = _t(2, 10, 100)
    t["B"], t["C"] = bc[..., :32].unflatten(-1, (2, 16)), bc[..., 32:64].unflatten(-1, (2, 16))
    _raises(m2.MAMBA2_ERR_NULL, "GPU", m2.selective_scan_forward, **t)
    one = {k: (v[:, 0] if k in ("u", "dt", "B", "C", "z") else v) for k, v in _scan_tensors().items()}
    one["u"], one["dt"] = one["u"].contiguous(), one["dt"].contiguous()
    state = one.pop("init_state")
    _raises(m2.MAMBA2_ERR_NULL, "GPU", m2.selective_scan_step, **one, state=state)
    _raises(m2.MAMBA2_ERR_DTYPE, "state", m2.selective_scan_step, **one, state=state.bfloat16())


def test_norm_tensors():
    f = torch.float32
    x, w = _t(10, 96), _t(96, dtype=f)
    n = m2.norm_forward
    _raises(m2.MAMBA2_ERR_NULL, "GPU", n, x, w)
    _raises(m2.MAMBA2_ERR_NULL, "GPU", n, _t(2, 5, 200)[..., :96], w, None, _t(2, 5, 96))
    _raises(m2.MAMBA2_ERR_DTYPE, "x", n, x.half(), w)
    _raises(m2.MAMBA2_ERR_DTYPE, "weight", n, x, w.bfloat16())
    _raises(m2.MAMBA2_ERR_DTYPE, "z", n, x, w, None, x.float())
    _raises(m2.MAMBA2_ERR_SHAPE, "z", n, x, w, None, _t(9, 96))
    _raises(m2.MAMBA2_ERR_SHAPE, "bias", n, x, w, _t(95, dtype=f))
    _raises(m2.MAMBA2_ERR_SHAPE, "dy", m2.norm_backward, x, w, None, None, _t(96, 10).t())
    _raises(m2.MAMBA2_ERR_DTYPE, "dy", m2.norm_backward, x, w, None, None, x.float())
    _raises(m2.MAMBA2_ERR_SHAPE, "x", n, _t(96), w)


def test_short_functions_refuse_what_is_missing():
    u, A, B, w = torch.zeros(2, 8, 4), torch.zeros(4, 3), torch.zeros(2, 8, 1, 3), torch.zeros(4)
    calls = [
        lambda: m2.conv1d_forward(None, torch.zeros(4, 4)),
        lambda: m2.conv1d_forward(u, None),
        lambda: m2.conv1d_backward(u, torch.zeros(4, 4), None, None, None),
        lambda: m2.conv1d_backward(u, torch.zeros(4, 4), None, None, (u, None)),
        lambda: m2.conv1d_step(u[:, 0], None, None, torch.zeros(2, 3, 4)),
        lambda: m2.selective_scan_forward(None, u, A, B, B),
        lambda: m2.selective_scan_forward(u, u, None, B, B),
        lambda: m2.selective_scan_backward(u, u, A, B, B, None, None, None, None, None),
        lambda: m2.norm_forward(u, None),
        lambda: m2.norm_backward(u, None, None, None, u),
        lambda: m2.norm_backward(u, w, None, None, None),
    ]
    for call in calls:
        with pytest.raises(m2.Mamba2Error) as e:
            call()
        assert e.value.status == m2.MAMBA2_ERR_NULL


@pytest.mark.parametrize("z", [(4,), (8, 4), (2, 2, 8, 4), (1, 8, 4)])
def test_gate_of_another_shape(z):
    u, A, B = torch.zeros(2, 8, 4), torch.zeros(4, 3), torch.zeros(2, 8, 1, 3)
    for call in (lambda: m2.selective_scan_forward(u, u, A, B, B, z=torch.zeros(z)),
                 lambda: m2.selective_scan_backward(u, u, A, B, B, None, torch.zeros(z), None,
                                                    None, u)):
        with pytest.raises(m2.Mamba2Error) as e:
            call()
        assert e.value.status == m2.MAMBA2_ERR_SHAPE

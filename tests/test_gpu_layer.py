"""The operators around the SSD (conv1d, selective_scan, norm) against plain
float64 forms, element by element, within bounds that count the roundings
(layer_reference)."""
import itertools

import pytest
import torch

import layer_reference as ref
from gpu_helpers import say
from layer_reference import F, U, half_step, to64, within

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def m2():
    import state_space_sequence_02_amd as lib
    return lib


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g)


def _wide(t, extra, fill=float("nan")):
    """t on the GPU as the first columns of rows with ``extra`` more, which hold ``fill``."""
    if not extra:
        return t.cuda()
    rows = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), fill, dtype=t.dtype)
    rows[..., :t.shape[-1]] = t
    return rows.cuda()[..., :t.shape[-1]]


def _cuda(t):
    return None if t is None else t.cuda()


def _token(v, i):
    """Token i of every sequence: a view, or a copy where that is not 16-byte aligned."""
    t = v[:, i]
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _behind(t, lengths, value=float("nan")):
    """t with ``value`` behind every sequence's length."""
    t = t.clone()
    if lengths is not None:
        for i, m in enumerate(ref.lengths_of(lengths, t.shape[0], t.shape[1])):
            t[i, m:] = value
    return t


def _lengths(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()


# ---------------------------------------------------------------------- conv1d

CONV = [
    # dtype, batch, tokens, parts, width, extra columns, act, bias, init, lengths
    ("bf16", 2, 77, (128, 32, 32), 4, 0, True, True, True, None),
    ("bf16", 2, 77, (128, 32, 32), 4, 40, True, True, False, None),   # rows of 16-byte steps
    ("bf16", 2, 40, (64, 16, 16), 4, 3, True, True, True, None),      # rows that are not
    ("bf16", 1, 300, (520,), 3, 8, False, False, True, None),
    ("bf16", 3, 45, (24, 3), 2, 0, True, True, True, [45, 0, 17]),    # scalar: a part of 3
    ("f32", 2, 130, (64, 4, 4), 4, 12, True, True, True, [130, 129]),
    ("f32", 3, 33, (37,), 4, 0, True, False, True, [1, 2, 33]),
    ("f32", 4, 9, (5, 1, 1), 3, 1, False, True, True, [0, 1, 2, 9]),
    ("f32", 1, 1, (1,), 2, 0, True, True, True, None),
    ("bf16", 2, 1, (64,), 4, 0, True, True, True, None),
    ("bf16", 2, 2, (64,), 4, 0, True, True, True, [0, 2]),
    ("bf16", 1, 3, (72,), 4, 0, True, True, False, None),
    ("f32", 2, 31, (8,), 4, 0, True, True, True, [-5, 900]),          # clamped to 0 and 31
    ("bf16", 1, 4100, (8,), 4, 0, True, True, True, None),            # many tiles
    ("bf16", 2, 100, (20, 12, 4), 4, 4, True, True, True, [100, 61]),  # rows of 8-byte steps
    ("bf16", 3, 700, (260, 64, 64), 2, 0, True, True, False, None),
]


def _conv_case(case, seed=3):
    dtype, b, n, parts, w, extra, act, bias, init, lengths = case
    io, c = TYPES[dtype], sum(case[3])
    r = _gen(seed)
    x = r(b, n, c).to(io)
    wt = r(c, w) / w ** 0.5
    bs = 0.1 * r(c) if bias else None
    h0 = r(b, w - 1, c).to(io) if init else None
    dys = [r(b, n, p).to(io) for p in parts]
    dfin = r(b, w - 1, c).to(io)
    return x, wt, bs, h0, dys, dfin


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_conv_forward(m2, case):
    say(f"conv forward {case}")
    dtype, b, n, parts, w, extra, act, bias, init, lengths = case
    x, wt, bs, h0, _, _ = _conv_case(case)
    ys, fin = m2.conv1d_forward(_wide(_behind(x, lengths), extra), wt.cuda(), _cuda(bs), _cuda(h0),
                                parts=parts, activation="silu" if act else "none",
                                lengths=_lengths(lengths))
    torch.cuda.synchronize()
    a = (to64(x), to64(wt), to64(bs), to64(h0))
    want, wfin = ref.conv(*a, lengths, act)
    bound = ref.conv_bound(*a, lengths, act, TYPES[dtype])
    assert [tuple(y.shape) for y in ys] == [(b, n, p) for p in parts]
    within("y", torch.cat([y.cpu() for y in ys], -1), want, bound)
    assert torch.equal(fin.cpu().to(F), wfin)


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_conv_backward(m2, case):
    """Bounds: the gradient of the sizes (every factor by its size, and silu's
    slope and curvature by 1.1 and 0.5) times the roundings on the way: W + 2
    of the recomputed sum (through silu's curvature), 3 |p| + 20 of the slope
    and the products, W + 1 of dx's sum; for the weights' sums a tree of at
    most 32 + 4 + B * tiles terms."""
    say(f"conv backward {case}")
    dtype, b, n, parts, w, extra, act, bias, init, lengths = case
    io = TYPES[dtype]
    x, wt, bs, h0, dys, dfin = _conv_case(case)
    got = m2.conv1d_backward(_wide(_behind(x, lengths), extra), wt.cuda(), _cuda(bs), _cuda(h0),
                             tuple(_behind(d, lengths).cuda() for d in dys), dfin.cuda(),
                             activation="silu" if act else "none", lengths=_lengths(lengths))
    torch.cuda.synchronize()
    a = [to64(x), to64(wt), to64(bs), to64(h0) if init else torch.zeros(b, w - 1, sum(parts), dtype=F)]
    dy, df = torch.cat([to64(d) for d in dys], -1), to64(dfin)
    want = ref.grads(lambda *v: ref.conv(*v, lengths, act), a, (dy, df))
    # sizes: g's, through the convolution without activation
    sizes = [None if v is None else v.abs() for v in a]
    p, _ = ref.conv(*a, lengths, False)
    ps, _ = ref.conv(*sizes, lengths, False)
    slope = 1.1 if act else 1.0
    eg = dy.abs() * (0.5 * (w + 2) * U * ps + slope * (3 * p.abs() + 20) * U) if act \
        else dy.abs() * 2 * U
    big = ref.grads(lambda *v: ref.conv(*v, lengths, False), sizes, (slope * dy.abs(), df.abs()))
    off = ref.grads(lambda *v: ref.conv(*v, lengths, False), sizes, (eg, 0 * df))
    terms = 36 + b * -(-n // 128)
    for name, i in (("dx", 0), ("dweight", 1), ("dbias", 2), ("dinit", 3)):
        if a[i] is None:
            assert got[name] is None
            continue
        count = w + 2 if name in ("dx", "dinit") else terms
        e = off[i] + count * U * big[i]
        if name in ("dx", "dinit"):
            e = e + half_step(io) * (want[i].abs() + e)
        within(name, got[name], want[i], e)


def test_conv_without_bias_initial_state_or_parts(m2):
    r = _gen(8)
    x, wt = r(2, 50, 64), r(64, 4) / 2
    y, fin = m2.conv1d_forward(x.cuda(), wt.cuda())
    a = (to64(x), to64(wt), None, None)
    within("y", y, ref.conv(*a)[0], ref.conv_bound(*a, None, True, torch.float32))
    got = m2.conv1d_backward(x.cuda(), wt.cuda(), None, None, x.cuda())
    assert got["dbias"] is None and got["dx"].shape == x.shape


@pytest.mark.parametrize("dtype,parts,w,extra", [
    ("bf16", (128, 16, 16), 4, 32), ("bf16", (64, 3), 3, 0), ("f32", (33,), 2, 1),
    ("f32", (64, 8, 8), 4, 0)])
def test_conv_steps_are_the_convolution(m2, dtype, parts, w, extra):
    """Steps from a state give the prompt's outputs and its final state, exactly
    (the same float32 sums in the same order)."""
    r = _gen(5)
    b, n, c = 5, 7, sum(parts)
    x = _wide(r(b, n, c).to(TYPES[dtype]), extra)
    wt, bs = r(c, w).cuda(), r(c).cuda()
    h0 = r(b, w - 1, c).to(TYPES[dtype]).cuda()
    ys, fin = m2.conv1d_forward(x, wt, bs, h0, parts=parts)
    state = h0.clone()
    for t in range(n):
        one = m2.conv1d_step(_token(x, t), wt, bs, state, parts=parts)
        for p, q in zip(one, ys):
            assert torch.equal(p, q[:, t])
    assert torch.equal(state, fin)


def test_conv_final_state_over_the_initial_one(m2):
    r = _gen(6)
    for n, c in ((2, 64), (70, 64), (40, 7)):
        x, wt, h0 = r(3, n, c).cuda(), r(c, 4).cuda(), r(3, 3, c).cuda()
        y, fin = m2.conv1d_forward(x, wt, None, h0)
        buf, y2 = h0.clone(), torch.empty_like(y)
        dims = m2.make_conv_dims(3, n, c, 4, None, torch.float32)
        m2.mamba2_conv1d_forward(dims, x, wt, None, buf, None, y2, None, None, buf)
        assert torch.equal(buf, fin) and torch.equal(y, y2)


def test_conv_gradient_into_wider_rows(m2):
    """dx as a column range of a wider gradient: the other columns stay."""
    r = _gen(7)
    for c, lo, width in ((64, 32, 128), (30, 8, 51)):
        x, wt = r(2, 45, c).cuda(), r(c, 4).cuda()
        dy = r(2, 45, c).cuda()
        want = m2.conv1d_backward(x, wt, None, None, dy)
        rows = torch.full((2, 45, width), 7.0, device="cuda")
        dims = m2.make_conv_dims(2, 45, c, 4, None, torch.float32, dx_stride=width)
        n = m2.mamba2_conv1d_backward_workspace_bytes(dims)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dw = torch.empty_like(wt)
        m2.mamba2_conv1d_backward(dims, x, wt, None, None, None, dy, None, None, None,
                                  rows[..., lo:lo + c], dw, None, None, ws, n)
        assert torch.equal(rows[..., lo:lo + c], want["dx"]) and torch.equal(dw, want["dweight"])
        assert (rows[..., :lo] == 7).all() and (rows[..., lo + c:] == 7).all()


# --------------------------------------------------------------- selective scan

SCAN = [
    # dtype, batch, tokens, channels, states, groups, gate, D, bias, init, lengths, softplus, extra
    ("bf16", 2, 40, 128, 16, 1, True, True, True, True, None, True, 64),
    ("bf16", 1, 333, 64, 16, 1, True, True, True, False, None, True, 0),    # several chunks
    ("f32", 2, 300, 70, 16, 1, False, True, True, True, [300, 100], True, 0),
    ("f32", 3, 100, 198, 7, 2, True, True, True, True, [100, 0, 37], True, 3),
    ("f32", 2, 17, 65, 1, 1, False, False, False, True, None, True, 0),
    ("f32", 1, 16, 63, 3, 1, True, False, True, True, None, True, 1),
    ("f32", 2, 15, 12, 4, 3, False, True, False, False, None, True, 0),
    ("bf16", 2, 70, 64, 8, 1, True, True, True, True, None, True, 24),
    ("bf16", 1, 130, 96, 17, 1, True, True, True, True, None, True, 5),
    ("f32", 1, 150, 80, 32, 4, True, True, True, True, [149], True, 8),
    ("bf16", 1, 90, 64, 40, 1, False, True, True, True, None, True, 0),
    ("f32", 2, 200, 66, 64, 2, True, True, True, True, [-1, 500], True, 0),
    ("bf16", 3, 1, 64, 16, 1, True, True, True, True, [1, 0, 1], True, 0),
    ("f32", 1, 1, 1, 1, 1, False, False, False, False, None, False, 0),
    ("f32", 2, 50, 64, 16, 1, True, True, True, True, None, False, 0),
    ("f32", 4, 2100, 8, 16, 1, False, True, True, True, [2100, 64, 65, 1999], True, 0),
    ("bf16", 2, 1100, 160, 24, 1, True, True, True, True, None, True, 40),
    ("f32", 1, 129, 64, 64, 1, True, True, True, True, None, True, 0),
    ("bf16", 66, 140, 500, 4, 1, True, True, True, True, None, True, 0),   # one pass, long enough to cut
]


def _scan_case(case, seed=11):
    dtype, b, n, ch, ns, g, gate, D, bias, init, lengths, sp, extra = case
    io = TYPES[dtype]
    r = _gen(seed)
    t = {}
    t["u"] = ref.silu(r(b, n, ch)).to(io)
    t["dt"] = (0.5 * r(b, n, ch)).to(io) if sp else (0.05 * r(b, n, ch).abs()).to(io)
    t["A"] = -torch.arange(1, ns + 1) * torch.exp(0.2 * r(ch, ns))
    t["B"], t["C"] = r(b, n, g, ns).to(io), r(b, n, g, ns).to(io)
    t["D"] = r(ch) if D else None
    t["z"] = r(b, n, ch).to(io) if gate else None
    dt0 = torch.exp(-6.9 + 4.6 * torch.rand(ch, generator=torch.Generator().manual_seed(seed)))
    t["dt_bias"] = (dt0 + torch.log(-torch.expm1(-dt0)) if sp else 0.01 * dt0) if bias else None
    t["init"] = r(b, ch, ns) if init else None
    t["dy"] = r(b, n, ch).to(io)
    t["dfinal"] = r(b, ch, ns)
    return t


def _scan_gpu(t, case):
    """The case's tensors on the GPU: NaN behind the lengths, z, B and C in wider rows."""
    g, ns, lengths, extra = case[5], case[4], case[10], case[12]
    k = {n: _cuda(_behind(t[n], lengths)) for n in ("u", "dt")}
    k |= {n: _cuda(t[n]) for n in ("A", "D", "dt_bias")}
    k["z"] = None if t["z"] is None else _wide(_behind(t["z"], lengths), extra)
    for n in ("B", "C"):
        k[n] = _wide(_behind(t[n], lengths).flatten(2), extra).unflatten(-1, (g, ns))
    return k


def _scan64(t):
    return [to64(t[k]) for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "init")]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_scan_forward(m2, case):
    say(f"scan forward {case}")
    lengths, sp = case[10], case[11]
    t = _scan_case(case)
    k = _scan_gpu(t, case)
    y, fin = m2.selective_scan_forward(**k, init_state=_cuda(t["init"]), softplus=sp,
                                       lengths=_lengths(lengths))
    torch.cuda.synchronize()
    a = _scan64(t)
    want, wfin = ref.scan(*a, lengths, sp)
    by, bf = ref.scan_bounds(*a, lengths, sp, TYPES[case[0]])
    within("y", y, want, by)
    within("final", fin, wfin, bf)


@pytest.mark.parametrize("case", [SCAN[0], SCAN[3], SCAN[6], SCAN[7], SCAN[8], SCAN[9], SCAN[11],
                                  SCAN[13], SCAN[14]],
                         ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_scan_steps_are_the_scan(m2, case):
    say(f"scan steps {case}")
    sp = case[11]
    case = case[:2] + (min(case[2], 6),) + case[3:10] + (None,) + case[11:]
    t = _scan_case(case)
    if t["init"] is None:
        t["init"] = torch.zeros(case[1], case[3], case[4])
    k = _scan_gpu(t, case)
    state = t["init"].cuda()
    ys = []
    for i in range(case[2]):
        one = {n: (None if v is None else v if n in ("A", "D", "dt_bias") else
                   _token(v, i).contiguous() if n in ("u", "dt") else _token(v, i))
               for n, v in k.items()}
        ys.append(m2.selective_scan_step(**one, state=state, softplus=sp))
    torch.cuda.synchronize()
    a = _scan64(t)
    want, wfin = ref.scan(*a, None, sp)
    by, bf = ref.scan_bounds(*a, None, sp, TYPES[case[0]])
    within("y", torch.stack(ys, 1), want, by)
    within("state", state, wfin, bf)


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_scan_backward(m2, case):
    """Bounds: the gradient of the sizes (every factor by its size, sums of sizes
    for sums), which the roundings of all that goes into an element multiply.
    A decay's relative error (scan_bounds) is at most 40 U at these inputs
    where the decay itself is not negligible, and a state or gradient of a
    state that has run over m tokens holds at most m of them; each of a
    token's own factors adds at most 60 U.  With decays of at most exp(-|d A|)
    what lies further back than the length of a sequence does not exist:
    m <= L, and what is carried forward and backward meets in dA and ddt: 2 L."""
    say(f"scan backward {case}")
    dtype, b, n, ch, ns, g, gate, D, bias, init, lengths, sp, extra = case
    io = TYPES[dtype]
    t = _scan_case(case)
    k = _scan_gpu(t, case)
    got = m2.selective_scan_backward(**k, init_state=_cuda(t["init"]),
                                     dy=_behind(t["dy"], lengths).cuda(),
                                     dfinal=t["dfinal"].cuda(), softplus=sp,
                                     lengths=_lengths(lengths))
    torch.cuda.synchronize()
    a = _scan64(t)
    if a[8] is None:
        a[8] = torch.zeros(b, ch, ns, dtype=F)
    dy, df = to64(t["dy"]), to64(t["dfinal"])
    want = ref.grads(lambda *v: ref.scan(*v, lengths, sp), a, (dy, df))
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")
    sizes = ref.scan_gradient_sizes(*a, lengths, sp, dy, df)
    most = max(ref.lengths_of(lengths, b, n))
    for name, w, size in zip(names, want, sizes):
        if w is None:
            assert got[name] is None, name
            continue
        e = (2 * 40 * most + 60 + (b * n + 64 if name in ("dA", "dD", "ddt_bias") else 0)) * U * size
        if name not in ("dA", "dD", "ddt_bias", "dinit"):
            e = e + half_step(io) * (w.abs() + e)
        within(name, got[name], w, e)


def test_scan_gate_gradient_into_wider_rows(m2):
    case = SCAN[3]
    t = _scan_case(case)
    k = _scan_gpu(t, case)
    b, n, ch, ns, g = case[1:6]
    lens, dy = _lengths(case[10]), t["dy"].cuda()
    want = m2.selective_scan_backward(**k, init_state=None, dy=dy, lengths=lens)
    wide = torch.full((b, n, 2 * ch + 3), 7.0, device="cuda")
    dims = m2.make_scan_dims(b, n, ch, ns, g, torch.float32, z_stride=k["z"].stride(1),
                             b_stride=k["B"].stride(1), c_stride=k["C"].stride(1),
                             dz_stride=2 * ch + 3)
    size = m2.mamba2_selective_scan_backward_workspace_bytes(dims)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    o = {q: torch.empty_like(v) for q, v in want.items()}
    m2.mamba2_selective_scan_backward(dims, k["u"], k["dt"], k["A"], k["B"], k["C"], k["D"], k["z"],
                                      k["dt_bias"], None, lens, dy, None, o["du"], o["ddt"],
                                      o["dA"], o["dB"], o["dC"], None, wide[..., :ch], None, None,
                                      ws, size)
    assert torch.equal(wide[..., :ch], want["dz"]) and (wide[..., ch:] == 7).all()
    for q in ("du", "ddt", "dA", "dB", "dC"):
        assert torch.equal(o[q], want[q]), q


def test_scan_final_state_over_the_initial_one(m2):
    for case in (SCAN[0], SCAN[2]):  # one chunk, several
        t = _scan_case(case)
        k = _scan_gpu(t, case)
        lens = _lengths(case[10])
        h0 = t["init"].cuda()
        y, fin = m2.selective_scan_forward(**k, init_state=h0, lengths=lens)
        buf, y2 = h0.clone(), torch.empty_like(y)
        dims = m2.make_scan_dims(case[1], case[2], case[3], case[4], case[5], TYPES[case[0]],
                                 z_stride=0 if k["z"] is None else k["z"].stride(1),
                                 b_stride=k["B"].stride(1), c_stride=k["C"].stride(1))
        n = m2.mamba2_selective_scan_workspace_bytes(dims)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        m2.mamba2_selective_scan_forward(dims, k["u"], k["dt"], k["A"], k["B"], k["C"], k["D"],
                                         k["z"], k["dt_bias"], buf, lens, y2, buf, ws, n)
        assert torch.equal(buf, fin) and torch.equal(y, y2)


def test_scan_small_time_steps_keep_their_digits(m2):
    """softplus far below zero: time steps of 1e-6 to 1e-3, where 1 + exp(dt)
    has lost them, to 1e-5 relative (the bound's (3 |raw| + 10) U is 4e-6)."""
    dt = torch.linspace(-14, -7, 64).view(1, 1, 64)
    one = torch.ones(1, 1, 64)
    A = torch.zeros(64, 1)
    BC = torch.ones(1, 1, 1, 1)
    _, fin = m2.selective_scan_forward(one.cuda(), dt.cuda(), A.cuda(), BC.cuda(), BC.cuda())
    want = ref.softplus(dt.to(F)).flatten()
    within("time step", fin.flatten(), want, 1e-5 * want)


def test_scan_masked_time_steps(m2):
    """dt of -inf and of the type's lowest value give time steps of zero: the
    state stays what it is; large ones are taken as they are."""
    for low in (float("-inf"), torch.finfo(torch.bfloat16).min):
        dt = torch.full((1, 5, 64), low)
        dt[0, 2] = 30.0
        r = _gen(2)
        u, B = r(1, 5, 64), r(1, 5, 1, 16)
        A = -torch.rand(64, 16) - 0.01
        h0 = r(1, 64, 16)
        _, fin = m2.selective_scan_forward(u.cuda(), dt.cuda(), A.cuda(), B.cuda(), B.cuda(),
                                           init_state=h0.cuda())
        want = torch.exp(30 * A.to(F)) * h0[0].to(F) + 30 * u[0, 2, :, None].to(F) * B[0, 2].to(F)
        within("state", fin[0], want, 64 * U * want.abs() + 200 * U * h0[0].abs().to(F))


# ------------------------------------------------------------------------ norm

NORM = [
    # dtype, rows, channels, groups, kind, gate, bias, eps, extra, shift
    ("bf16", 37, 2048, 1, "rms", True, False, 1e-5, 512, 0),
    ("bf16", 300, 1536, 8, "rms", True, False, 1e-5, 24, 0),
    ("bf16", 5, 512, 1, "layer", False, True, 1e-5, 0, 0),
    ("bf16", 9, 520, 1, "layer", True, True, 1e-6, 7, 0),          # rows of odd steps
    ("bf16", 3, 4096, 1, "rms", False, False, 1e-5, 0, 0),
    ("bf16", 2, 8192, 1, "layer", True, True, 1e-5, 0, 0),
    ("bf16", 11, 200, 1, "rms", True, True, 1e-5, 0, 0),
    ("f32", 1003, 1001, 1, "layer", False, True, 1e-5, 0, 0),
    ("f32", 3, 8191, 1, "layer", True, True, 1e-5, 0, 0),
    ("f32", 2, 8192, 1, "rms", True, False, 1e-5, 4, 0),
    ("f32", 50, 96, 3, "rms", True, True, 1e-5, 3, 0),
    ("f32", 6, 30, 6, "layer", False, False, 1e-5, 0, 0),
    ("f32", 1, 1, 1, "layer", False, True, 1e-5, 0, 0),
    ("f32", 4, 7, 7, "rms", True, False, 1e-5, 0, 0),
    ("f32", 20, 256, 1, "layer", False, True, 1e-5, 0, 30),        # a large mean
    ("f32", 4, 512, 1, "rms", False, False, 0.0, 0, 0),
    ("f32", 2, 3000, 1, "layer", True, True, 1e-5, 0, 0),
    ("f32", 2, 130, 1, "layer", True, True, 1e-5, 0, 0),
    ("bf16", 2, 1000, 2, "layer", True, True, 1e-5, 1, 0),
]


def _norm_case(case, seed=21):
    dtype, rows, ch, g, kind, gate, bias, eps, extra, shift = case
    io = TYPES[dtype]
    r = _gen(seed)
    x = (r(rows, ch) + shift).to(io)
    z = r(rows, ch).to(io) if gate else None
    return x, 1 + 0.2 * r(ch), 0.1 * r(ch) if bias else None, z, r(rows, ch).to(io)


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_norm_forward(m2, case):
    say(f"norm forward {case}")
    dtype, rows, ch, g, kind, gate, bias, eps, extra, _ = case
    x, w, b, z, _ = _norm_case(case)
    y = m2.norm_forward(_wide(x, extra), w.cuda(), _cuda(b), None if z is None else _wide(z, extra),
                        ngroups=g, kind=kind, eps=eps)
    torch.cuda.synchronize()
    a = (to64(x), to64(w), to64(b), to64(z), g, kind, eps)
    within("y", y, ref.norm(*a), ref.norm_bound(*a, TYPES[dtype]))


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_norm_backward(m2, case):
    """Bounds: with d = dy w, dv = rstd (d - mean(d) - xh mean(d xh)) is off by
    rstd times [n + 4 roundings of the means' terms, and xh's error in each of
    its two places] plus rstd's own relative error; dx and dz add the gate's
    (3 |z| + 24) U.  dweight sums dy xh over the rows in at most
    rows + 12 additions."""
    say(f"norm backward {case}")
    dtype, rows, ch, g, kind, gate, bias, eps, extra, _ = case
    io = TYPES[dtype]
    x, w, b, z, dy = _norm_case(case)
    got = m2.norm_backward(_wide(x, extra), w.cuda(), _cuda(b),
                           None if z is None else _wide(z, extra), dy.cuda(), ngroups=g, kind=kind,
                           eps=eps)
    torch.cuda.synchronize()
    x, w, b, z, dy = (to64(v) for v in (x, w, b, z, dy))
    want = ref.grads(lambda *v: ref.norm(*v, g, kind, eps), (x, w, b, z), (dy,))
    xh, e, rstd, er = ref.norm_terms(x, z, g, kind, eps)
    n = ch // g
    d = (dy * w).view(xh.shape).abs()
    mean = (lambda v: v.mean(-1, keepdim=True))
    sizes = d + (mean(d) if kind == "layer" else 0) + xh.abs() * mean(d * xh.abs())
    off = (n + 4) * U * sizes + e * mean(d * xh.abs()) + xh.abs() * mean(d * e)
    edv = (rstd * (off + (er + 4 * U) * sizes)).view(x.shape)
    big = (rstd * sizes).view(x.shape)

    def out(name, want, err):
        within(name, got[name], want, err + half_step(io) * (want.abs() + err))

    if z is None:
        assert got["dz"] is None
        out("dx", want[0], edv)
    else:
        gate_off = (3 * z.abs() + 24) * U
        out("dx", want[0], (edv + gate_off * big) * ref.silu(z).abs() + 0 * x)
        slope = 1.1 * torch.ones_like(z)
        out("dz", want[3], (edv + gate_off * big) * x.abs() * slope)
    xhf, ef = xh.reshape(x.shape), e.reshape(x.shape)
    within("dweight", got["dweight"], want[1],
           (dy.abs() * ef).sum(0) + (rows + 12) * U * (dy * xhf).abs().sum(0))
    if b is None:
        assert got["dbias"] is None
    else:
        within("dbias", got["dbias"], want[2], (rows + 12) * U * dy.abs().sum(0))


def test_norm_of_more_axes(m2):
    r = _gen(4)
    x, z, w, dy = r(3, 5, 64).cuda(), r(3, 5, 100).cuda()[..., :64], r(64).cuda(), r(3, 5, 64).cuda()
    y = m2.norm_forward(x, w, None, z)
    assert torch.equal(y.view(15, 64), m2.norm_forward(x.view(15, 64), w, None, z.reshape(15, 64)))
    g = m2.norm_backward(x, w, None, z, dy)
    assert g["dx"].shape == x.shape and g["dz"].shape == z.shape


def test_norm_gate_gradient_into_wider_rows(m2):
    r = _gen(9)
    for rows, ch, width in ((33, 64, 128), (8, 50, 99)):
        x, z, w, dy = (r(rows, ch).cuda() for _ in range(4))
        w = w[0].contiguous()
        want = m2.norm_backward(x, w, None, z, dy)
        wide = torch.full((rows, width), 7.0, device="cuda")
        dims = m2.make_norm_dims(rows, ch, 1, torch.float32, dz_stride=width)
        n = m2.mamba2_norm_backward_workspace_bytes(dims)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        m2.mamba2_norm_backward(dims, x, z, w, dy, dx, wide[:, :ch], dw, None, ws, n)
        assert torch.equal(wide[:, :ch], want["dz"]) and torch.equal(dx, want["dx"])
        assert (wide[:, ch:] == 7).all()


def test_norm_rows_of_zeros(m2):
    """A row of zeros (a padded token's) has a finite norm and gradient with eps > 0."""
    x = torch.zeros(4, 64, device="cuda")
    w, dy = torch.ones(64, device="cuda"), torch.ones(4, 64, device="cuda")
    for kind in ("rms", "layer"):
        assert (m2.norm_forward(x, w, kind=kind) == 0).all()
        g = m2.norm_backward(x, w, None, None, dy, kind=kind)
        assert torch.isfinite(g["dx"]).all() and (g["dweight"] == 0).all()

"""The forms of the kernels around the SSD that only larger problems reach,
element by element against float64: longer tiles of the convolution, teams of
the norm that walk several rows, the step that takes two sequences per
thread, long sequences of the scan.  A comment at each case says what reaches
the form; the bounds are those of layer_reference and layer_bounds."""
import pytest
import torch

import layer_reference as ref
from gpu_helpers import say
from layer_bounds import conv_gradients, norm_gradients, scan_gradients
from layer_reference import F, half_step, to64, within

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")


@pytest.fixture(scope="module")
def m2():
    import state_space_sequence_02_amd as lib
    return lib


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g)


def _cuda(t):
    return None if t is None else t.cuda()


def _wide(t, extra):
    if not extra:
        return t.cuda()
    rows = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), NAN, dtype=t.dtype)
    rows[..., :t.shape[-1]] = t
    return rows.cuda()[..., :t.shape[-1]]


def _behind(t, lengths):
    t = t.clone()
    if lengths is not None:
        for i, m in enumerate(lengths):
            t[i, m:] = NAN
    return t


def _lengths(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()


def _id(case):
    return "-".join(map(str, case)).replace(" ", "")


# ---------------------------------------------------------------------- conv1d

# Tiles of 32 tokens from 2^17 threads on: batch * channels / 4 (or channels) * tiles.
CONV_FORWARD = [
    # dtype, batch, tokens, parts, width, extra, act, init, lengths
    ("f32", 2, 4165, (1024, 16, 1024), 4, 0, True, True, [4165, 1000]),
    ("bf16", 3, 2800, (2048, 64, 64), 4, 8, True, False, None),
    ("bf16", 2, 4100, (500, 7, 8), 4, 3, True, True, [33, 4100]),        # one element per thread
    ("f32", 2, 4101, (515,), 3, 0, False, True, None),
    ("bf16", 1, 8200, (2080,), 2, 0, True, True, [8197]),
]
# Tiles of 16 and 32 tokens where they give 2048 wavefronts or more.
CONV_BACKWARD = [
    ("f32", 4, 4200, (65,), 4, 0, True, True, None),                     # 16, one element
    ("f32", 4, 4200, (130, 126, 4), 4, 4, True, True, [4200, 4199, 0, 77]),   # 16, vectors
    ("bf16", 4, 4200, (256, 4), 3, 8, False, True, [17, 4200, 31, 32]),  # 16, vectors
    ("f32", 4, 8200, (65,), 4, 0, True, False, [8200, 8193, 1, 100]),    # 32, one element
    ("bf16", 4, 8230, (130, 126, 4), 4, 4, True, True, None),            # 32, vectors
    ("f32", 5, 6600, (256, 4), 2, 0, True, True, [6600, 6599, 6593, 33, 2]),  # 32, vectors
]


def _conv(case, seed=3):
    dtype, b, n, parts, w, extra, act, init, lengths = case
    io, c = TYPES[dtype], sum(parts)
    r = _gen(seed)
    return (r(b, n, c).to(io), r(c, w) / w ** 0.5, 0.1 * r(c),
            r(b, w - 1, c).to(io) if init else None, [r(b, n, p).to(io) for p in parts],
            r(b, w - 1, c).to(io))


@pytest.mark.parametrize("case", CONV_FORWARD, ids=_id)
def test_conv_forward_in_long_tiles(m2, case):
    say(f"conv forward {case}")
    dtype, b, n, parts, w, extra, act, init, lengths = case
    x, wt, bias, h0, _, _ = _conv(case)
    threads = b * (sum(parts) // (1 if any(p % 4 for p in parts) or extra % 4 else 4))
    assert threads * -(-n // 32) >= 1 << 17
    ys, fin = m2.conv1d_forward(_wide(_behind(x, lengths), extra), wt.cuda(), bias.cuda(),
                                _cuda(h0), parts=parts, activation="silu" if act else "none",
                                lengths=_lengths(lengths))
    a = (to64(x), to64(wt), to64(bias), to64(h0))
    want, wfin = ref.conv(*a, lengths, act)
    within("y", torch.cat([y.cpu() for y in ys], -1), want,
           ref.conv_bound(*a, lengths, act, TYPES[dtype]))
    assert torch.equal(fin.cpu().to(F), wfin)


@pytest.mark.parametrize("case", CONV_BACKWARD, ids=_id)
def test_conv_backward_in_long_tiles(m2, case):
    say(f"conv backward {case}")
    dtype, b, n, parts, w, extra, act, init, lengths = case
    x, wt, bias, h0, dys, dfin = _conv(case)
    lanes = sum(parts) // (1 if any(p % 4 for p in parts) or extra % 4 else 4)
    assert -(-lanes // 64) * b * -(-n // 16) >= 2048
    got = m2.conv1d_backward(_wide(_behind(x, lengths), extra), wt.cuda(), bias.cuda(), _cuda(h0),
                             tuple(_behind(d, lengths).cuda() for d in dys), dfin.cuda(),
                             activation="silu" if act else "none", lengths=_lengths(lengths))
    want = conv_gradients(to64(x), to64(wt), to64(bias), to64(h0), lengths, act,
                          torch.cat([to64(d) for d in dys], -1), to64(dfin), TYPES[dtype])
    for name, v in want.items():
        within(name, got[name], *v)


# ------------------------------------------------------------------------ norm

# A workgroup walks rows from rows > 4096 (backward: 1024) * 256 / its size / groups * its teams on;
# the backward's also from 257 workgroups on (four rows to a team).
NORM = [
    # dtype, rows, groups, group's channels, kind, gate, bias, extra
    ("f32", 33000, 1, 16, "rms", True, True, 0),           # teams of 32, vectors
    ("bf16", 5003, 8, 24, "layer", True, True, 8),
    ("f32", 4500, 8, 30, "layer", False, True, 1),         # teams of 32, one element
    ("bf16", 9000, 16, 31, "rms", True, False, 0),
    ("f32", 2051, 16, 200, "rms", True, False, 4),         # teams of 64
    ("bf16", 1100, 16, 640, "layer", True, True, 0),
    ("bf16", 1030, 32, 200, "layer", True, True, 1),       # teams of 64, one element
    ("f32", 301, 16, 1100, "rms", False, True, 0),         # teams of 256
    ("bf16", 270, 32, 1500, "layer", True, True, 3),
    ("bf16", 601, 8, 2200, "rms", True, True, 0),          # a team of 256 in the backward alone
    ("f32", 150, 8, 5000, "layer", True, True, 0),         # teams of 1024
    ("f32", 70, 16, 4097, "rms", True, True, 0),           # teams of 1024, one element
]


@pytest.mark.parametrize("case", NORM, ids=_id)
def test_norm_teams_that_walk_rows(m2, case):
    say(f"norm {case}")
    dtype, rows, g, dg, kind, gate, bias, extra = case
    io, ch = TYPES[dtype], g * dg
    r = _gen(dg)
    x, dy = r(rows, ch).to(io), r(rows, ch).to(io)
    z = r(rows, ch).to(io) if gate else None
    w, b = 1 + 0.2 * r(ch), 0.1 * r(ch) if bias else None
    xg, zg = _wide(x, extra), None if z is None else _wide(z, extra)
    y = m2.norm_forward(xg, w.cuda(), _cuda(b), zg, ngroups=g, kind=kind)
    got = m2.norm_backward(xg, w.cuda(), _cuda(b), zg, dy.cuda(), ngroups=g, kind=kind)
    a = [to64(v) for v in (x, w, b, z)]
    within("y", y, ref.norm(*a, g, kind, 1e-5), ref.norm_bound(*a, g, kind, 1e-5, io))
    for name, v in norm_gradients(*a, g, kind, 1e-5, to64(dy), io).items():
        if v is None:
            assert got[name] is None
        else:
            within(name, got[name], *v)


# --------------------------------------------------------------- selective scan

# Two sequences per thread from batch * channels * lanes of a row = 2^19 on (states / 4 lanes).
STEP = [
    # dtype, batch, channels, states, groups, extra columns of B, C and z, gate
    ("bf16", 128, 1040, 16, 1, 0, True),
    ("bf16", 129, 1030, 16, 2, 5, True),     # an odd batch, rows of odd steps, a block not full
    ("f32", 65, 2050, 16, 1, 0, False),
    ("f32", 257, 2044, 4, 4, 4, True),
    ("bf16", 65, 4060, 8, 1, 1, True),
    ("bf16", 33, 1986, 32, 2, 0, True),
    ("f32", 67, 1000, 64, 1, 3, True),
]


@pytest.mark.parametrize("case", STEP, ids=_id)
def test_scan_step_of_two_sequences(m2, case):
    say(f"scan step {case}")
    dtype, b, ch, ns, g, extra, gate = case
    assert b * ch * ns // 4 >= 1 << 19
    io, r = TYPES[dtype], _gen(b)
    u, dt = r(b, ch).to(io), (0.5 * r(b, ch)).to(io)
    A = -torch.arange(1, ns + 1) * torch.exp(0.2 * r(ch, ns))
    B, C = r(b, g * ns).to(io), r(b, g * ns).to(io)
    z = r(b, ch).to(io) if gate else None
    D, bias, init = r(ch), r(ch) - 3, r(b, ch, ns)
    k = dict(u=u.cuda(), dt=dt.cuda(), A=A.cuda(), B=_wide(B, extra).unflatten(-1, (g, ns)),
             C=_wide(C, extra).unflatten(-1, (g, ns)), D=D.cuda(),
             z=None if z is None else _wide(z, extra), dt_bias=bias.cuda())
    state = init.cuda()
    y = m2.selective_scan_step(**k, state=state)
    token = lambda v: None if v is None else to64(v)[:, None]
    a = [token(u), token(dt), to64(A), token(B).unflatten(-1, (g, ns)),
         token(C).unflatten(-1, (g, ns)), to64(D), token(z), to64(bias), to64(init)]
    want, wfin = ref.scan(*a)
    by, bf = ref.scan_bounds(*a, None, True, io)
    within("y", y, want[:, 0], by[:, 0])
    within("state", state, wfin, bf)
    # the same sequences a few at a time: one sequence per thread, the same sums
    few = init[:3].cuda()
    some = m2.selective_scan_step(**{q: v if v is None or q in ("A", "D", "dt_bias") else
                                     v[:3].clone() for q, v in k.items()}, state=few)
    assert torch.equal(some, y[:3]) and torch.equal(few, state[:3])


LONG = [
    # dtype, batch, tokens, channels, states, groups, gate, softplus, lengths
    ("f32", 4, 2100, 8, 16, 1, False, True, [2100, 64, 65, 1999]),
    ("f32", 2, 1500, 70, 16, 2, True, True, None),
    ("bf16", 2, 1100, 160, 24, 1, True, True, None),
    ("f32", 1, 1300, 66, 4, 1, True, False, [1299]),
    ("f32", 1, 1000, 33, 64, 1, True, True, None),
    ("bf16", 1, 2048, 64, 7, 4, False, True, [1025]),
]


@pytest.mark.parametrize("case", LONG, ids=_id)
def test_scan_of_long_sequences(m2, case):
    """Bounds that decay with the values: a value rounded to bfloat16 on the way, or a
    term lost between two chunks, shows at any length."""
    say(f"scan long {case}")
    dtype, b, n, ch, ns, g, gate, sp, lengths = case
    io, r = TYPES[dtype], _gen(n)
    u, dy = ref.silu(r(b, n, ch)).to(io), r(b, n, ch).to(io)
    dt = (0.5 * r(b, n, ch)).to(io) if sp else (0.2 * r(b, n, ch).abs()).to(io)
    A = -torch.arange(1, ns + 1) * torch.exp(0.2 * r(ch, ns))
    B, C = r(b, n, g, ns).to(io), r(b, n, g, ns).to(io)
    D, z, bias = r(ch), r(b, n, ch).to(io) if gate else None, 0.3 * r(ch).abs()
    init, dfinal = r(b, ch, ns), r(b, ch, ns)
    a = (u, dt, A, B, C, D, z, bias, init)
    behind = [v if i in (2, 5, 7, 8) or v is None else _behind(v, lengths)
              for i, v in enumerate(a)]
    y, fin = m2.selective_scan_forward(*map(_cuda, behind), softplus=sp, lengths=_lengths(lengths))
    got = m2.selective_scan_backward(*map(_cuda, behind), _behind(dy, lengths).cuda(),
                                     dfinal.cuda(), softplus=sp, lengths=_lengths(lengths))
    a64 = [to64(v) for v in a]
    by, bf = ref.scan_bounds(*a64, lengths, sp, io)
    wy, wf = ref.scan(*a64, lengths, sp)
    within("y", y, wy, by)
    within("final", fin, wf, bf)
    want = scan_gradients(*a64, lengths, sp, to64(dy), to64(dfinal), io)
    rounded = ("du", "ddt", "dB", "dC", "dz")
    for name, v in want.items():
        if v is None:
            assert got[name] is None
            continue
        within(name, got[name], *v)
        # the bound itself is far below a value's bfloat16 step, but for the output's own
        # rounding; sums over all tokens cancel (of n terms about sqrt(n) is left), so that
        # their bound, a count of U times the terms' sizes, says less about their value
        if name in ("dA", "dD", "ddt_bias"):
            continue
        own = half_step(io) * v[0].abs() if name in rounded else 0
        assert ((v[1] - own).pow(2).mean().sqrt() <= 2.0 ** -12 * v[0].pow(2).mean().sqrt()), name

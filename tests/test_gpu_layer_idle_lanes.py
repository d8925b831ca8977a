"""Lanes and teams of the operators around the SSD that have nothing to do (a
channel tile that is not full, a workgroup with fewer rows than teams): what
they compute on the side does not reach the results."""
import pytest
import torch

import layer_reference as ref
from gpu_helpers import say
from layer_bounds import norm_gradients, scan_gradients
from layer_reference import to64, within

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=("f32", "bf16"))
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows", [1, 3, 5, 9, 33])
@pytest.mark.parametrize("group,ngroups", [(32, 1), (32, 3), (64, 1), (256, 2), (512, 1), (30, 2)])
def test_norm_gradients_without_eps(m2, dtype, kind, rows, group, ngroups):
    """eps = 0: a team without a row has a standard deviation of zero."""
    say(f"norm eps 0 {dtype} {kind} {rows} {group} {ngroups}")
    r = _gen(rows + group)
    ch = group * ngroups
    x, z, dy = (r(rows, ch).to(dtype) for _ in range(3))
    w, b = 1 + 0.2 * r(ch), 0.1 * r(ch)
    for bias, gate in ((b, z), (None, None)):
        got = m2.norm_backward(x.cuda(), w.cuda(), _cuda(bias), _cuda(gate), dy.cuda(),
                               ngroups=ngroups, kind=kind, eps=0.0)
        want = norm_gradients(to64(x), to64(w), to64(bias), to64(gate), ngroups, kind, 0.0,
                              to64(dy), dtype)
        for name, v in want.items():
            if v is None:
                assert got[name] is None
            else:
                within(name, got[name], *v)


SCAN = [
    # dtype, batch, tokens, channels, states, groups, gate, bias, smallest time step's bias
    (torch.float32, 2, 200, 70, 16, 1, True, -0.5),
    (torch.float32, 1, 130, 198, 16, 2, False, -0.5),   # 99 channels a group
    (torch.bfloat16, 2, 150, 63, 16, 1, True, -1.0),
    (torch.float32, 1, 70, 65, 4, 1, True, -2.0),
    (torch.float32, 2, 90, 130, 7, 2, False, -2.0),
    (torch.float32, 1, 100, 66, 32, 1, True, -0.5),
    (torch.float32, 1, 66, 3, 64, 1, False, -0.5),
    (torch.float32, 1, 16, 10, 16, 1, True, -3.0),      # one chunk
    (torch.float32, 2, 16, 10, 16, 1, False, -20.0),
]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c[1:])))
def test_scan_with_a_negative_bias_of_the_time_step(m2, case):
    """softplus off, dt_bias < 0 < dt + dt_bias.  A lane without a channel has dt = 0: its
    time step must not be the bias alone, with which its state would grow without bound
    and be 0 * infinity in the sums over channels."""
    dtype, b, n, ch, ns, g, gate, bias = case
    say(f"scan negative bias {case}")
    r = _gen(n)
    u, dy = r(b, n, ch).to(dtype), r(b, n, ch).to(dtype)
    dt = (-bias * (1 + 0.02 * r(b, n, ch).abs()) + 1e-2).to(dtype)
    A = -torch.arange(1, ns + 1) * torch.exp(0.2 * r(ch, ns))
    B, C = r(b, n, g, ns).to(dtype), r(b, n, g, ns).to(dtype)
    D, z = r(ch), r(b, n, ch).to(dtype) if gate else None
    dt_bias = torch.full((ch,), bias)
    init, dfinal = r(b, ch, ns), r(b, ch, ns)
    a = (u, dt, A, B, C, D, z, dt_bias, init)
    y, fin = m2.selective_scan_forward(*map(_cuda, a), softplus=False)
    got = m2.selective_scan_backward(*map(_cuda, a), dy.cuda(), dfinal.cuda(), softplus=False)
    a64 = [to64(v) for v in a]
    assert (a64[1] + a64[7] >= 0).all()
    by, bf = ref.scan_bounds(*a64, None, False, dtype)
    wy, wf = ref.scan(*a64, None, False)
    within("y", y, wy, by)
    within("final", fin, wf, bf)
    want = scan_gradients(*a64, None, False, to64(dy), to64(dfinal), dtype)
    for name, v in want.items():
        if v is None:
            assert got[name] is None
        else:
            within(name, got[name], *v)

"""Padded batches of the operators around the SSD whose real part holds values
that are not finite: what stands behind a sequence stays zero, and the sums
over tokens take nothing from there (0 * infinity is no term of theirs)."""
import pytest
import torch

import layer_reference as ref
from gpu_helpers import say
from layer_bounds import scan_gradients
from layer_reference import F, to64, within

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


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


def _scan(seed, b, n, ch, ns, g, gate, dtype):
    r = _gen(seed)
    t = dict(u=r(b, n, ch).to(dtype), dt=(0.5 * r(b, n, ch)).to(dtype),
             A=-torch.exp(0.3 * r(ch, ns)), B=r(b, n, g, ns).to(dtype), C=r(b, n, g, ns).to(dtype),
             D=r(ch), z=r(b, n, ch).to(dtype) if gate else None, dt_bias=0.1 * r(ch),
             init_state=r(b, ch, ns), dy=r(b, n, ch).to(dtype), dfinal=r(b, ch, ns))
    return t


ROWS = ("du", "ddt", "dB", "dC", "dz")
SIZES = [(150, 70, 16, 1), (16, 64, 16, 1), (100, 33, 4, 3), (90, 66, 8, 1), (70, 64, 32, 1),
         (50, 20, 64, 2)]


@pytest.mark.parametrize("n,ch,ns,g", SIZES)
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=("f32", "bf16"))
def test_scan_gradients_behind_a_sequence_are_zero(m2, n, ch, ns, g, gate, dtype):
    say(f"scan padding {n} {ch} {ns} {g} {gate} {dtype}")
    lens = [n, n // 3, 0, 5]
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    t = _scan(n, 4, n, ch, ns, g, gate, dtype)
    clean = m2.selective_scan_backward(**{k: _cuda(v) for k, v in t.items()}, lengths=lengths)
    for bad in ("u", "dy", "init_state", "dfinal"):
        for value in (NAN, INF):
            k = {name: None if v is None else v.clone() for name, v in t.items()}
            k[bad][1:] = value   # the first sequence stays as it is
            got = m2.selective_scan_backward(**{q: _cuda(v) for q, v in k.items()},
                                             lengths=lengths)
            for name in ROWS:
                if got[name] is None:
                    continue
                for i, m in enumerate(lens):
                    assert (got[name][i, m:] == 0).all(), (bad, value, name, i)
                assert torch.equal(got[name][0], clean[name][0]), (bad, value, name)
            assert torch.equal(got["dinit"][0], clean["dinit"][0])


@pytest.mark.parametrize("n,ch,ns,g", SIZES)
@pytest.mark.parametrize("gate", [True, False])
def test_an_empty_sequence_adds_nothing_to_the_parameters(m2, n, ch, ns, g, gate):
    """The gradients of A, D and dt_bias are sums over tokens; a sequence without any
    passes its dfinal on to its initial state and adds nothing to them."""
    t = {k: _cuda(v) for k, v in _scan(n + 1, 3, n, ch, ns, g, gate, torch.float32).items()}
    lengths = torch.tensor([n, 0, n // 2], dtype=torch.int32).cuda()
    clean = m2.selective_scan_backward(**t, lengths=lengths)
    for name in ("dfinal", "init_state"):
        for value in (NAN, INF):
            k = dict(t)
            k[name] = t[name].clone()
            k[name][1] = value
            got = m2.selective_scan_backward(**k, lengths=lengths)
            for q in ("dA", "dD", "ddt_bias"):
                assert torch.equal(got[q], clean[q]), (name, value, q)
            assert torch.equal(got["dinit"][1].isnan(), k["dfinal"][1].isnan())


@pytest.mark.parametrize("n,m,ch,ns", [(100, 37, 64, 16), (100, 64, 70, 16), (16, 5, 10, 16),
                                       (40, 16, 64, 16), (80, 30, 64, 64), (60, 33, 8, 4)])
def test_a_state_that_overflows_at_the_last_token(m2, n, m, ch, ns):
    """h is infinite after the last token of a padded sequence; the gradient of A only
    multiplies the states before a token, which are finite."""
    t = _scan(n + 2, 1, n, ch, ns, 1, False, torch.float32)
    t["dt_bias"], t["dt"] = None, torch.full((1, n, ch), 1.0)
    t["u"][0, m - 1], t["B"][0, m - 1] = 2e38, 4.0
    t["dy"], t["dfinal"] = 1e-2 * t["dy"], 1e-4 * t["dfinal"]
    t["D"] = None
    lengths = torch.tensor([m], dtype=torch.int32).cuda()
    got = m2.selective_scan_backward(**{k: _cuda(v) for k, v in t.items()}, lengths=lengths)
    a = [to64(t[k]) for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "init_state")]
    want = scan_gradients(*a, [m], True, to64(t["dy"]), to64(t["dfinal"]), torch.float32)
    for name in ("dA", "dinit", "du", "dB"):
        v, bound = want[name]
        fits = v.abs() < 1e38
        assert fits.any()
        within(name, torch.where(fits, got[name].cpu().to(F), v), v, bound)


@pytest.mark.parametrize("n,m,c,w", [(40, 17, 64, 4), (130, 100, 64, 4), (20, 5, 33, 3),
                                     (9, 1, 8, 2), (40, 32, 64, 4), (40, 31, 7, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=("f32", "bf16"))
def test_convolution_gradient_with_an_infinite_last_token(m2, n, m, c, w, dtype):
    """Without an activation an infinite last row meets only the last tap's gradient; the
    taps before it would meet it in the padding, where g is zero."""
    r = _gen(n + c)
    x, dy = r(2, n, c).to(dtype), r(2, n, c).to(dtype)
    wt, bias = r(c, w), r(c)
    x[1, m - 1] = INF
    lens = [n, m]
    got = m2.conv1d_backward(x.cuda(), wt.cuda(), bias.cuda(), None, dy.cuda(), activation="none",
                             lengths=torch.tensor(lens, dtype=torch.int32).cuda())
    a = (to64(x), to64(wt), to64(bias), torch.zeros(2, w - 1, c, dtype=F))
    want = ref.grads(lambda *v: ref.conv(*v, lens, False), a, (to64(dy), None))
    assert torch.isfinite(want[1][:, :-1]).all() and torch.isinf(want[1][:, -1]).all()
    g = got["dweight"].cpu().to(F)
    # two roundings a product, at most 32 + 4 + the tiles' additions, on the terms' sizes
    size = torch.where(torch.isinf(a[0]), torch.zeros_like(a[0]), a[0]).abs()
    big = ref.grads(lambda *v: ref.conv(*v, lens, False), (size,) + a[1:], (to64(dy).abs(), None))
    within("dweight", g[:, :-1], want[1][:, :-1], (40 + 2 * n) * ref.U * big[1][:, :-1])
    assert torch.equal(g[:, -1], want[1][:, -1])
    assert (got["dx"][1, m:] == 0).all() and torch.isfinite(got["dx"]).all()

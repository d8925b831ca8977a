"""Teams of the operators around the SSD that have nothing to do (a workgroup
with fewer rows than teams): what they compute on the side does not reach the
results."""
import pytest
import torch

from gpu_helpers import say
from layer_bounds import norm_gradients
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

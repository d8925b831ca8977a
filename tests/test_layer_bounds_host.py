"""The float64 gradient formulas that the GPU tests compare with, against
automatic differentiation of the float64 operators."""
import pytest
import torch

import layer_reference as ref
from layer_bounds import scan_gradients
from layer_reference import F


@pytest.mark.parametrize("gate,sp,lengths,full", [
    (True, True, None, True), (False, True, [9, 0, 4], True), (True, False, [-3, 1, 70], True),
    (False, False, None, False)])
def test_scan_formulas_are_the_derivatives(gate, sp, lengths, full):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=F)
    b, n, ch, ns, groups = 3, 9, 6, 3, 2
    a = [r(b, n, ch), r(b, n, ch).abs(), -r(ch, ns).abs(), r(b, n, groups, ns), r(b, n, groups, ns),
         r(ch) if full else None, r(b, n, ch) if gate else None, r(ch).abs() if full else None,
         r(b, ch, ns)]
    dy, df = r(b, n, ch), r(b, ch, ns)
    want = ref.grads(lambda *v: ref.scan(*v, lengths, sp), a, (dy, df))
    got = scan_gradients(*a, lengths, sp, dy, df, torch.float32)
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")
    for name, w in zip(names, want):
        if w is None:
            assert got[name] is None
            continue
        v, bound = got[name]
        assert torch.allclose(v, w, rtol=1e-10, atol=1e-12), name
        assert (bound >= 0).all() and (bound <= 1e-4 * (1 + v.abs().max())).all(), name

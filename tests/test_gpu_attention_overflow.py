"""Scores beyond float32.  A query and a key whose product is infinite make the
query's o and lse NaN: lse = -infinity says that a row sees no key, and this
one does.  A product beyond float32 on the other side is a weight of 0, and
rows that do not see the key are what they are without it."""
import math

import pytest
import torch

import attention_reference as ref
from gpu_helpers import say
from test_gpu_attention import BF, F32, close, m2, rnd, whole  # noqa: F401

pytestmark = pytest.mark.gpu
HUGE = 1e20  # finite in either type, its square is not


def pair(g, dtype, B, nq, nk, H, G, D, i, j, sign):
    """Inputs of which only query i (head 1) and key j (of its group) of sequence 0 meet beyond
    float32: both hold HUGE in column 0, all others 0."""
    q, k, v = rnd(g, B, nq, H, D, dtype=dtype), rnd(g, B, nk, G, D, dtype=dtype), \
        rnd(g, B, nk, G, D, dtype=dtype)
    q[..., 0] = k[..., 0] = 0
    q[0, i, 1, 0], k[0, j, 1 // (H // G), 0] = sign * HUGE, HUGE
    return q, k, v


CASES = [
    # dtype, B, queries, keys, H, G, D, query, key, parts
    (BF, 9, 300, 300, 16, 8, 64, 200, 130, False),   # one set of wavefronts
    (BF, 1, 150, 150, 2, 1, 128, 70, 3, False),      # two sets
    (BF, 2, 9, 4000, 8, 8, 128, 5, 3001, True),      # parts, joined
    (F32, 1, 70, 70, 2, 1, 64, 60, 40, False),
    (F32, 2, 5, 2600, 2, 1, 64, 0, 0, True),
]


@pytest.mark.parametrize("dtype,B,nq,nk,H,G,D,i,j,parts", CASES)
def test_prompt(m2, dtype, B, nq, nk, H, G, D, i, j, parts):  # noqa: F811
    say(f"[overflow] {dtype} {B} {nq} {nk} {H} {G} {D}")
    scale = 1 / math.sqrt(D)
    dims = m2.make_attention_dims(B, nq, nk, H, G, D, dtype)
    assert (m2.mamba2_attention_workspace_bytes(dims) > 256) == parts
    assert j <= i + nk - nq
    for sign in (1, -1):
        q, k, v = pair(torch.Generator().manual_seed(61), dtype, B, nq, nk, H, G, D, i, j, sign)
        o, lse = m2.attention_forward(*(x.cuda() for x in (q, k, v)))
        # sequence 0; in float64 the product has its size: exp(-1e39) is 0, and the bounds of the
        # one row are not looked at
        want, bound = ref.attention(ref.to64(q[0]), ref.to64(k[0]), ref.to64(v[0]), [(0, nq)],
                                    [(0, nk)], True, scale, dtype)
        torch.cuda.synchronize()
        rows = torch.ones(nq, H, dtype=torch.bool)
        rows[i, 1] = False
        for name, got in (("o", o), ("lse", lse)):
            close(got[0].cpu()[rows], want[name][rows], bound[name][rows], name)
        one, l = o[0, i, 1].cpu(), lse[0, i, 1].cpu()
        if sign > 0:
            assert torch.isnan(one).all() and torch.isnan(l)
        else:  # the same row without the key
            kept = [n for n in range(i + nk - nq + 1) if n != j]
            if not kept:
                continue
            own = [ref.to64(t[0, kept, 1 // (H // G)])[:, None] for t in (k, v)]
            alone, limit = ref.attention(ref.to64(q[0, i:i + 1, 1:2]) * (torch.arange(D) > 0), *own,
                                         [(0, 1)], [(0, len(kept))], False, scale, dtype)
            close(one, alone["o"][0, 0], limit["o"][0, 0], "o without the key")
            close(l, alone["lse"][0, 0], limit["lse"][0, 0], "lse without the key")


@pytest.mark.parametrize("dtype,B,nq,nk,H,G,D,i,j,parts", CASES)
def test_products_within_and_scores_beyond(m2, dtype, B, nq, nk, H, G, D, i, j, parts):  # noqa: F811
    """A product of 1e10 that the scale (1e30) takes beyond float32; all others are 0."""
    say(f"[scores] {dtype} {B} {nq} {nk} {H} {G} {D}")
    for sign in (1, -1):
        q, k, v = pair(torch.Generator().manual_seed(65), dtype, B, nq, nk, H, G, D, i, j, sign)
        q, k = (torch.where(x.abs() == x.abs().max(), 1e5 * x.sign(), 0 * x) for x in (q, k))
        o, lse = m2.attention_forward(*(x.cuda() for x in (q, k, v)), scale=1e30)
        # the same scores by a scale of 1: 0, and below -1e38 or not looked at
        want, bound = ref.attention(ref.to64(q[0]) * 1e15, ref.to64(k[0]) * 1e15, ref.to64(v[0]),
                                    [(0, nq)], [(0, nk)], True, 1.0, dtype)
        torch.cuda.synchronize()
        rows = torch.ones(nq, H, dtype=torch.bool)
        rows[i, 1] = False
        for name, got in (("o", o), ("lse", lse)):
            close(got[0].cpu()[rows], want[name][rows], bound[name][rows], name)
        one, l = o[0, i, 1].cpu(), lse[0, i, 1].cpu()
        if sign > 0:
            assert torch.isnan(one).all() and torch.isnan(l)
        elif i + nk - nq:  # the mean of the other keys
            n = i + nk - nq + 1
            rest = ref.to64(v[0, :n, 1 // (H // G)])
            rest = (rest.sum(0) - rest[j]) / (n - 1)
            assert ((ref.to64(one) - rest).abs() <= 2 * ref.half_step(dtype) * (rest.abs() + 1)).all()
            assert abs(float(l) - math.log(n - 1)) <= 16 * ref.U * math.log(n)


@pytest.mark.parametrize("dtype,B,nq,nk,H,G,D,i,j,parts", CASES)
def test_queries_that_are_not_numbers(m2, dtype, B, nq, nk, H, G, D, i, j, parts):  # noqa: F811
    """A row of which no score is a number is no row without keys either."""
    q, k, v = pair(torch.Generator().manual_seed(66), dtype, B, nq, nk, H, G, D, i, j, 1)
    q[0, i, 1] = float("nan")
    o, lse = m2.attention_forward(*(x.cuda() for x in (q, k, v)))
    torch.cuda.synchronize()
    assert torch.isnan(o[0, i, 1]).all() and torch.isnan(lse[0, i, 1])
    rows = torch.ones(nq, H, dtype=torch.bool)
    rows[i, 1] = False
    assert torch.isfinite(o[0].cpu()[rows]).all() and torch.isfinite(lse[0].cpu()[rows]).all()


def test_gradients(m2):  # noqa: F811
    """dq of the row is not a number either, nor what its keys get from it; another sequence's
    gradients do not feel it."""
    for dtype in (BF, F32):
        x = pair(torch.Generator().manual_seed(62), dtype, 2, 70, 70, 2, 1, 64, 60, 40, 1)
        dout = rnd(torch.Generator().manual_seed(63), 2, 70, 2, 64, dtype=dtype)
        dev = [t.cuda() for t in (*x, dout)]
        o, lse = m2.attention_forward(*dev[:3])
        got = m2.attention_backward(*dev[:3], o, lse, dev[3])
        one = [t[1:].contiguous() for t in dev]
        want = m2.attention_backward(*one[:3], *m2.attention_forward(*one[:3]), one[3])
        torch.cuda.synchronize()
        assert torch.isnan(got["dq"][0, 60, 1]).all() and torch.isnan(got["dv"][0, :61]).all()
        for n in want:
            assert torch.isfinite(want[n]).all() and torch.equal(got[n][1:], want[n]), n


@pytest.mark.parametrize("huge,scale", [(HUGE, None), (1e5, 1e30)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,prefix", [(100, 0), (2000, 0), (100, 300)])
def test_step(m2, dtype, rows, prefix, huge, scale):  # noqa: F811
    """One token: against a key of the cache, and of the prefix; with a scale that takes a product
    there all other scores are 0."""
    B, H, G, D = 3, 4, 2, 64
    g = torch.Generator().manual_seed(64)
    for place in ("cache", "prefix") if prefix else ("cache",):
        q, k, v = (rnd(g, B, n, D, dtype=dtype) for n in (H, G, G))
        kc, vc = (rnd(g, B, rows, G, D, dtype=dtype) for _ in range(2))
        kp, vp = (rnd(g, prefix, G, D, dtype=dtype) if prefix else None for _ in range(2))
        for x in (q, k, kc, kp):
            if x is not None:
                x[..., :1 if scale is None else D] = 0
        q[1, 3, 0] = huge
        (kc[1] if place == "cache" else kp)[70, 1, 0] = huge
        lens = [rows - 1, rows, 20]
        o = m2.attention_step(*(x.cuda() for x in (q, k, v, kc, vc)), whole(lens),
                              None if kp is None else kp.cuda(), None if vp is None else vp.cuda(),
                              scale=scale)
        torch.cuda.synchronize()
        o = o.cpu()
        want, bound, _, _ = ref.step(*(ref.to64(t) for t in (q, k, v, kc, vc)), lens, ref.to64(kp),
                                     ref.to64(vp), 1 / math.sqrt(D) if scale is None else 1.0, dtype)
        assert torch.isnan(o[1, 3]).all(), place
        others = torch.ones(B, H, dtype=torch.bool)
        others[1, 3] = False
        close(o[others], want[others], bound[others], f"o, {place}")

"""Gradients of attention to scores far above one.

Most weights are then 0 or 1 and most dS = P (dP - delta) vanish by
cancellation.  P is exp(s - lse) with an lse that is good to its own rounding,
so all weights of a row carry one common factor 1 + e, with e about |lse| 2^-24
times a few: it may scale a row's dS, but it must not reach the difference.
The bounds below hold for a delta that is formed as the mean of dP under the
same weights.  First order, with E_j the relative error of weight j and n keys:
    delta = sum P dP / sum P is off by
        sum_j p_j (E_j |dP_j - delta| + |error of dP_j|) + (n + 4) U sum_j p_j |dP_j|
    (n + 1 roundings of either sum at most, the division, the quotient's own);
    dS_j is off by p_j (errors of dP_j and delta, two roundings) + E_j |dS_j|.
Rows that see more than FEW keys take delta = dO . o instead, which is o's error
(sum_j p_j E_j |v_j - o| by element, n + 8 roundings of its sum of sizes) times dO;
here in float32 only, where o has no rounding to fewer bits.  What is below
TINY, the smallest normal float32 (and bfloat16), may be taken as 0: a weight, a
dS, a product of it.  A dot product of D terms is off by (D + 1) U times its
terms' sizes.
"""
import math

import pytest
import torch

import attention_reference as ref
from attention_reference import U, half_step, to64, weight_step
from gpu_helpers import say

BF, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -126
FEW = 32


def gradients(q, k, v, dout, scale, dtype):
    """Float64 dq, dk of causal q[L,H,D], k, v [L,G,D], dout[L,H,D], and their bounds."""
    n, h, d = q.shape
    rep = h // k.shape[1]
    want, err = {}, {}
    for name, t in (("dq", q), ("dk", k)):
        want[name], err[name] = torch.zeros_like(t), torch.zeros_like(t)
    ws, hs = weight_step(dtype), half_step(dtype)
    for j in range(h):
        a, b, c, t = q[:, j], k[:, j // rep], v[:, j // rep], dout[:, j]
        s, p, _, lse = ref.one_head(a, b, c, True, scale)
        e = ref.score_error(a, b, s, lse, scale) + 2 * U * lse.abs()[:, None]
        dp = t @ c.t()
        delta = (p * dp).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        edp = (d + 1) * U * (t.abs() @ c.abs().t())
        ed = (p * (e * (dp - delta).abs() + edp)).sum(-1, keepdim=True) + \
            (n + 4) * U * (p * dp.abs()).sum(-1, keepdim=True)
        if n > FEW:
            assert dtype is F32
            o = p @ c
            eo = ((p * e)[..., None] * (c[None] - o[:, None]).abs()).sum(1) + (n + 8) * U * (p @ c.abs())
            many = (t.abs() * eo).sum(-1, keepdim=True) + (d + 1) * U * (t * o).abs().sum(-1, keepdim=True)
            ed[FEW:] = many[FEW:]
        # the second order: a factor of 1 + e on the terms of the first
        size = dp.abs() + delta.abs()
        eds = (1 + 2 * e) * (p * (edp + ed + 2 * U * size) + ds.abs() * (e + ws)) + TINY * (size + 1)
        want["dq"][:, j] = scale * (ds @ b)
        err["dq"][:, j] = scale * (eds @ b.abs() + (n + 8) * U * (ds.abs() @ b.abs()))
        want["dk"][:, j // rep] += scale * (ds.t() @ a)
        err["dk"][:, j // rep] += scale * (eds.t() @ a.abs() + (n * rep + 8) * U * (ds.abs().t() @ a.abs()))
    for name in want:
        err[name] += hs * (want[name].abs() + err[name]) + (n * rep + 1) * TINY
    return want, err


def inputs(dtype, H, G, D, size, n, seed=51):
    """n tokens whose scores (scale 1) are about `size`."""
    g = torch.Generator().manual_seed(seed)
    x = math.sqrt(size) / D ** 0.25
    q, k = x * torch.randn(n, H, D, generator=g), x * torch.randn(n, G, D, generator=g)
    v, dout = torch.randn(n, G, D, generator=g), torch.randn(n, H, D, generator=g)
    return [t.to(dtype) for t in (q, k, v, dout)]


def steep(dtype, D, n):
    """Scores from -1e4 to 1e4 in steps of hundreds: the newest key has all the weight."""
    q, k = torch.zeros(n, 2, D), torch.zeros(n, 2, D)
    q[..., 0] = 100.0
    k[:, :, 0] = torch.linspace(-100, 100, n)[:, None]
    g = torch.Generator().manual_seed(52)
    return [t.to(dtype) for t in (q, k, torch.randn(n, 2, D, generator=g),
                                  torch.randn(n, 2, D, generator=g))]


CASES = [(dtype, H, G, D, size, FEW) for dtype in (F32, BF)
         for H, G, D, size in ((4, 2, 8, 30), (4, 2, 8, 100), (4, 2, 8, 1000), (2, 1, 64, 1000),
                               (2, 2, 128, 3000), (2, 2, 8, 0), (2, 2, 64, 0))]
CASES += [(F32, 4, 2, 8, 100, 70), (F32, 2, 1, 64, 1000, 70), (F32, 2, 2, 64, 0, 70)]


def make(dtype, H, G, D, size, n):
    return inputs(dtype, H, G, D, size, n) if size else steep(dtype, D, n)


def over(got, want, err):
    """How far above its bound the worst element of each gradient is, as a factor."""
    return {n: float(((to64(got[n]).reshape(want[n].shape) - want[n]).abs() /
                      err[n]).max()) for n in want}


def emulated(q, k, v, dout, scale, normalised):
    """The formula in float32 as the kernels evaluate it: weights from a rounded lse."""
    n, h, d = q.shape
    rep = h // k.shape[1]
    got = {"dq": torch.zeros(n, h, d), "dk": torch.zeros(n, k.shape[1], d)}
    c = torch.tensor(scale * 1.4426950408889634, dtype=F32)
    gone = torch.ones(n, n).triu(1).bool()
    for j in range(h):
        a, b, w, t = (x.float() for x in (q[:, j], k[:, j // rep], v[:, j // rep], dout[:, j]))
        s = (a @ b.t()).masked_fill(gone, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp2((s.double() * c.double() - (m * c).double()).float())
        lse = ((m.double() * c.double()).float() + p.sum(-1, keepdim=True).log2()) * math.log(2)
        p = torch.exp2((s.double() * c.double() - (lse * 1.4426950408889634).double()).float())
        dp = t @ w.t()
        delta = (p * dp).sum(-1, keepdim=True)
        if normalised:
            delta = delta / p.sum(-1, keepdim=True)
        first = torch.exp2((s.double() * c.double() - (m * c).double()).float())
        o = first @ w / first.sum(-1, keepdim=True)
        delta[FEW:] = (t * o).sum(-1, keepdim=True)[FEW:]
        ds = (p * (dp - delta)).to(q.dtype).float()
        got["dq"][:, j] = scale * (ds @ b)
        got["dk"][:, j // rep] += scale * (ds.t() @ a)
    return {n: x.to(q.dtype) for n, x in got.items()}


@pytest.mark.parametrize("dtype,H,G,D,size,n", CASES)
def test_bounds_tell_the_mean_from_the_plain_sum(dtype, H, G, D, size, n):
    """The bounds on the CPU: a mean under the same weights keeps them, a plain sum does not (but
    for scores of tens, whose lse is too small)."""
    x = make(dtype, H, G, D, size, n)
    want, err = gradients(*(to64(t) for t in x), 1.0, dtype)
    good, bad = (over(emulated(*x, 1.0, normalised), want, err) for normalised in (True, False))
    say(f"[scores] {dtype} {H} {G} {D} {size} {n}: mean {good}, sum {bad}")
    assert max(good.values()) <= 1
    if size != 30:
        assert max(bad.values()) > 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,G,D,size,n", CASES)
def test_gradients_of_large_scores(dtype, H, G, D, size, n):
    import state_space_sequence_02_amd as m2
    x = make(dtype, H, G, D, size, n)
    want, err = gradients(*(to64(t) for t in x), 1.0, dtype)
    q, k, v, dout = (t[None].cuda() for t in x)
    o, lse = m2.attention_forward(q, k, v, scale=1.0)
    got = m2.attention_backward(q, k, v, o, lse, dout, scale=1.0)
    torch.cuda.synchronize()
    far = over(got, want, err)
    say(f"[scores] {dtype} {H} {G} {D} {size} {n}: {far}")
    assert max(far.values()) <= 1, far

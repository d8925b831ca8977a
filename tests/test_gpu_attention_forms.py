"""The forms of attention that only larger problems reach: tiles that fill the
device without being split, walks that are split with parts (each recognised by
its workspace), long walks of an even and an odd number of steps, several row
tiles of a step's groups; against float64 as in test_gpu_attention.py."""
import math

import pytest
import torch

import attention_reference as ref
from gpu_helpers import say
from test_gpu_attention import BF, F32, build, close, m2, rnd, whole  # noqa: F401

pytestmark = pytest.mark.gpu


CASES = [
    # dtype, H, G, D, form, causal, queries, keys, forward's parts, backward's parts
    (BF, 16, 8, 64, "padded", True, [300] * 9, [300] * 9, False, False),
    (BF, 16, 8, 128, "padded", False, [130, 70, 0] * 6, [130, 70, 0] * 6, False, False),
    (BF, 24, 8, 104, "packed", True, [250, 1, 77, 128, 129] * 4, [250, 1, 77, 128, 129] * 4, False,
     False),
    (F32, 16, 8, 64, "padded", True, [170] * 10, [170] * 10, False, False),
    (F32, 24, 8, 72, "cross", True, [100] * 12, [60, 100, 140] * 4, False, False),
    (BF, 2, 1, 64, "padded", True, [1100], [1100], True, True),
    (BF, 2, 1, 128, "cross", False, [700], [1300], True, True),
    (F32, 3, 1, 128, "padded", True, [260], [260], True, True),
    (F32, 2, 2, 40, "packed", False, [200, 90], [200, 90], True, True),
]


@pytest.mark.parametrize("dtype,H,G,D,form,causal,nq,nk,parts,back_parts", CASES)
def test_attention_forms(m2, dtype, H, G, D, form, causal, nq, nk, parts, back_parts):  # noqa: F811
    say(f"[forms] {dtype} H={H} G={G} D={D} {form} causal={causal} {len(nq)} sequences")
    g = torch.Generator().manual_seed(41)
    (q, k, v), kw, flat, qs, ks = build(g, dtype, H, G, D, form, nq, nk, 0, 0, 0.0)
    packed = form == "packed"
    dims = m2.make_attention_dims(len(nq), q.shape[-3], k.shape[-3], H, G, D, dtype, causal=causal,
                                  q_packed=packed, k_packed=packed)
    rows = flat[0].shape[0] * H * 8 + 511
    assert (m2.mamba2_attention_workspace_bytes(dims) > 256) == parts
    assert (m2.mamba2_attention_backward_workspace_bytes(dims) > rows) == back_parts
    dout = rnd(g, *q.shape, dtype=dtype)
    scale = 1 / math.sqrt(D)
    o, lse = m2.attention_forward(q, k, v, causal=causal, **kw)
    got = m2.attention_backward(q, k, v, o, lse, dout.cuda(), causal=causal, **kw)
    torch.cuda.synchronize()
    want, bound = ref.attention(*flat, qs, ks, causal, scale, dtype, ref.to64(dout).view(-1, H, D))
    got |= {"o": o, "lse": lse}
    for name in want:
        close(got[name], want[name], bound[name], name)
        # the bounds add every rounding up; in the 2-norm, where they average out, the error is
        # within the output's rounding and as much again for weights of the same type
        w = want[name][torch.isfinite(want[name])]
        x = ref.to64(got[name]).reshape(want[name].shape)[torch.isfinite(want[name])]
        step = ref.half_step(got[name].dtype)
        assert float((x - w).norm()) <= (2 if dtype is BF else 60) * step * float(w.norm()), name


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_step_of_many_sequences(m2, dtype, D):  # noqa: F811
    """Enough sequences that no cache is split, 40 heads of a group in two row tiles."""
    B, rows, H, G = 150, 70, 80, 2
    g = torch.Generator().manual_seed(42)
    q, k, v = (rnd(g, B, n, D, dtype=dtype) for n in (H, G, G))
    kc, vc = (rnd(g, B, rows, G, D, dtype=dtype) for _ in range(2))
    lens = [(11 * i) % (rows + 1) for i in range(B)]
    dims = m2.make_attention_step_dims(B, rows, H, G, D, dtype)
    assert m2.mamba2_attention_step_workspace_bytes(dims) == 256
    o = m2.attention_step(*(t.cuda() for t in (q, k, v, kc, vc)), whole(lens))
    torch.cuda.synchronize()
    some = [0, 1, 6, 77, 149]
    want, bound, _, _ = ref.step(*(ref.to64(t[some]) for t in (q, k, v, kc, vc)),
                                 [lens[i] for i in some], None, None, 1 / math.sqrt(D), dtype)
    close(o[some], want, bound, "o")


def test_step_of_long_caches(m2):  # noqa: F811
    """Long caches without a split: workgroups of eight wavefronts; and the same split."""
    for B, rows in ((200, 1500), (3, 9000)):
        H, G, D = 8, 2, 128
        g = torch.Generator().manual_seed(43)
        q, k, v = (rnd(g, B, n, D, dtype=BF) for n in (H, G, G))
        gpu = torch.Generator(device="cuda").manual_seed(44)
        kc, vc = (torch.randn(B, rows, G, D, generator=gpu, device="cuda").to(BF) for _ in range(2))
        lens = [(977 * i + rows - 7) % (rows + 1) for i in range(B)]
        o = m2.attention_step(q.cuda(), k.cuda(), v.cuda(), kc.clone(), vc.clone(), whole(lens))
        torch.cuda.synchronize()
        for i in (0, 1, B - 1):
            one = [ref.to64(t[i:i + 1]) for t in (q, k, v, kc, vc)]
            want, bound, _, _ = ref.step(*one, [lens[i]], None, None, 1 / math.sqrt(D), BF)
            close(o[i:i + 1], want, bound, f"o of {B} x {rows}, {i}")


def test_tiny_scale(m2):  # noqa: F811
    """A scale that leaves every score 0 in float32: plain means, lse = log of the keys seen."""
    g = torch.Generator().manual_seed(45)
    q, k, v = rnd(g, 1, 90, 2, 32).cuda(), rnd(g, 1, 90, 2, 32).cuda(), rnd(g, 1, 90, 2, 32).cuda()
    o, lse = m2.attention_forward(q, k, v, scale=1e-40)
    torch.cuda.synchronize()
    n = torch.arange(1, 91, device="cuda", dtype=torch.float64)
    want = v[0].double().cumsum(0) / n[:, None, None]
    # a mean of n values: n + 3 roundings of the sum of their sizes over n, at most 4
    assert ((o[0].double() - want).abs() <= (n[:, None, None] + 3) * ref.U * 4).all()
    assert ((lse[0].double() - n.log()[:, None]).abs() <= 8 * ref.U * (1 + n.log()[:, None])).all()


def test_rotary_of_more_tokens_than_workgroups(m2):  # noqa: F811
    """Over 2^23 tokens: workgroups take more than one table of tokens."""
    n = (1 << 23) + 777
    gpu = torch.Generator(device="cuda").manual_seed(46)
    q = torch.randn(n, 1, 2, generator=gpu, device="cuda")
    inv = torch.tensor([0.37], device="cuda")
    y = m2.rotary_forward(q, None, inv)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(50), torch.arange((1 << 23) - 20, n, 3), torch.randint(0, n, (500,))])
    x = ref.to64(q[at.cuda()])
    want = ref.rotary(x, inv.cpu(), at, "half", 1.0)
    close(y[at.cuda()], want, ref.rotary_bound(x, want, 2, "half", 1.0, F32), "y")

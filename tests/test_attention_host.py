"""Host-only checks of the operators of an attention layer: their structs,
refusals of the C interface before anything touches a device, the wrappers'
checks of tensors, and the float64 forms that the GPU tests compare with.
None of these calls launches a kernel."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import attention_reference as ref
import state_space_sequence_02_amd as m2
from test_asm_hazards import CSRC, HIPCC, ROOT, _hazards

OK = 1 << 20  # a 16-byte aligned address that is never read: checks fail first
BIG = 1 << 40
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def test_struct_layouts():
    assert ctypes.sizeof(m2.Mamba2RotaryDims) == 10 * 8 + 4 * 4
    assert m2.Mamba2RotaryDims.scale.offset == 80 and m2.Mamba2RotaryDims.reserved.offset == 92
    assert ctypes.sizeof(m2.Mamba2AttentionDims) == 12 * 8 + 6 * 4
    assert m2.Mamba2AttentionDims.scale.offset == 96
    assert m2.Mamba2AttentionDims.dtype.offset == 112
    assert ctypes.sizeof(m2.Mamba2AttentionStepDims) == 9 * 8 + 2 * 4
    assert m2.Mamba2AttentionStepDims.dtype.offset == 76


def rdims(**kw):
    a = dict(batch=2, seqlen=10, nheads=4, ngroups=2, headdim=64, rotary=32, dtype=BF)
    return m2.make_rotary_dims(**(a | kw))


def adims(**kw):
    a = dict(batch=2, q_len=100, k_len=120, nheads=4, ngroups=2, headdim=64, dtype=BF)
    return m2.make_attention_dims(**(a | kw))


def sdims(**kw):
    a = dict(batch=2, rows=100, nheads=4, ngroups=2, headdim=64, dtype=BF)
    return m2.make_attention_step_dims(**(a | kw))


def rotary(d, back=False, **over):
    a = dict(q=OK, k=OK, inv=OK, pos=None, yq=OK, yk=OK) | over
    fn = m2._lib.mamba2_rotary_backward if back else m2._lib.mamba2_rotary_forward
    return fn(ctypes.byref(d) if d else None, *a.values(), 0)


def forward(d, **over):
    a = dict(q=OK, k=OK, v=OK, qs=None, ks=None, o=OK, lse=OK, ws=OK, n=BIG) | over
    return m2._lib.mamba2_attention_forward(ctypes.byref(d) if d else None, *a.values(), 0)


def backward(d, **over):
    a = dict(q=OK, k=OK, v=OK, qs=None, ks=None, o=OK, lse=OK, do=OK, dq=OK, dk=OK, dv=OK, ws=OK,
             n=BIG) | over
    return m2._lib.mamba2_attention_backward(ctypes.byref(d) if d else None, *a.values(), 0)


def step(d, **over):
    a = dict(q=OK, k=OK, v=OK, kc=OK, vc=OK, lens=OK, kp=None, vp=None, o=OK, ws=OK, n=BIG) | over
    return m2._lib.mamba2_attention_step(ctypes.byref(d) if d else None, *a.values(), 0)


def _set(d, **kw):
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), m2.MAMBA2_ERR_DTYPE),
    (dict(batch=0), m2.MAMBA2_ERR_SHAPE),
    (dict(seqlen=0), m2.MAMBA2_ERR_SHAPE),
    (dict(nheads=0), m2.MAMBA2_ERR_SHAPE),
    (dict(ngroups=-1), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=0), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=31), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=66), m2.MAMBA2_ERR_SHAPE),
    (dict(scale=0.0), m2.MAMBA2_ERR_SHAPE),
    (dict(scale=float("nan")), m2.MAMBA2_ERR_SHAPE),
    (dict(scale=float("inf")), m2.MAMBA2_ERR_SHAPE),
    (dict(q_stride=255), m2.MAMBA2_ERR_SHAPE),
    (dict(yk_stride=127), m2.MAMBA2_ERR_SHAPE),
    (dict(k_stride=1 << 25), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(headdim=1026), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=1 << 16), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=2, seqlen=1 << 28), m2.MAMBA2_ERR_UNSUPPORTED),
])
def test_rotary_refuses_sizes(kw, status):
    for back in (False, True):
        assert rotary(rdims(**kw), back) == status
        assert m2.mamba2_last_error() != ""


def test_rotary_refuses_pointers():
    assert rotary(None) == m2.MAMBA2_ERR_NULL
    for name in ("q", "k", "inv", "yq", "yk"):
        assert rotary(rdims(), **{name: None}) == m2.MAMBA2_ERR_NULL
        assert rotary(rdims(), **{name: OK + 8}) == m2.MAMBA2_ERR_ALIGN
    assert rotary(rdims(), pos=OK + 4) == m2.MAMBA2_ERR_ALIGN
    assert rotary(_set(rdims(), reserved=1)) == m2.MAMBA2_ERR_SHAPE
    assert rotary(_set(rdims(), layout=2)) == m2.MAMBA2_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), m2.MAMBA2_ERR_DTYPE),
    (dict(batch=0), m2.MAMBA2_ERR_SHAPE),
    (dict(q_len=0), m2.MAMBA2_ERR_SHAPE),
    (dict(k_len=0), m2.MAMBA2_ERR_SHAPE),
    (dict(ngroups=3), m2.MAMBA2_ERR_SHAPE),
    (dict(ngroups=0), m2.MAMBA2_ERR_SHAPE),
    (dict(headdim=0), m2.MAMBA2_ERR_SHAPE),
    (dict(headdim=60), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(headdim=136), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(nheads=2048, ngroups=1), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(scale=0.0), m2.MAMBA2_ERR_SHAPE),
    (dict(scale=-1.0), m2.MAMBA2_ERR_SHAPE),
    (dict(scale=float("inf")), m2.MAMBA2_ERR_SHAPE),
    (dict(q_stride=248), m2.MAMBA2_ERR_SHAPE),
    (dict(q_stride=260), m2.MAMBA2_ERR_UNSUPPORTED),          # no multiple of 16 bytes
    (dict(dv_stride=132), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(dtype=F32, k_stride=130), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(k_stride=(1 << 22) + 8), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(q_len=1 << 29), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=2, k_len=1 << 28), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=1, q_len=1 << 27, nheads=32, ngroups=2), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=1, q_len=1 << 28, nheads=1024, ngroups=1024), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=1, k_len=1 << 27, nheads=16, ngroups=16), m2.MAMBA2_ERR_UNSUPPORTED),
])
def test_attention_refuses_sizes(kw, status):
    d = adims(**kw)
    assert forward(d) == status and backward(d) == status
    assert m2.mamba2_last_error() != ""
    assert m2.mamba2_attention_workspace_bytes(d) == 0
    assert m2.mamba2_attention_backward_workspace_bytes(d) == 0


def test_attention_refuses_pointers():
    assert forward(None) == m2.MAMBA2_ERR_NULL and backward(None) == m2.MAMBA2_ERR_NULL
    for name in ("q", "k", "v", "o", "lse"):
        for fn in (forward, backward):
            assert fn(adims(), **{name: None}) == m2.MAMBA2_ERR_NULL
            assert fn(adims(), **{name: OK + 8}) == m2.MAMBA2_ERR_ALIGN
    for name in ("do", "dq", "dk", "dv"):
        assert backward(adims(), **{name: None}) == m2.MAMBA2_ERR_NULL
    for name in ("qs", "ks"):
        assert forward(adims(), **{name: OK + 4}) == m2.MAMBA2_ERR_ALIGN
    # packed sides need their starts
    assert forward(adims(q_packed=True), ks=OK) == m2.MAMBA2_ERR_NULL
    assert forward(adims(k_packed=True), qs=OK) == m2.MAMBA2_ERR_NULL
    for flag in ("causal", "q_packed", "k_packed"):
        assert forward(_set(adims(), **{flag: 2})) == m2.MAMBA2_ERR_SHAPE
    assert forward(_set(adims(), reserved=1)) == m2.MAMBA2_ERR_SHAPE
    for fn, need in ((forward, m2.mamba2_attention_workspace_bytes(adims())),
                     (backward, m2.mamba2_attention_backward_workspace_bytes(adims()))):
        assert need >= 256
        assert fn(adims(), n=need - 1) == m2.MAMBA2_ERR_WORKSPACE
        assert fn(adims(), ws=None) == m2.MAMBA2_ERR_WORKSPACE
        assert fn(adims(), ws=OK + 16) == m2.MAMBA2_ERR_WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), m2.MAMBA2_ERR_DTYPE),
    (dict(batch=0), m2.MAMBA2_ERR_SHAPE),
    (dict(rows=0), m2.MAMBA2_ERR_SHAPE),
    (dict(prefix=-1), m2.MAMBA2_ERR_SHAPE),
    (dict(ngroups=3), m2.MAMBA2_ERR_SHAPE),
    (dict(headdim=12), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(scale=0.0), m2.MAMBA2_ERR_SHAPE),
    (dict(batch=1 << 16), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(rows=1 << 29), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(prefix=1 << 29), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(k_stride=132), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(batch=65535, nheads=256, ngroups=256), m2.MAMBA2_ERR_UNSUPPORTED),
])
def test_step_refuses_sizes(kw, status):
    d = sdims(**kw)
    assert step(d, kp=OK, vp=OK) == status
    assert m2.mamba2_last_error() != ""
    assert m2.mamba2_attention_step_workspace_bytes(d) == 0


def test_step_refuses_pointers():
    assert step(None) == m2.MAMBA2_ERR_NULL
    for name in ("q", "k", "v", "kc", "vc", "lens", "o"):
        assert step(sdims(), **{name: None}) == m2.MAMBA2_ERR_NULL
        assert step(sdims(), **{name: OK + 8}) == m2.MAMBA2_ERR_ALIGN
    assert step(sdims(prefix=8), kp=OK) == m2.MAMBA2_ERR_NULL
    assert step(sdims(prefix=8), vp=OK) == m2.MAMBA2_ERR_NULL
    need = m2.mamba2_attention_step_workspace_bytes(sdims(prefix=8))
    assert step(sdims(prefix=8), kp=OK, vp=OK, n=need - 1) == m2.MAMBA2_ERR_WORKSPACE


# --------------------------------------------------------- the wrappers' checks


def _refused(status, fn, *a, text=None, **kw):
    with pytest.raises(m2.Mamba2Error) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value
    if text:
        assert text in str(e.value)


def test_rotary_wrapper():
    q, k, inv = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.ones(32)
    f = m2.rotary_forward
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, inv, text="GPU")  # all else is right
    _refused(m2.MAMBA2_ERR_NULL, f, None, k, inv)
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, None)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, [1], inv)
    _refused(m2.MAMBA2_ERR_DTYPE, f, q.half(), k.half(), inv)
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k.bfloat16(), inv, text="k")
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k, inv.double(), text="inv_freq")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, torch.ones(4, 8))
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k[:, :4], inv)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q[:, :1].expand(2, 5, 4, 64), k, inv)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, inv, torch.zeros(2, 4, dtype=I32), text="positions")
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k, inv, torch.zeros(2, 5), text="positions")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, inv, torch.zeros(5, 2, dtype=I32).t(), text="positions")
    _refused(m2.MAMBA2_ERR_UNSUPPORTED, f, q, k, inv, layout="other")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, inv, scale="x")
    _refused(m2.MAMBA2_ERR_NULL, m2.rotary_backward, q, None, inv, text="GPU")


def test_attention_wrapper():
    q, k = torch.zeros(2, 5, 4, 64), torch.zeros(2, 7, 2, 64)
    f = m2.attention_forward
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, k, text="GPU")
    _refused(m2.MAMBA2_ERR_NULL, f, q, None, k)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, 3)
    _refused(m2.MAMBA2_ERR_DTYPE, f, q.half(), k.half(), k.half())
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k.bfloat16(), k, text="k")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k[:, :6])
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k[:1], k[:1])
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k[..., :32], k[..., :32])
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k[:, :1].expand(2, 7, 2, 64), k)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k.transpose(1, 2).contiguous().transpose(1, 2), k)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, k_lengths=torch.zeros(3, dtype=I32), text="k_seqs")
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k, k, q_lengths=torch.zeros(2, dtype=torch.int64))
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, q_starts=torch.zeros(3, dtype=I32))
    _refused(m2.MAMBA2_ERR_SHAPE, f, q[0], k, k, q_starts=torch.zeros(3, dtype=I32),
             q_lengths=torch.zeros(2, dtype=I32))
    _refused(m2.MAMBA2_ERR_SHAPE, f, q[0], k, k, q_starts=torch.zeros(1, dtype=I32))
    _refused(m2.MAMBA2_ERR_SHAPE, f, q[0], k, k, q_starts=[0, 5])
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, scale="x")
    _refused(m2.MAMBA2_ERR_WORKSPACE, f, q, k, k, workspace=5)
    b, lse = m2.attention_backward, torch.zeros(2, 5, 4)
    _refused(m2.MAMBA2_ERR_NULL, b, q, k, k, q, lse, q, text="GPU")
    _refused(m2.MAMBA2_ERR_SHAPE, b, q, k, k, q, lse[:, :4], q, text="lse")
    _refused(m2.MAMBA2_ERR_SHAPE, b, q, k, k, q, lse, q[:, :4], text="dout")
    _refused(m2.MAMBA2_ERR_DTYPE, b, q, k, k, q.bfloat16(), lse, q, text="o is")
    _refused(m2.MAMBA2_ERR_SHAPE, b, q, k, k, q, lse,
             q.transpose(1, 2).contiguous().transpose(1, 2), text="dout")


def test_step_wrapper():
    q, k, c = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64), torch.zeros(2, 9, 2, 64)
    n, p = torch.zeros(2, dtype=I32), torch.zeros(6, 2, 64)
    f = m2.attention_step
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, k, c, c, n, text="GPU")
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, k, c, c, n, p, p, text="GPU")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, c, c, n, p)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, c, c, n, p, p[:5], text="v_prefix")
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, c, c[:, :8], n, text="v_cache")
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, k, c, None, n)
    _refused(m2.MAMBA2_ERR_DTYPE, f, q, k, k, c, c, n.long(), text="lengths")
    _refused(m2.MAMBA2_ERR_NULL, f, q, k, k, c, c, None)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k[:, :1], c, c, n)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q, k, k, c[:, :1].expand(2, 9, 2, 64), c, n)
    _refused(m2.MAMBA2_ERR_SHAPE, f, q[:, :, :32], k, k, c, c, n)


# ------------------------------------------------------------------ frequencies


def test_frequencies():
    inv, scale = m2.rotary_frequencies(8, 10000.0)
    assert scale == 1.0
    assert torch.equal(inv, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64).float())
    lin, _ = m2.rotary_frequencies(8, 10000.0, scaling="linear", factor=4)
    assert torch.equal(lin, (inv.double() / 4).float()) or torch.allclose(lin, inv / 4, rtol=1e-7)
    base, _ = m2.rotary_frequencies(8, 10000.0, scaling="base", factor=4)
    assert base[0] == 1.0  # the fastest stays, the slowest is stretched by the factor
    assert abs(float(base[-1]) * 4 / float(inv[-1]) - 1) < 1e-6
    n = 4096
    parts, scale = m2.rotary_frequencies(64, 10000.0, scaling="parts", factor=8, original_length=n)
    plain, _ = m2.rotary_frequencies(64, 10000.0)
    assert abs(scale - (0.1 * math.log(8) + 1)) < 1e-12
    turns = plain.double() * n / (2 * math.pi)
    ratio = (plain / parts).double()
    assert (ratio[turns > 33 * 1.4] == 1).all()
    assert torch.allclose(ratio[turns < 0.7], torch.full_like(ratio[turns < 0.7], 8.0), rtol=1e-6)
    assert (ratio[1:] >= ratio[:-1] * (1 - 1e-6)).all()


@pytest.mark.parametrize("kw,status", [
    (dict(rotary=7), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=0), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=8, base=1.0), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=8, factor=0.5, scaling="linear"), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=8, scaling="other"), m2.MAMBA2_ERR_UNSUPPORTED),
    (dict(rotary=8, scaling="parts", factor=2), m2.MAMBA2_ERR_SHAPE),
    (dict(rotary=8, scaling="parts", factor=2, original_length=100, fast=1.0, slow=2.0),
     m2.MAMBA2_ERR_SHAPE),
])
def test_frequencies_refused(kw, status):
    _refused(status, m2.rotary_frequencies, **kw)


# -------------------------------------------------------------- the float64 forms


def test_reference_gradients_against_differences():
    """The formula's gradients against central differences in float64 (step 1e-5: the cubic term
    is below 1e-9 of these values, the subtraction's roundings below 1e-10)."""
    g = torch.Generator().manual_seed(5)
    h, gr, d, spans_q, spans_k = 4, 2, 8, [(0, 3), (3, 0), (3, 5)], [(1, 4), (5, 2), (7, 3)]
    q = torch.randn(9, h, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(10, gr, d, generator=g, dtype=torch.float64) for _ in range(2))
    dout = torch.randn(9, h, d, generator=g, dtype=torch.float64)

    def run(causal, *x):
        return ref.attention(*x, spans_q, spans_k, causal, 0.4, F32, dout)[0]

    for causal in (True, False):
        out = run(causal, q, k, v)
        for i, name in enumerate(("dq", "dk", "dv")):
            x = [q, k, v]
            for at in torch.randint(0, x[i].numel(), (12,), generator=g).tolist():
                vals = []
                for e in (1e-5, -1e-5):
                    y = [t.clone() for t in x]
                    y[i].view(-1)[at] += e
                    vals.append((run(causal, *y)["o"] * dout).sum())
                diff = float(vals[0] - vals[1]) / 2e-5
                assert abs(diff - float(out[name].view(-1)[at])) < 1e-7
        # rows that see nothing, rows of no sequence
        assert torch.isinf(out["lse"][8]).all() and (out["o"][8] == 0).all()
        if causal:  # 5 queries on 3 keys: the first two see none
            assert torch.isinf(out["lse"][3:5]).all() and (out["dq"][3:5] == 0).all()


@pytest.mark.skipif(shutil.which(HIPCC) is None and not os.path.exists(HIPCC),
                    reason="hipcc not available")
@pytest.mark.parametrize("name", ["attention", "attention_bwd", "attention_step"])
def test_loads_from_scalar_bases_have_their_wait_states(tmp_path, name):
    out = tmp_path / "k.s"
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops",
                    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "--cuda-device-only",
                    "-S", os.path.join(CSRC, name + ".hip"), "-o", str(out)],
                   check=True, capture_output=True)
    asm = out.read_text()
    assert "global_load_lds_dwordx4" in asm
    bad = _hazards(asm)
    assert not bad, bad[:4]
    # nothing spills: a load counted by hand would be joined by others
    assert not [s for s in asm.split(".vgpr_spill_count:")[1:] if int(s.split()[0])]

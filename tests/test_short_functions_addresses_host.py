"""The mamba2_* functions take addresses (whole numbers) in place of tensors; the
short functions do not: a length for all sequences, or a row number, given where
a tensor belongs would be read as an address on the device.  They are refused
with the package's error.  None of these calls launches a kernel."""
import pytest
import torch

import state_space_sequence_02_amd as m2

I32 = torch.int32


def refused(name, fn, *a, **kw):
    with pytest.raises(m2.Mamba2Error) as e:
        fn(*a, **kw)
    assert e.value.status == m2.MAMBA2_ERR_SHAPE and "not a tensor" in str(e.value), e.value
    assert f"{name} is a" in str(e.value), e.value


@pytest.mark.parametrize("v", [0, 16, 1 << 20, True])
def test_attention(v):
    q, k, lse = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 4)
    inv = torch.ones(32)
    for fn in (m2.rotary_forward, m2.rotary_backward):
        first = "dyq" if fn is m2.rotary_backward else "q"
        refused(first, fn, v, k, inv)
        refused(first.replace("q", "k"), fn, q, v, inv)
        refused("inv_freq", fn, q, k, v)
        refused("positions", fn, q, k, inv, v)
    for fn, rest in ((m2.attention_forward, ()), (m2.attention_backward, (q, lse, q))):
        for i, name in enumerate("qkv"):
            a = [q, k, k]
            a[i] = v
            refused(name, fn, *a, *rest)
        refused("q_lengths", fn, q, k, k, *rest, q_lengths=v)
        refused("k_lengths", fn, q, k, k, *rest, k_lengths=v)
        refused("q_starts", fn, q[0], k, k, *rest, q_starts=v)
        refused("k_starts", fn, q, k[0], k[0], *rest, k_starts=v)
    for i, name in enumerate(("o", "lse", "dout")):
        a = [q, lse, q]
        a[i] = v
        refused(name, m2.attention_backward, q, k, k, *a)
    n, p = torch.zeros(2, dtype=I32), torch.zeros(6, 2, 64)
    names = ("q", "k", "v", "k_cache", "v_cache", "lengths", "k_prefix", "v_prefix")
    for i, name in enumerate(names):
        a = [q[:, 0], k[:, 0], k[:, 0], k, k, n, p, p]
        a[i] = v
        refused(name, m2.attention_step, *a)


@pytest.mark.parametrize("v", [0, 16, 1 << 20, True])
def test_layer(v):
    x, w, c, st = torch.zeros(2, 8, 4), torch.zeros(4, 4), torch.zeros(4), torch.zeros(2, 3, 4)
    one = x[:, 0].contiguous()
    refused("weight", m2.conv1d_forward, x, v)
    refused("bias", m2.conv1d_forward, x, w, v)
    refused("init_state", m2.conv1d_forward, x, w, c, v)
    refused("lengths", m2.conv1d_forward, x, w, c, st, lengths=v)
    refused("bias", m2.conv1d_step, one, w, v, st)
    refused("state", m2.conv1d_step, one, w, c, v)
    refused("bias", m2.conv1d_backward, x, w, v, st, x)
    refused("init_state", m2.conv1d_backward, x, w, c, v, x)
    refused("dfinal", m2.conv1d_backward, x, w, c, st, x, v)
    refused("lengths", m2.conv1d_backward, x, w, c, st, x, st, lengths=v)
    A, bc, h = torch.zeros(4, 3), torch.zeros(2, 8, 1, 3), torch.zeros(2, 4, 3)
    names = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "init_state")
    for i, name in enumerate(names):
        a = [x, x, A, bc, bc, c, x, c, h]
        a[i] = v
        refused(name, m2.selective_scan_forward, *a)
        refused(name, m2.selective_scan_backward, *a, x, h)
        if i < 8:
            a = [t[:, 0] if torch.is_tensor(t) and t.dim() > 2 else t for t in a[:8]]
            refused(name, m2.selective_scan_step, *a, h)
    good = [x, x, A, bc, bc, c, x, c, h]
    refused("lengths", m2.selective_scan_forward, *good, lengths=v)
    refused("dy", m2.selective_scan_backward, *good, v)
    refused("dfinal", m2.selective_scan_backward, *good, x, v)
    refused("lengths", m2.selective_scan_backward, *good, x, h, lengths=v)
    refused("state", m2.selective_scan_step, one, one, A, bc[:, 0], bc[:, 0], c, one, c, v)
    for fn, rest in ((m2.norm_forward, ()), (m2.norm_backward, (x,))):
        refused("x", fn, v, c, c, x, *rest)
        refused("weight", fn, x, v, c, x, *rest)
        refused("bias", fn, x, c, v, x, *rest)
        refused("z", fn, x, c, c, v, *rest)
    refused("dy", m2.norm_backward, x, c, c, x, v)


def test_the_calls_without_them_are_right():
    """The same arguments with tensors come as far as the device's check."""
    q, k, lse = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 4)
    n, p = torch.zeros(2, dtype=I32), torch.zeros(6, 2, 64)
    x, w, c, st = torch.zeros(2, 8, 4), torch.zeros(4, 4), torch.zeros(4), torch.zeros(2, 3, 4)
    scan = [x, x, torch.zeros(4, 3), *[torch.zeros(2, 8, 1, 3)] * 2, c, x, c, torch.zeros(2, 4, 3)]
    for call in (lambda: m2.conv1d_forward(x, w, c, st, lengths=n),
                 lambda: m2.conv1d_backward(x, w, c, st, x, st, lengths=n),
                 lambda: m2.selective_scan_forward(*scan, lengths=n),
                 lambda: m2.selective_scan_backward(*scan, x, scan[-1], lengths=n),
                 lambda: m2.norm_backward(x, c, c, x, x),
                 lambda: m2.attention_forward(q, k, k, q_lengths=n, k_lengths=n),
                 lambda: m2.attention_backward(q, k, k, q, lse, q, q_lengths=n, k_lengths=n),
                 lambda: m2.attention_step(q[:, 0], k[:, 0], k[:, 0], k, k, n, p, p)):
        with pytest.raises(m2.Mamba2Error) as e:
            call()
        assert e.value.status == m2.MAMBA2_ERR_NULL and "GPU" in str(e.value), e.value

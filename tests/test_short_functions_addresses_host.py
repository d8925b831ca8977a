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


def test_the_calls_without_them_are_right():
    """The same arguments with tensors come as far as the device's check."""
    q, k, lse = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 4)
    n, p = torch.zeros(2, dtype=I32), torch.zeros(6, 2, 64)
    for call in (lambda: m2.attention_forward(q, k, k, q_lengths=n, k_lengths=n),
                 lambda: m2.attention_backward(q, k, k, q, lse, q, q_lengths=n, k_lengths=n),
                 lambda: m2.attention_step(q[:, 0], k[:, 0], k[:, 0], k, k, n, p, p)):
        with pytest.raises(m2.Mamba2Error) as e:
            call()
        assert e.value.status == m2.MAMBA2_ERR_NULL and "GPU" in str(e.value), e.value

"""The largest sizes that the header names as supported by the operators around
the SSD, and the first ones beyond them: sizes that are refused need no
workspace (0 bytes)."""
import pytest

import torch

import state_space_sequence_02_amd as m2

BF16 = torch.bfloat16


def _conv(b, n, c, stride=0):
    return m2.mamba2_conv1d_backward_workspace_bytes(
        m2.make_conv_dims(b, n, c, 4, None, BF16, x_stride=stride))


def _scan(b, n, ch, ns, g, stride=0):
    d = m2.make_scan_dims(b, n, ch, ns, g, BF16, b_stride=stride)
    fwd = m2.mamba2_selective_scan_workspace_bytes(d)
    assert (fwd > 0) == (m2.mamba2_selective_scan_backward_workspace_bytes(d) > 0)
    return fwd


def _norm(rows, ch, g, stride=0):
    return m2.mamba2_norm_backward_workspace_bytes(
        m2.make_norm_dims(rows, ch, g, BF16, z_stride=stride))


@pytest.mark.parametrize("of,last,beyond", [
    (_conv, (65535, 1, 8), (65536, 1, 8)),
    (_conv, (1, 1 << 30, 8), (1, (1 << 30) + 1, 8)),
    (_conv, (4, 1 << 28, 8), (4, (1 << 28) + 1, 8)),
    (_conv, (1, 8, 1 << 20), (1, 8, (1 << 20) + 4)),
    (_conv, (2, 8 * (1 << 14), 1 << 16), (2, 8 * (1 << 14) + 1, 1 << 16)),
    (_conv, (1, 8, 8, 1 << 24), (1, 8, 8, (1 << 24) + 4)),
    (_scan, (64, 16, 1 << 20, 16, 1), (65, 16, 1 << 20, 16, 1)),
    # workgroups: 64 channels of one group each
    (_scan, (1, 16 * 4095, 1 << 12, 1, 1 << 12), (1, 16 * 4096, 1 << 12, 1, 1 << 12)),
    (_scan, (1, 16 * 4095, 1 << 18, 2, 1), (1, 16 * 4096, 1 << 18, 2, 1)),
    (_scan, (1, 16 * 2047, 65 * 4096, 1, 4096), (1, 16 * 2048, 65 * 4096, 1, 4096)),
    # sums over channels
    (_scan, (2, 1 << 22, 64, 64, 1), (2, (1 << 22) + 1, 64, 64, 1)),
    (_scan, (1, 1 << 25, 16, 16, 1), (1, (1 << 25) + 1, 16, 16, 1)),
    (_scan, (2, 1 << 27, 1, 1, 1), (2, (1 << 27) + 1, 1, 1, 1)),
    (_scan, (1, 16, 64, 16, 1, 1 << 24), (1, 16, 64, 16, 1, (1 << 24) + 8)),
    (_norm, (1 << 30, 64, 1), ((1 << 30) + 1, 64, 1)),
    (_norm, (8, 1 << 20, 128), (8, (1 << 20) + 128, 128)),
    (_norm, (8, 8192, 1), (8, 8193, 1)),
    (_norm, (8, 64, 1, 1 << 24), (8, 64, 1, (1 << 24) + 8)),
], ids=str)
def test_documented_bounds(of, last, beyond):
    assert of(*last) >= 256
    assert of(*beyond) == 0
    assert m2.mamba2_last_error()

"""Attention takes its exponentials to base 2: scale * log2(e) has to be a
float32 number too, or every score is infinite or NaN (0 * infinity) where
the formula has one.  None of these calls launches a kernel."""
import ctypes

import pytest

import state_space_sequence_02_amd as m2
from test_attention_host import adims, backward, forward, rdims, rotary, sdims, step

LARGEST = 2.3586e38  # below the largest float32, 3.4028e38, over log2(e)


@pytest.mark.parametrize("scale", [2.3587e38, 3.0e38, 3.4028234e38])
def test_scales_beyond_float32_in_base_2(scale):
    assert ctypes.c_float(scale).value < float("inf")
    for status in (forward(adims(scale=scale)), backward(adims(scale=scale)), step(sdims(scale=scale))):
        assert status == m2.MAMBA2_ERR_UNSUPPORTED and "scale" in m2.mamba2_last_error()
    assert m2.mamba2_attention_workspace_bytes(adims(scale=scale)) == 0
    assert m2.mamba2_attention_backward_workspace_bytes(adims(scale=scale)) == 0
    assert m2.mamba2_attention_step_workspace_bytes(sdims(scale=scale)) == 0


def test_scales_within():
    for scale in (LARGEST, 1e-40):
        assert m2.mamba2_attention_workspace_bytes(adims(scale=scale)) >= 256
        assert m2.mamba2_attention_backward_workspace_bytes(adims(scale=scale)) >= 256
        assert m2.mamba2_attention_step_workspace_bytes(sdims(scale=scale)) >= 256
    # rotary's factor meets no exponential: refused for its pointer alone
    assert rotary(rdims(scale=3.4e38), q=None) == m2.MAMBA2_ERR_NULL

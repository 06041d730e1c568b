"""Ends of the prompt operators' argument ranges, before any CUDA call."""
import ctypes
import math

import pytest

import bit_ternary_weight_b200 as bl

A = 0x7f0000000000          # a 16-byte aligned address that is never read


def _attention(scale):
    q, k, v, out = (bl.HeadsC(A + 4096 * i, 8, 256, 128) for i in range(4))
    return bl.lib.bitlinear_attention_prefill(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), A, A, 2, 2, 2, 128,
                                              scale, ctypes.byref(out), A, 1 << 40, 0, None)


@pytest.mark.parametrize("scale", [2.36e38, 2.9e38, 3.0e38, 3.4e38])
def test_a_scale_that_is_infinite_in_base_two_is_refused(scale):
    assert scale * math.log2(math.e) > (2 - 2 ** -23) * 2.0 ** 127
    assert _attention(scale) == bl.BL_ERR_SHAPE


@pytest.mark.parametrize("scale", [1e-45, 1e-30, 128 ** -0.5, 1e30, 2.35e38])
def test_scales_in_range_pass_the_checks(scale):
    # no such memory: what is reported comes after the checks of the shape
    assert _attention(scale) not in (bl.BL_OK, bl.BL_ERR_SHAPE)

"""Scales that are refused: the kernels take the scores in log2 units, where the largest floats are infinite."""
import pytest

import sparse_mixture_experts_moe_gb300 as moe
from test_attention_host import cache, decode, prompt


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, float("inf"), 0.0, -1e-44])
def test_scales_without_a_finite_log2_form_are_refused(scale):
    assert prompt(scale=scale) == moe.MOE_ERR_INVALID_ARG
    assert decode(cache(), scale=scale) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [2.3e38, 1.0, 1e-38, 1e-44])
def test_others_are_not(scale):
    assert prompt(scale=scale, Tq=0, Tkv=0) == moe.MOE_OK
    assert decode(cache(), scale=scale, n=0) == moe.MOE_OK

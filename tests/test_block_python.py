"""Refusals of the operator plans' Python classes that need no device."""
import math

import pytest

import fft_circulant_attention_gb300 as cat


@pytest.mark.parametrize("scale", [0, 0.0, -0.5, math.nan])
def test_attn_plan_takes_no_scale_that_is_not_positive(scale):
    # (0 would be taken for the default.)
    with pytest.raises(ValueError, match="scale"):
        cat.AttnPlan(16, 1, 2, 2, 64, "bf16", scale=scale)

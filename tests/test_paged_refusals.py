"""What the paged calls and QuarotRope refuse."""
import math

import pytest
import torch

import w4a4_rotated_quantized_gb300 as q


@pytest.mark.parametrize("bad", [
    dict(base=math.inf), dict(base=math.nan), dict(factor=math.inf), dict(factor=math.nan),
    dict(scaling="smooth", factor=2.0, original_len=4096, low_freq=4.0, high_freq=4.0),
    dict(scaling="smooth", factor=2.0, original_len=4096, low_freq=4.0, high_freq=1.0),
    dict(scaling="smooth", factor=2.0, original_len=4096, low_freq=0.0),
    dict(scaling="yarn", factor=2.0, original_len=4096, beta_slow=0.0), dict(scaling="yarn", factor=2.0, original_len=4096, beta_fast=0.0),
    dict(scaling="yarn", factor=2.0, original_len=4096, beta_fast=0.5), dict(scaling="yarn", factor=2.0, original_len=-1)])
def test_frequencies_that_say_nothing(bad):
    with pytest.raises(q.QuarotError) as e:
        q.QuarotRope(64, device="cpu", **bad)
    assert e.value.status == 1


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn", "smooth"])
def test_frequencies_are_finite(scaling):
    for factor in (1.0, 8.0, 1e6):
        r = q.QuarotRope(64, scaling=scaling, factor=factor, original_len=4096, device="cpu")
        assert torch.isfinite(r.inv_freq).all() and (r.inv_freq > 0).all() and math.isfinite(r.scale)

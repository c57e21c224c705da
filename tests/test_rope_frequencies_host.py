"""What rope_frequencies refuses, and that what it returns is finite."""
import math

import pytest
import torch

import kda_recurrent_gb300 as K


@pytest.mark.parametrize("over", [
    dict(factor=0.5), dict(factor=math.inf), dict(factor=math.nan), dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(base=math.nan),
    dict(base=1e-300), dict(original_length=-1), dict(original_length=math.nan), dict(original_length=math.inf), dict(slow_turns=math.nan),
    dict(slow_turns=32.0), dict(slow_turns=-math.inf), dict(fast_turns=math.inf)])
def test_refused(over):
    with pytest.raises(ValueError):
        K.rope_frequencies(64, device="cpu", **{**dict(factor=2.0, original_length=8192), **over})


@pytest.mark.parametrize("rot", [0, 16, 64, 128])
@pytest.mark.parametrize("over", [dict(), dict(factor=4.0), dict(factor=4.0, original_length=1), dict(base=0.5), dict(base=1e7, factor=1e6)])
def test_finite(rot, over):
    f, magnitude = K.rope_frequencies(rot, device="cpu", **over)
    assert f.shape == (rot // 2,) and f.dtype == torch.float32 and torch.isfinite(f).all() and math.isfinite(magnitude)

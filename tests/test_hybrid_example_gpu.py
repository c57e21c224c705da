"""The hybrid serving example end to end: every step against a plain FP32 pass over the whole history (before
any eviction), then with a budget that makes it evict.

Tolerance: the two sides round the residual stream to BF16 after each of three layers, whose inputs differ by
the layers' own errors (5.9e-3 each at most): relL2 of the logits <= 3 x 5.9e-3 + 3 x 2^-8 = 3e-2."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_every_step_matches_a_plain_pass():
    import hybrid_serving
    r = hybrid_serving.serve(batch=2, new_tokens=5, budget=0, check=True)
    assert r["evictions"] == 0 and 0 < r["worst"] <= 3e-2, r["worst"]


def test_serving_with_a_budget():
    import hybrid_serving
    r = hybrid_serving.serve(batch=4, new_tokens=60, budget=64)
    assert r["evictions"] >= 1 and max(r["lens"]) <= 64 + 16
    assert torch.isfinite(r["logits"]).all()

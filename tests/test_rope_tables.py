"""Scaled frequencies whose ramp ends at the first pairs (no GPU)."""
import math

import pytest
import torch

import exact_attention_18_gb300 as fa
from exact_attention_18_gb300 import build as fab
from oracle import rope


@pytest.fixture(scope="module", autouse=True)
def lib():
    fab.build_library()
    return fa.load_library()


@pytest.mark.parametrize("original_len", [0.5, 3.0, 5.0, 6.2, 6.4, 7.0, 40.0, 200.0, 202.0, 1000.0])
@pytest.mark.parametrize("rot", [4, 16, 64])
def test_pairs_below_and_above_the_ramp(rot, original_len):
    """Each pair by its own turns: below slow_turns over the factor, above fast_turns as it is, else between."""
    factor, plain = 8.0, fa.rope_inv_freq(rot)[0]
    kw = dict(scaling="parts", factor=factor, original_len=original_len)
    got, ref = fa.rope_inv_freq(rot, **kw)[0], rope.inv_freq(rot, **kw)[0]
    assert torch.allclose(got, ref, rtol=1e-14, atol=0)
    turns = original_len * plain / (2 * math.pi)
    slow, fast = turns < 1, turns > 32
    assert torch.allclose(got[slow], plain[slow] / factor, rtol=1e-14, atol=0)
    assert torch.allclose(got[fast], plain[fast], rtol=1e-14, atol=0)
    assert bool(((got >= plain / factor * (1 - 1e-14)) & (got <= plain * (1 + 1e-14))).all())

"""The hybrid stack example: every layer kind, the append, the attention and the norms together."""
import os
import sys

import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,kv_heads", [("ra", 2), ("rrra", 1), ("aa", 6)])
def test_split_into_calls_gives_the_same_activations(layers, kv_heads):
    """The whole prompt at once, and in chunks and single tokens: the bf16 tolerance of the parity tests."""
    import hybrid_stack

    s = hybrid_stack.HybridStack(layers, kv_heads=kv_heads, seed=3)
    whole, parts = hybrid_stack.run(150, 100, 64, s)
    assert bool(torch.isfinite(whole).all())
    assert float((whole.double() - parts.double()).norm() / whole.double().norm()) <= 2e-2
    assert gdn.gdn_check_device_error() == 0

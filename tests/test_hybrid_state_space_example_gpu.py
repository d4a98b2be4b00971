"""The hybrid stack example with state space layers: the same tokens in chunks and one by one as in one call."""
import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers", ["s", "rsa", "sras"])
def test_state_space_layers_run_in_pieces(layers):
    from examples.hybrid_stack import HybridStack, run

    whole, parts = run(60, 40, 17, HybridStack(layers, heads=4, kv_heads=2, width=64, batch=3, max_tokens=64))
    assert whole.shape == parts.shape and bool(torch.isfinite(whole).all())
    # bf16 activations through the layers: products of other shapes round elsewhere
    assert float((whole.double() - parts.double()).norm() / whole.double().norm()) < 2e-2
    assert gdn.gdn_check_device_error() == 0

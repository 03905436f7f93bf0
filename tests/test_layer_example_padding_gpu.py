"""The layers of examples/layer.py: what lies behind a prompt's end reaches nothing."""
import pytest
import torch

from test_layer_example_gpu import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["ssd", "scan"])
def test_padding_reaches_no_state_and_no_real_token(kind):
    ex = example()
    torch.manual_seed(3)
    f32 = torch.float32
    layer = ex.SSDLayer(64, 4, 32, 64, dtype=f32) if kind == "ssd" else ex.ScanLayer(64, 96, dtype=f32)
    n = [40, 0, 17, 1]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    clean = torch.randn(4, 40, 64, device="cuda")
    spoiled = clean.clone()
    for i, k in enumerate(n):
        clean[i, k:] = 0
        spoiled[i, k:] = float("nan")
    want, cache = layer.forward(clean, lengths)
    got, dirty = layer.forward(spoiled, lengths)
    for a, b in zip(cache, dirty):
        assert torch.isfinite(b).all() and torch.equal(a, b)
    for i, k in enumerate(n):
        assert torch.equal(got[i, :k], want[i, :k])

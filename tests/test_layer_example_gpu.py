"""The layers of examples/layer.py: prompts and tokens against the whole sequence, and the
chained gradients against differences."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("layer_example", os.path.join(ROOT, "examples", "layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kind,dtype,bound", [
    # fp32: a few products of 64 .. 256 terms, 2^-24 each, the two orders of the scan: 1e-5 of the
    # output.  bf16: each of about six roundings of 2^-9 differs between the two forms.
    ("ssd", torch.float32, 2e-5), ("ssd", torch.bfloat16, 2e-2), ("scan", torch.float32, 2e-5),
    ("scan", torch.bfloat16, 2e-2)])
def test_prompt_then_tokens_is_the_whole_sequence(kind, dtype, bound):
    ex = example()
    torch.manual_seed(1)
    layer = ex.SSDLayer(64, 4, 32, 64, dtype=dtype) if kind == "ssd" else ex.ScanLayer(64, 96, dtype=dtype)
    u = torch.randn(3, 40, 64, device="cuda").to(dtype)
    lengths = torch.tensor([33, 1, 20], dtype=torch.int32, device="cuda")
    got, cache = ex.generate(layer, u, 33, lengths)
    whole, _ = layer.forward(u)
    for i, g in enumerate(got):
        w = whole[i, :len(g)].float()
        assert (g.float() - w).norm() <= bound * w.norm(), i


@pytest.mark.parametrize("kind", ["ssd", "scan"])
def test_training_step_against_differences(kind):
    """sum(out dout) along a random direction of every parameter: central difference in fp32.
    The loss of about 2000 terms is good to 1e-6 of its terms' norm, h = 1e-2 of the parameter's
    scale: 1e-4 of rounding and (1e-2)^2 of truncation, held to 2e-2 of the largest slope."""
    ex = example()
    torch.manual_seed(2)
    f32 = torch.float32
    layer = ex.SSDLayer(32, 2, 16, 16, dtype=f32) if kind == "ssd" else ex.ScanLayer(32, 48, 8, dtype=f32)
    u, dout = torch.randn(2, 37, 32, device="cuda"), torch.randn(2, 37, 32, device="cuda")
    keep = {}
    layer.forward(u, keep=keep)
    du, grads = layer.backward(dout, keep)

    def loss(x=u):
        return (layer.forward(x)[0].double() * dout.double()).sum().item()

    slopes = {}
    for name, g in list(grads.items()) + [("u", du)]:
        p = u if name == "u" else getattr(layer, name)
        v = torch.randn_like(p) * p.abs().mean()
        h, base = 1e-2, p.clone()
        ends = []
        for sign in (1, -1):
            p.copy_(base + sign * h * v)
            ends.append(loss())
        p.copy_(base)
        slopes[name] = ((ends[0] - ends[1]) / (2 * h), (g.double() * v.double()).sum().item(),
                        (g.double().norm() * v.double().norm()).item())
    for name, (want, got, scale) in slopes.items():
        assert abs(want - got) <= 2e-2 * max(abs(want), 0.1 * scale), (name, want, got, scale)

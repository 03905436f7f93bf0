"""The blocks of examples/layer.py, whose projections are in 8 bits: tokens against the whole
sequence, and the chained gradients against those of the same blocks without 8 bits."""
import importlib.util
import os

import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("layer_example", os.path.join(ROOT, "examples", "layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_tokens_are_the_whole_sequence():
    """Token by token, values differ by bf16 roundings (2^-9 each, some ten of them a block); where
    that moves one across a rounding border of e4m3 it moves by 2^-3 of itself, one value in 20 at
    most: 2^-3 / sqrt(20) = 3% of an operand's norm a product, four products: 6%."""
    ex = example()
    torch.manual_seed(3)
    blocks = [ex.SSDBlock(64, 4, headdim=32, dstate=64) for _ in range(2)]
    x = torch.randn(3, 40, 64, device="cuda").bfloat16()
    whole, _ = ex.stack(blocks, x)
    _, caches = ex.stack(blocks, x[:, :30])
    for t in range(30, 40):
        got = ex.stack_step(blocks, x[:, t], caches)
        assert (got - whole[:, t]).norm() <= 6e-2 * whole[:, t].norm()
    assert m2.device_error() == 0


def test_gradients_are_near_those_without_8_bits():
    """A rounding to e4m3 is at most 2^-4 of a value, evenly spread in sign and size: 2^-4 / sqrt(3) =
    3.6% of a tensor's norm.  A weight's gradient sees those of the forward operands (two products of
    two) and of the backward's (two products of two, x twice): ten, 11% together, held to twice that."""
    ex = example()
    torch.manual_seed(4)
    block = ex.SSDBlock(128, 4, headdim=32, dstate=64)
    x = torch.randn(2, 200, 128, device="cuda").bfloat16()
    res = torch.randn(2, 200, 128, device="cuda")
    dout, dtotal = torch.randn(2, 200, 128, device="cuda").bfloat16(), torch.randn(2, 200, 128, device="cuda")
    keep = {}
    out, total, _ = block.forward(x, res, keep=keep)
    dx, dres, g = block.backward(dout, dtotal, keep)
    plain, kept = ex.SSDLayer(128, 4, headdim=32, dstate=64), {}
    for name in ("w_in", "w_out", "w_conv", "b_conv", "A", "D", "dt_bias", "w_norm"):
        setattr(plain, name, getattr(block, name))
    u, t = m2.add_norm_fwd(x, res, block.w_pre)
    want, _ = plain.forward(u, keep=kept)
    du, ref = plain.backward(dout, kept)
    n = m2.add_norm_bwd(t, block.w_pre, du, dtotal)
    ref["w_pre"] = n["dw"]
    assert torch.equal(total, t)
    pairs = [("out", out, want), ("dx", dx, n["dx"]), ("dresidual", dres, n["dresidual"])]
    for name, got, r in pairs + [(k, g[k], ref[k]) for k in ref]:
        far = (got.float() - r.float()).norm() / r.float().norm()
        assert far <= 0.22, (name, far.item())
    assert m2.device_error() == 0


def test_main_runs(capsys):
    example().main()
    assert "blocks in 8 bits" in capsys.readouterr().out

"""The Python binding of the layer operators: what it refuses beside test_layer_gpu."""
import pytest
import torch

import mamba_ssd_chunked_02_gb300 as m2

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_a_width_beyond_32_bits_is_not_cut_down():
    x, w = torch.zeros(1, 2, 0, device="cuda"), torch.zeros(0, (1 << 32) + 4, device="cuda")
    with pytest.raises(m2.Mamba2Error, match="conv_fwd"):
        m2.conv_fwd(x, w)

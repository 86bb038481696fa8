"""Rules of the few-token serving operators beside their formulas: the state of
quantised modules, and what the packing calls refuse."""
import io

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build
from backward_tcgen05_tma_gb300.module import SwiGLUMLP
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@torch.no_grad()
def test_quantized_modules_through_a_file():
    torch.manual_seed(3)
    mlp = W4SwiGLUMLP(SwiGLUMLP(264, 136, device="cuda", gate_multiplier=1.5), group=32, zeros=True)
    moe = MoESwiGLU(264, 72, 6, 2, device="cuda").quantize(group=64)
    x = torch.randn(5, 264, device="cuda", dtype=torch.bfloat16)
    for m, new in ((mlp, W4SwiGLUMLP(device="cuda")), (moe, MoESwiGLU(264, 72, 6, 2, device="cuda"))):
        y = m(x)
        f = io.BytesIO()
        torch.save(m.state_dict(), f)
        f.seek(0)
        new.load_state_dict(torch.load(f, map_location="cpu", weights_only=True))
        assert torch.equal(new(x), y)
        new.cpu()
        assert new.down_w4.packed.device.type == "cpu"
        with pytest.raises(ValueError):
            new(x)
        assert torch.equal(new.cuda()(x), y)

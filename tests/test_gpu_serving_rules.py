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


@pytest.mark.parametrize("lead", [(), (3,)])
def test_zero_points_above_15_are_refused(lead):
    g = gen(2)
    c = torch.randint(0, 256, (*lead, 16, 64), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.ones(*lead, 16, 2, device="cuda", dtype=torch.float16)
    z = torch.randint(0, 16, (*lead, 16, 2), generator=g, device="cuda", dtype=torch.uint8)
    assert api.swiglu_mlp_w4_pack(c, s, z, 64).zeros
    z.view(-1)[-1] = 16  # some formats store a zero point less one and add it on loading
    with pytest.raises(ValueError, match="0..15"):
        api.swiglu_mlp_w4_pack(c, s, z, 64)
    with pytest.raises(ValueError, match="0..15"):
        W4SwiGLUMLP.from_codes((c, s, z), (c, s, z), 64)

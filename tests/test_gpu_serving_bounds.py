"""The debug build's index checks over sizes whose last tiles lie partly past
the matrix: the build skips an access outside its buffers and reports it."""
import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _debug_library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    prev = api.use_debug_library(True)
    yield
    api.use_debug_library(prev)


def packed(g, N, K, group, zeros, pair=False, experts=()):
    c = torch.randint(0, 256, (*experts, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((*experts, N, -(-K // group)), 0.01, device="cuda", dtype=torch.bfloat16)
    z = torch.full(s.shape, 7, device="cuda", dtype=torch.uint8) if zeros else None
    return api.swiglu_mlp_w4_pack(c, s, z, group, pair)


# an odd number of 16-row tiles (32-row tiles from 9 tokens on: the last is half
# past the matrix), and blocks that take one to many of them
@pytest.mark.parametrize("N", [16, 40, 2 * 32 * 152 + 16, 3 * 32 * 152 + 8, 7 * 32 * 152 + 1, 14 * 32 * 152 + 16])
@pytest.mark.parametrize("M,K,group,zeros", [(1, 72, 64, False), (8, 520, 32, True), (12, 264, 128, False),
                                             (16, 1096, 32, True), (20, 136, 64, False), (32, 584, 128, True),
                                             (40, 264, 32, False), (64, 200, 64, True)])
def test_w4_linear_stays_in_its_buffers(M, N, K, group, zeros):
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    assert torch.isfinite(api.swiglu_mlp_w4_linear(X, packed(g, N, K, group, zeros))).all()


@pytest.mark.parametrize("M,N,K", [(16, 8200, 8200), (12, 1000, 11008), (30, 4904, 4096), (24, 8, 20488)])
def test_w4_linear_over_clusters_stays_in_its_buffers(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    assert torch.isfinite(api.swiglu_mlp_w4_linear(X, packed(g, N, K, 64, True))).all()


# an odd number of tiles of 8 hidden units, of output tiles, or both
@pytest.mark.parametrize("M", [5, 9, 31, 50])
@pytest.mark.parametrize("D,H", [(24, 8), (264, 7304), (7304, 264), (8200, 4872)])
def test_w4_mlp_stays_in_its_buffers(M, D, H):
    g = torch.Generator(device="cuda").manual_seed(D)
    X = torch.randn(M, D, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    Y, A = api.swiglu_mlp_fwd_nograd_w4(X, packed(g, 2 * H, D, 64, False, True), packed(g, D, H, 64, False))
    assert torch.isfinite(Y).all() and torch.isfinite(A).all()


@pytest.mark.parametrize("four_bits", [False, True])
@pytest.mark.parametrize("T,D,H,E,k", [(1, 24, 8, 5, 2), (9, 2440, 264, 3, 2), (40, 264, 2824, 4, 3),
                                       (64, 1032, 520, 27, 8), (64, 72, 40, 512, 16)])
def test_moe_stays_in_its_buffers(T, D, H, E, k, four_bits):
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").mul_(s[-1] ** -0.5).to(torch.bfloat16)
    X, Wr = rnd(T, D), rnd(E, D)
    if four_bits:
        w = packed(g, 2 * H, D, 32, True, True, (E,)), packed(g, D, H, 32, True, False, (E,))
    else:
        w = rnd(E, 2 * H, D), rnd(E, D, H)
    Y, idx, wt = api.swiglu_mlp_moe_fwd_nograd(X, Wr, *w, k)
    assert torch.isfinite(Y).all() and int(idx.min()) >= 0 and int(idx.max()) < E

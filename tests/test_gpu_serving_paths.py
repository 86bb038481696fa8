"""The 4-bit products' less common paths (contractions split over clusters and
taken in phases, several runs of tiles a block, 17 to 32 columns), and calls
that follow one another closely: inputs that change, one workspace for all.

Tolerances, fixed before any run: those of test_gpu_serving_sums.py, u |y| and
(96 + K / 32) 2^-23 of the sum of the terms' magnitudes.  An MLP's output is
held to its own stored hidden values."""
import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def codes(g, lead, N, K, group, zeros, dtype):
    ng = -(-K // group)
    c = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(*lead, N, ng, generator=g, device="cuda") + 0.5).mul_(0.2 * K ** -0.5).to(dtype)
    z = torch.randint(0, 16, (*lead, N, ng), generator=g, device="cuda", dtype=torch.uint8)
    return c, s, z if zeros else None


def product64(x, w, group, rows=4096):
    """x W^T and |x| |W|^T in 64 bits, some rows of W at a time."""
    c, s, z = w
    ys, ts = [], []
    for i in range(0, c.shape[0], rows):
        part = slice(i, i + rows)
        q = torch.stack((c[part] & 15, c[part] >> 4), -1).flatten(-2).double()
        K = q.shape[-1]
        q -= 8.0 if z is None else z[part].double().repeat_interleave(group, -1)[..., :K]
        q *= s[part].double().repeat_interleave(group, -1)[..., :K]
        ys.append(x @ q.T)
        ts.append(x.abs() @ q.abs().T)
    return torch.cat(ys, 1), torch.cat(ts, 1)


def close(got, y, terms, u, K):
    assert bool(((got.double() - y).abs() <= u * y.abs() + (96 + K / 32) * 2.0 ** -23 * terms).all())


# on 152 SMs: blocks of a cluster x phases x runs of tiles in a block
@pytest.mark.parametrize("dtn,M,N,K,group,zeros", [
    ("bf16", 16, 8200, 40968, 64, True),    # 8 x 2 x 2
    ("f16", 31, 900, 20488, 128, False),    # 8 x 2 x 1
    ("bf16", 8, 600, 147464, 128, True),    # 8 x 3 x 1
    ("f16", 9, 40, 73736, 32, True),        # 8 x 2 x 1, fewer tiles than clusters
    ("bf16", 24, 2000, 4104, 128, False),   # 2 x 1 x 1
    ("f16", 24, 2000, 8192, 32, True),      # 4 x 1 x 1
    ("bf16", 20, 1000, 16448, 32, True),    # 8 x 1 x 1
    ("bf16", 12, 14000, 8200, 128, False),  # 2 x 1 x 1, many tiles
    ("bf16", 24, 66000, 496, 32, True),     # 1 x 1 x 2
    ("f16", 16, 70000, 264, 64, False),     # 1 x 1 x 2
    ("bf16", 5, 70008, 328, 128, True),     # 1 x 1 x 2
    ("f16", 29, 300, 1032, 32, False), ("bf16", 32, 4000, 2056, 128, False),
    ("f16", 18, 8000, 4096, 64, True), ("bf16", 17, 31, 4096, 32, True),
    # large ones on either side of the rule by which the tensor-core form takes
    # 17 to 32 tokens: rows x K x tokens (twice as many in groups of 32)
    ("f16", 32, 11016, 4104, 128, False), ("f16", 31, 11016, 4104, 128, False),
    ("bf16", 19, 4104, 18440, 64, True), ("bf16", 18, 4104, 18440, 64, True),
    ("bf16", 32, 21000, 4232, 32, True), ("bf16", 31, 21000, 4232, 32, True)])
def test_w4_linear_split_phased_and_in_runs(dtn, M, N, K, group, zeros):
    g = gen(M + N + K)
    w, X = codes(g, (), N, K, group, zeros, DT[dtn]), normal(g, M, K, dtype=DT[dtn])
    W = api.swiglu_mlp_w4_pack(*w, group)
    Y = api.swiglu_mlp_w4_linear(X, W)
    close(Y, *product64(X.double(), w, group), U[dtn], K)
    assert torch.equal(api.swiglu_mlp_w4_linear(X, W), Y)
    m = min(2, M - 1)  # a token's output does not depend on the ones beside it
    X2 = X.flip(0).contiguous()
    assert torch.equal(api.swiglu_mlp_w4_linear(X2, W)[M - 1 - m], Y[m])


@pytest.mark.parametrize("dtn,M,D,H,group,zeros", [
    ("bf16", 20, 16448, 200, 32, True),   # gate/up over clusters of 8
    ("f16", 31, 200, 20488, 128, False),  # down in phases
    ("bf16", 6, 81928, 600, 64, False)])  # gate/up over clusters, one column
def test_w4_mlp_split_and_phased(dtn, M, D, H, group, zeros):
    g = gen(M + D + H)
    gu, dn = codes(g, (), 2 * H, D, group, zeros, DT[dtn]), codes(g, (), D, H, group, zeros, DT[dtn])
    X = normal(g, M, D, dtype=DT[dtn])
    Y, A = api.swiglu_mlp_fwd_nograd_w4(X, api.swiglu_mlp_w4_pack(*gu, group, gate_up=True),
                                        api.swiglu_mlp_w4_pack(*dn, group))
    (gate, up), (tg, tu) = (t.chunk(2, 1) for t in product64(X.double(), gu, group))
    a = gate * torch.sigmoid(gate) * up
    n = (96 + D / 32) * 2.0 ** -23  # SiLU grows by at most 1.1 per unit of gate; 2^-20: the exponential
    tol = (U[dtn] + 2.0 ** -20) * a.abs() + 1.01 * n * (1.1 * tg * up.abs() + tu * gate.abs())
    assert bool(((A.double() - a).abs() <= tol + 1e-30).all())
    close(Y, *product64(A.double(), dn, group), U[dtn], H)


# ---------------------------------------------------------------------------
# calls that follow one another
# ---------------------------------------------------------------------------
OPS = ["w4_linear", "w4_mlp", "moe", "moe_w4"]


def operators(T, seed=0, D=1088, H=1600, N=12800):
    """Inputs, and each operator as a function of a workspace.  With 33 tokens and
    more the products' tiles are shared by blocks, two tiles a block at places."""
    g, dt, E, k = gen(seed), torch.bfloat16, 12, 3
    X, Wr = normal(g, T, D), normal(g, E, D, std=2 * D ** -0.5)
    lin = api.swiglu_mlp_w4_pack(*codes(g, (), N, D, 64, True, dt), 64)
    gu = api.swiglu_mlp_w4_pack(*codes(g, (), 2 * H, D, 128, False, dt), 128, gate_up=True)
    dn = api.swiglu_mlp_w4_pack(*codes(g, (), D, H, 128, False, dt), 128)
    h = 328
    e16 = normal(g, E, 2 * h, D, std=D ** -0.5), normal(g, E, D, h, std=h ** -0.5)
    e4 = (api.swiglu_mlp_w4_pack(*codes(g, (E,), 2 * h, D, 64, False, dt), 64, gate_up=True),
          api.swiglu_mlp_w4_pack(*codes(g, (E,), D, h, 64, False, dt), 64))
    ops = {
        "w4_linear": (lambda ws: (api.swiglu_mlp_w4_linear(X, lin, ws=ws),),
                      lambda: api.w4_linear_workspace(T, N, D, X.device)),
        "w4_mlp": (lambda ws: api.swiglu_mlp_fwd_nograd_w4(X, gu, dn, ws=ws),
                   lambda: api.w4_workspace(T, D, H, X.device)),
        "moe": (lambda ws: api.swiglu_mlp_moe_fwd_nograd(X, Wr, *e16, k, ws=ws),
                lambda: api.moe_workspace(T, D, h, E, k, X.device)),
        "moe_w4": (lambda ws: api.swiglu_mlp_moe_fwd_nograd(X, Wr, *e4, k, ws=ws),
                   lambda: api.moe_workspace(T, D, h, E, k, X.device)),
    }
    return X, ops


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T", [5, 20, 41, 64])
def test_calls_on_inputs_that_change(op, T):
    # launches overlap: partial tiles, token rows and hidden values of the call
    # before are still there, and must not be taken for this one's
    X, ops = operators(T)
    call, new_ws = ops[op]
    ws = new_ws()
    xs = [normal(gen(70 + i), *X.shape) for i in range(4)]
    want = []
    for x in xs:
        X.copy_(x)
        want.append([o.clone() for o in call(new_ws())])
        torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for x in xs:
            X.copy_(x)
            got.append(call(ws))
    torch.cuda.synchronize()
    assert all(same(o, want[i % 4]) for i, o in enumerate(got))
    assert not same(want[0], want[1])


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T", [20, 41, 64])
def test_graphs_on_inputs_that_change(op, T):
    if api._use_debug:
        pytest.skip("the binding waits for every call of the debug build, which a capture forbids")
    X, ops = operators(T)
    call, new_ws = ops[op]
    ws = new_ws()
    xs = [normal(gen(90 + i), *X.shape) for i in range(3)]
    want = []
    for x in xs:
        X.copy_(x)
        want.append([o.clone() for o in call(new_ws())])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # launches of one graph overlap as well
            out = call(ws)
    for i in (0, 1, 2, 0, 2, 1):
        X.copy_(xs[i])
        graph.replay()
        assert same(out, want[i])


def test_one_workspace_serves_all_calls_in_turn():
    mixes = [operators(64, 1), operators(40, 2, D=520, H=1416, N=20008), operators(9, 3, D=264, H=200, N=333),
             operators(20, 4, D=2056, H=4104, N=16400)]
    calls = [(ops[name][0], ops[name][1]()) for _, ops in mixes for name in OPS]
    want = [[o.clone() for o in call(ws)] for call, ws in calls]
    torch.cuda.synchronize()
    one = torch.zeros(max(ws.numel() for _, ws in calls), dtype=torch.uint8, device="cuda")
    order = torch.randperm(len(calls) * 4, generator=torch.Generator().manual_seed(5)).tolist()
    got = [(i % len(calls), calls[i % len(calls)][0](one)) for i in order]
    torch.cuda.synchronize()
    assert all(same(out, want[i]) for i, out in got)
    assert api.swiglu_mlp_query_error(one) == 0

"""Rules of the layer norm and the linear layers that need no GPU to be checked:
launch plans at every size, what the build rebuilds, the order of waits and
accesses in the kernels' sources, the modules' defaults."""
import os
import re
import subprocess

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, block, build, module
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, PackedW4, W4SwiGLUMLP

PLANS = r"""
#include <algorithm>
#include <cstdio>
#include "tc_plan.h"
#include "simt_plan.h"
using namespace swiglu;
#define HOLD(what) if (!(what)) { printf("%s: line %d at %lld %lld %lld\n", #what, __LINE__, (long long)a, (long long)b, (long long)c); return 1; }
int main() {
  const int64_t sizes[] = {0, 1, 2, 4, 7, 8, 9, 16, 44, 75, 76, 77, 151, 152, 153, 300, 2047, 16384, 1 << 20};
  // tiles, blocks of k, SMs
  for (int64_t a : sizes) for (int64_t b : sizes) for (int c : {1, 75, 76, 148, 152, 256}) {
    const TcPlan p = tc_plan(a, b, c);
    HOLD(p.grid >= std::min<int64_t>(a, 1) && p.grid <= c);
    HOLD(p.sk_tiles >= 0 && p.sk_tiles < c && p.sk_tiles <= a && p.seg_max >= 1);
    HOLD(a > 0 || (p.grid == 0 && p.sk_tiles == 0));
    HOLD(p.sk_tiles == 0 || p.grid * (int64_t)(p.seg_max - 1) * b >= (int64_t)p.sk_tiles * b);
  }
  // rows, columns, k of an fp32 product
  const int64_t more[] = {0, 1, 4, 8, 9, 12, 31, 32, 33, 64, 132, 1000, 2048, 9004, 120000};
  for (int64_t a : more) for (int64_t b : more) for (int64_t c : more) {
    const SlPlan p = sl_plan(a, b, c, 152);
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    HOLD((int64_t)p.m_tiles * 16 * p.tm >= a && (int64_t)p.n_tiles * SL_BN >= b);
    HOLD(p.parts >= 1 && p.per >= SL_BK && p.per % SL_BK == 0 && (int64_t)p.parts * p.per >= c);
    HOLD(p.whole >= 0 && p.whole <= tiles && (p.parts > 1 || p.whole == tiles));
    HOLD(p.parts == 1 || (int64_t)(p.parts - 1) * p.per < c);  // no part is empty
  }
  return 0;
}
"""


def test_plans_hold_at_every_size(tmp_path):
    # an empty batch among them: the sizes of its backward pass's workspace come
    # from the same plans (a division by zero ends the process on some machines)
    (tmp_path / "plans.cpp").write_text(PLANS)
    exe = str(tmp_path / "plans")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=integer-divide-by-zero",
                    "-fno-sanitize-recover=all", "-I", build.CSRC, "-I", build.CSRC_BLOCK, "-o", exe,
                    str(tmp_path / "plans.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_an_object_is_rebuilt_for_every_file_that_it_includes(tmp_path):
    # as the compiler lists them; an older object would stay in the library unseen
    for src in build.SOURCES:
        out = str(tmp_path / "deps")
        subprocess.run([build._nvcc(), *build.NVCC_FLAGS, "-MM", src, "-o", out], check=True)
        with open(out) as f:
            named = f.read().split(":", 1)[1].replace("\\\n", " ").split()
        named = {os.path.normpath(os.path.join(build.ROOT, n)) for n in named}
        ours = {n for n in named if n.startswith(build.ROOT + os.sep)}
        known = {os.path.normpath(d) for d in build._deps(src)}
        assert len(ours) > 3 and ours <= known, sorted(ours - known)


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_a_sublayers_norm_takes_after_4_bit_weights(device):
    # their packed bytes are a buffer, so there is no parameter to go by
    packed = lambda n, k, pair: PackedW4(api.W4Weights(torch.zeros(64, dtype=torch.uint8, device=device), n, k, 64,
                                                       False, pair, torch.float16, None))
    w4 = W4SwiGLUMLP()
    w4.gate_up_w4, w4.down_w4 = packed(32, 72, True), packed(72, 16, False)
    norm = block.MLPBlock(w4).norm
    assert norm.weight.dtype is torch.float16 and norm.weight.device.type == device and norm.hidden_size == 72
    norm = block.MLPBlock(w4, hidden_size=72, dtype=torch.bfloat16, device="cpu").norm
    assert norm.weight.dtype is torch.bfloat16 and norm.weight.device.type == "cpu"
    moe = MoESwiGLU(72, 16, 4, 2, dtype=torch.float16, device=device)
    moe._experts_w4(packed(32, 72, True), packed(72, 16, False))
    norm = block.MLPBlock(moe).norm
    assert norm.weight.dtype is torch.float16 and norm.weight.device.type == device and norm.hidden_size == 72
    # empty until a state is loaded: the place is known, the sizes are not
    empty = block.MLPBlock(W4SwiGLUMLP(device=device), hidden_size=72)
    assert empty.norm.weight.device.type == device
    with pytest.raises(RuntimeError):
        block.MLPBlock(W4SwiGLUMLP())


def test_forward_mode_is_refused_by_every_layer():
    # a dual tensor that does not require a gradient, with and without recording;
    # (CPU tensors: what is not refused for its tangent is a ValueError)
    x, w, v = torch.zeros(4, 64), torch.zeros(64, 64), torch.zeros(64)
    pair, down = torch.zeros(192, 64), torch.zeros(64, 96)
    w4 = W4SwiGLUMLP(device="cpu")
    moe, mlp = MoESwiGLU(64, 96, 4, 2), module.SwiGLUMLP(64, 96, dtype=torch.float32)
    mlp._packed = (x, mlp._weights_state())
    fs = [lambda d: block.layer_norm(d(x)), lambda d: block.layer_norm(x, d(v)), lambda d: block.layer_norm(x, v, d(v)),
          lambda d: block.layer_norm(x, residual=d(x)), lambda d: block.linear(d(x), w), lambda d: block.linear(x, d(w)),
          lambda d: block.linear(x, w, d(v)), lambda d: block.linear(x, w, residual=d(x)),
          lambda d: block.mlp(d(x), w, v, w, v), lambda d: block.mlp(x, w, v, d(w), v),
          lambda d: block.mlp(x, w, v, w, v, residual=d(x)), lambda d: module.swiglu_mlp(d(x), pair, down),
          lambda d: module.swiglu_mlp(x, pair, d(down)), lambda d: mlp(d(x)), lambda d: w4(d(x)), lambda d: moe(d(x))]
    ad = torch.autograd.forward_ad
    for f in fs:
        for recording in (True, False):
            with ad.dual_level(), torch.set_grad_enabled(recording):
                with pytest.raises(RuntimeError, match="forward-mode"):
                    f(lambda t: ad.make_dual(t, torch.ones_like(t)))
    with ad.dual_level(), pytest.raises(ValueError):  # a level without tangents is nothing to refuse
        block.linear(x, w)


# kernels that are launched before the one in front of them has ended: file, kernel,
# its arguments' structures, what waits
EARLY = [("csrc_block/layer_norm.cuh", "ln_fwd_kernel", ["LnFwdArgs"], "pdl_wait();"),
         ("csrc_block/layer_norm.cuh", "ln_bwd_kernel", ["LnBwdArgs"], "pdl_wait();"),
         ("csrc_block/column_sums.cuh", "dact_kernel", ["DactArgs"], "pdl_wait();"),
         ("csrc_block/column_sums.cuh", "column_sum_kernel", ["ColumnSumArgs"], "pdl_wait();"),
         ("csrc_block/linear_few.cuh", "linear_few_kernel", ["LfArgs"], "pdl_wait();"),
         ("csrc_block/linear_mid.cuh", "linear_mid_kernel", ["LmArgs"], "pdl_wait();"),
         ("csrc/tc_gemm.cuh", "tc_gemm_kernel", ["TcShape"], "tc_begin(s);"),
         ("csrc/tc2_gemm.cuh", "tc2_gemm_kernel", ["TcShape"], "tc_begin(s);")]
ACCESS = (r"\btma_load|\btma_store|\bcp16\(|\bld_stream\(|\bld\.global|\bst\.global|cp\.async|\bprefetch\.global|__ldcg|"
          r"__ldg|\batomic|\bred\.")


def without_comments(name):
    with open(os.path.join(build.HERE, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def pointers_of(text, struct):
    body = text[text.index("struct %s {" % struct):]
    return re.findall(r"\*\s*(\w+)\s*;", body[:body.index("\n};")])


def before_the_wait(text, kernel, wait):
    """A kernel's body up to its wait."""
    at = re.search(r"__global__[^;{]*\b%s\(" % kernel, text).end()
    at = text.index(") {", at)
    return text[at:text.index(wait, at)]


def accesses(head, pointers):
    """What a kernel's head does with global memory, but for descriptors."""
    found = re.findall(ACCESS, head) + re.findall(r"\b(?:a|s|ep)\.(?:%s)\b" % "|".join(pointers), head)
    return found + re.findall(r"\bep\.\w+", head)


@pytest.mark.parametrize("name,kernel,structs,wait", EARLY, ids=[e[1] for e in EARLY])
def test_early_kernels_touch_nothing_before_their_wait(name, kernel, structs, wait):
    text = without_comments(name)
    defined = text + without_comments("csrc/tc_gemm.cuh")
    pointers = [p for s in structs for p in pointers_of(defined, s)]
    assert len(pointers) >= 3
    head = before_the_wait(text, kernel, wait)
    assert accesses(head, pointers) == []
    # the same check sees a read that is planted there
    for planted in ("const float x = a.%s[0];" % pointers[0], "tma_load_2d(s, &tmX, full(0), 0, 0);",
                    "x = *s.%s;" % pointers[-1], 'asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));'):
        assert accesses(head + planted, pointers) != []
    # the wait is every thread's: at the body's own level
    assert head.count("{") - head.count("}") == 1


def test_what_waits_waits_first():
    # tc_begin waits where the launch was early; TMEM that a kernel beside it may
    # still ask for is not asked for before the wait
    text = without_comments("csrc/tc_gemm.cuh")
    body = text[text.index("void tc_begin("):]
    body = body[:body.index("\n}\n")]
    assert re.search(r"if \(s\.early\) \{\s*pdl_wait\(\);\s*pdl_launch_dependents\(\);", body)
    assert body.index("pdl_wait") < body.index("*s.err")
    mid = without_comments("csrc_block/linear_mid.cuh")
    assert "tmem_alloc" not in before_the_wait(mid, "linear_mid_kernel", "pdl_wait();")
    assert mid.index("tmem_alloc(") < mid.index("pdl_launch_dependents();")
    # and every launch of this part that is early is of one of the kernels above
    host = without_comments("csrc_block/block.cu")
    started = set(re.findall(r"\b(\w+_kernel)\b", host))
    plain = {"simt_rows_kernel", "simt_linear_kernel", "simt_sum_kernel"}
    assert started - plain == {e[1] for e in EARLY if e[0].startswith("csrc_block")}
    for name in plain:
        assert re.findall(r"%s<[^;]*?>(<<<|\()" % name, host) and not re.search(r"auto kern = %s" % name, host)


def test_outputs_may_be_changed_in_place(monkeypatch):
    # as nn.Linear's may: the outputs that autograd hands out are no views.  The
    # calls are restated on the host, as there is no GPU here.
    def put(out, name, value):
        t = out[name] if out and out.get(name) is not None else torch.empty_like(value)
        return t.copy_(value)

    def norm_fwd(X, weight, bias, eps, residual=None, out=None, stats=True):
        S = X if residual is None else put(out, "S", X + residual)
        mean, rstd = S.mean(1), S.var(1, correction=0).add(eps).rsqrt()
        return put(out, "Y", (S - mean[:, None]) * rstd[:, None]), S, mean, rstd

    def linear_fwd(X, W, bias=None, activation="none", residual=None, keep=False, out=None, ws=None):
        return put(out, "Y", X @ W.T), X @ W.T if keep else None
    monkeypatch.setattr(api, "swiglu_mlp_layer_norm_fwd", norm_fwd)
    monkeypatch.setattr(api, "swiglu_mlp_linear_fwd", linear_fwd)
    monkeypatch.setattr(api, "swiglu_mlp_fwd", lambda X, *a, **k: (put(a[2] if len(a) > 2 else None, "Y", X), X))
    w, pair, down = torch.randn(64, 64), torch.randn(192, 64), torch.randn(64, 96)
    for shape in ((4, 64), (2, 3, 64), (64,), (2, 0, 64)):
        x = torch.randn(shape, requires_grad=True)
        for y in (block.layer_norm(x), *block.layer_norm(x, residual=x), block.linear(x, w, None, "relu"),
                  block.mlp(x, w, None, w, None), module.swiglu_mlp(x, pair, down)):
            ref = y.detach().clone()
            assert y.shape == shape and y.requires_grad
            y += 1
            assert torch.equal(y, ref + 1)


def test_rows_start_where_the_calls_can_read_them():
    # contiguous slices that start inside 16 bytes
    buf = torch.arange(8 * 64 + 8, dtype=torch.float32).to(torch.bfloat16)
    x = buf[3:3 + 8 * 64].view(8, 64)
    assert x.is_contiguous() and x.data_ptr() % 16
    for rows in (module.rows_of(x, 64), module.rows_of(x.view(2, 4, 64), 64), block._grad_rows(x.view(4, 2, 64), 64, x.dtype)):
        assert rows.data_ptr() % 16 == 0 and torch.equal(rows, x)
    y = buf[:8 * 64].view(8, 64)
    assert module.rows_of(y, 64).data_ptr() == y.data_ptr()  # nothing to move


def test_the_binding_names_what_is_missing():
    x, w, v = torch.zeros(4, 64), torch.zeros(64, 64), torch.zeros(4)
    for name, call in (("X", lambda: api.swiglu_mlp_layer_norm_fwd(None)), ("X", lambda: api.swiglu_mlp_linear_fwd(None, w)),
                       ("W", lambda: api.swiglu_mlp_linear_fwd(x, None)),
                       ("dY", lambda: api.swiglu_mlp_layer_norm_bwd(None, x, None, v, v)),
                       ("S", lambda: api.swiglu_mlp_layer_norm_bwd(x, None, None, v, v)),
                       ("mean", lambda: api.swiglu_mlp_layer_norm_bwd(x, x, None, None, v)),
                       ("rstd", lambda: api.swiglu_mlp_layer_norm_bwd(x, x, None, v, None)),
                       ("dY", lambda: api.swiglu_mlp_linear_bwd(None, x, w)), ("X", lambda: api.swiglu_mlp_linear_bwd(x, None, w)),
                       ("W", lambda: api.swiglu_mlp_linear_bwd(x, x, None))):
        with pytest.raises(ValueError, match=r": %s is needed" % name):
            call()

"""Calls that the header allows at its edges: a process whose first call is a
captured one, very wide rows, both outputs of a norm over its inputs (needs a
B200).  Tolerances as in test_gpu_linear and test_gpu_norm."""
import os
import subprocess
import sys

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests import test_gpu_linear, test_gpu_norm
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
from sparse_mixture_experts_noisy_b200 import moe
g = torch.Generator(device="cuda")
g.manual_seed(1)
n, d_in, d_out, dtype = {n}, {d_in}, {d_out}, torch.{dtype}
x, dy = torch.randn(n, d_in, generator=g, device="cuda").to(dtype), torch.randn(n, d_out, generator=g, device="cuda").to(dtype)
W = (torch.randn(d_out, d_in, generator=g, device="cuda") / d_in ** 0.5).to(dtype)

def step():
    h, s, mean, rstd = moe.moe_layer_norm(x, residual=x, want_stats=True)
    y, z = moe.moe_linear(h, W, act=moe.ACT_GELU, keep_z=True)
    b = moe.moe_linear_backward(dy, h, W, act=moe.ACT_GELU, z=z)
    c = moe.moe_layer_norm_backward(b["dx"], s, mean, rstd)
    return [h, s, y, z, *b.values(), *c.values()]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert moe.check_linear_status() == (0, 0)
print("same")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,d_in,d_out", [(3, 256, 264), (50, 512, 1000), (3000, 1024, 2048), (700, 333, 77)])
def test_first_call_of_a_process_is_captured(n, d_in, d_out, dtype):
    require_gpu()
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, n=n, d_in=d_in, d_out=d_out, dtype=dtype)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", (r.returncode, r.stdout[-500:], r.stderr[-2000:])


DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


@DTYPES
@pytest.mark.parametrize("shape", [(1, 1000003, 3), (6, 1000000, 5), (70, 300008, 9), (1, 5, 1000003), (6, 8, 1000000),
                                   (70, 9, 300008)], ids=lambda s: "x".join(map(str, s)))
def test_long_and_wide_products(shape, dtype):
    require_gpu()
    t = test_gpu_linear.make(*shape, dtype, seed=sum(shape))
    for act in ("gelu", "none"):
        _, z = test_gpu_linear.check_forward(t, act)
        test_gpu_linear.check_backward(t, z, act)
    assert moe.check_linear_status() == (0, 0)


@DTYPES
@pytest.mark.parametrize("n,d", [(1, 1000003), (3, 1000000), (2, 4000001)])
def test_very_wide_norms(n, d, dtype):
    require_gpu()
    t = test_gpu_norm.make(n, d, dtype, seed=d)
    _, h, mean, rstd = test_gpu_norm.check_forward(t, n, d, dtype, t["gamma"], t["beta"], True)
    test_gpu_norm.check_backward(t, h, mean, rstd, n, d, dtype, t["gamma"], True)


@DTYPES
@pytest.mark.parametrize("d", [768, 1001, 4096, 9000, 40000])
def test_both_outputs_of_a_norm_in_place(d, dtype):
    require_gpu()
    t = test_gpu_norm.make(300, d, dtype, seed=d + 2)
    want = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], residual=t["res"])
    for y, s in (("x", "res"), ("res", "x")):
        c = {q: v.clone() for q, v in t.items()}
        got = moe.moe_layer_norm(c["x"], t["gamma"], t["beta"], residual=c["res"], y=c[y], sum_out=c[s])
        assert got[0] is c[y] and got[1] is c[s]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@DTYPES
def test_block_without_rows(dtype):
    """An empty batch: empty outputs, zero gradients of the weights."""
    require_gpu()
    d, E, f = 64, 4, 128
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    layer = moe.MoELayer(r(E, d), r(E, f, d).to(dtype), r(E, d, f).to(dtype), 2, 1.25)
    block = moe.MoEBlock(layer, shared=(r(96, d).to(dtype), r(96), r(d, 96).to(dtype), None))
    x = torch.empty(0, d, device="cuda", dtype=dtype)
    assert [o.shape for o in block(x, x)] == [(0, d), (0, d)]
    s, m, saved = block.train(x, x)
    assert s.shape == m.shape == (0, d)
    g = block.backward(x, x, saved)
    assert g.pop("dx").shape == (0, d)
    assert len(g) == 10 and not any(bool(v.any()) for v in g.values())


@DTYPES
def test_blocks_on_two_streams(dtype):
    """Two blocks with layers of their own, forward and backward on two streams at
    once and joined by events, give the bits of one after the other."""
    require_gpu()
    d, E, f, n = 256, 8, 320, 500

    def make(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        layer = moe.MoELayer(r(E, d) / 16, (r(E, f, d) / 16).to(dtype), (r(E, d, f) / 18).to(dtype), 2, 1.25)
        shared = ((r(384, d) / 16).to(dtype), r(384), (r(d, 384) / 20).to(dtype), r(d))
        return moe.MoEBlock(layer, shared=shared, shared_act=moe.ACT_GELU), r(n, d).to(dtype), r(n, d).to(dtype)

    def run(block, x, ds):
        s, m, saved = block.train(x, x)
        g = block.backward(ds, ds, saved)
        return [s, m, *(g[q] for q in sorted(g))]

    sets = [make(1), make(2)]
    want = [run(*t) for t in sets]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(10):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append(run(*sets[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
    assert moe.check_linear_status() == (0, 0)

"""A captured layer keeps its workspace when the layer grows (needs a B200)."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def make(N, d=256, E=8, d_ff=512, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    layer = moe.MoELayer(r(E, d), (r(E, d_ff, d) / 16).bfloat16(), (r(E, d, d_ff) / 23).bfloat16(), 2, 1.25)
    return layer, r(N, d).bfloat16(), r(8 * N, d).bfloat16()


@pytest.mark.parametrize("block", [False, True], ids=["layer", "block"])
def test_replay_after_a_larger_batch(block):
    """The larger batch takes a new workspace.  The graph's one must not go back to
    the allocator, whose next user would find the replay's intermediates in it."""
    require_gpu()
    layer, x, big = make(700)
    b = moe.MoEBlock(layer)
    run = (lambda: torch.cat(b(x))) if block else (lambda: layer(x))
    want = run().clone()
    size = layer.workspace.numel()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    layer(big)
    assert layer.workspace.numel() > size
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((o == 7).all()) for o in others)
    # the next capture takes the larger one
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        got2 = run()
    for g, out in ((graph, got), (graph2, got2), (graph, got)):
        g.replay()
        assert torch.equal(out, want)

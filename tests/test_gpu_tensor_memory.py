"""Kernels that hold tensor memory while their clusters wait, on two streams at
once: routers of many experts (all 512 columns) beside dense layers of few tiles
(up to 256 columns and half an SM's shared memory).  Needs a B200."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [16, 32, 64, 80, 96, 128, 130, 160])
@pytest.mark.parametrize("N", [64, 700, 5000])
def test_router_beside_dense_layer(E, N):
    require_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(E + N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, W_g = r(N, 1024).bfloat16(), r(E, 1024)
    u, W = r(200, 1024).bfloat16(), (r(1024, 1024) / 32).bfloat16()
    route = lambda s=None: moe.moe_route(x, W_g, 2, stream=s)  # noqa: E731
    dense = lambda s=None: moe.moe_linear(u, W, stream=s)  # noqa: E731
    want = route(), dense()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(50):
        for s, f in zip(streams, (route, dense)):
            with torch.cuda.stream(s):
                got.append(f())
    for _ in range(20):   # in one stream, each the other's dependent
        got += [route(), dense()]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        if i % 2:
            assert torch.equal(out, want[1])
        else:
            assert all(torch.equal(a, b) for a, b in zip(out, want[0]))
    assert moe.check_linear_status() == (0, 0) and moe.check_route_status() == (0, 0)

"""Router and backward calls that launch the same kernel with different amounts
of shared memory, from two host threads (needs a B200)."""
import ctypes
import threading

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def randn(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


class Route:
    def __init__(self, E, N=1100, d=64, k=2):
        r = randn(E)
        self.x, self.W = r(N, d), r(E, d)
        self.out = [torch.empty(N, k, dtype=torch.int32, device="cuda"), torch.empty(N, k, device="cuda")]
        self.dims = N, d, E, k

    def bind(self, stream):
        L, p = moe.load_library(), moe._p
        args = (p(self.x), 0, p(self.W), None, None, 0.0, *self.dims, None, p(self.out[0]), p(self.out[1]),
                ctypes.c_void_p(stream.cuda_stream))
        return lambda: L.moe_route(*args)


class Backward:
    def __init__(self, E, N=40, d=32, d_ff=16, k=2):
        r = randn(E)
        self.x, self.W_g, self.W_up, self.W_down, self.dy = r(N, d), r(E, d), r(E, d_ff, d), r(E, d, d_ff), r(N, d)
        self.topk, self.gates, _ = moe.moe_route(self.x, self.W_g, k)
        self.dsp = moe.moe_dispatch(self.topk, self.x, E, None)
        self.o, self.H = moe.moe_expert_ffn_train(self.dsp["x_gathered"], self.dsp["offsets"], self.dsp["counts"],
                                                  self.W_up, self.W_down)
        self.dims = N, d, E, d_ff, k, self.dsp["rows"]
        self.ws = moe.new_workspace(moe.load_library().moe_backward_workspace_size(*self.dims, 0), "cuda")
        self.out = [torch.empty_like(t) for t in (self.x, self.W_g)] + [torch.empty(E, device="cuda")]
        self.out += [torch.empty_like(t) for t in (self.W_up, self.W_down)]

    def bind(self, stream):
        L, p, q = moe.load_library(), moe._p, self.dsp
        args = (p(self.x), 0, p(self.W_g), p(self.W_up), p(self.W_down), *self.dims, p(self.topk), p(self.gates),
                p(q["slot"]), p(q["offsets"]), p(q["counts"]), p(q["x_gathered"]), p(self.H), p(self.o), p(self.dy),
                *(p(o) for o in self.out), p(self.ws), self.ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        return lambda: L.moe_backward(*args)


@pytest.mark.parametrize("kind,counts", [(Route, (256, 130)), (Backward, (256, 100))], ids=["route", "backward"])
def test_two_threads_of_one_kernel(kind, counts):
    require_gpu()
    calls = [kind(E) for E in counts]
    want = []
    for c in calls:
        assert c.bind(torch.cuda.current_stream())() == 0
        torch.cuda.synchronize()
        want.append([o.clone() for o in c.out])
        for o in c.out:
            o.zero_()
    torch.cuda.synchronize()
    said = [set(), set()]
    start = threading.Barrier(2)

    def work(k):
        s = torch.cuda.Stream()
        call = calls[k].bind(s)
        start.wait()
        for _ in range(20):
            for _ in range(500):
                if call() != 0:
                    said[k].add(moe.load_library().moe_last_error().decode())
            s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert said == [set(), set()]
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c.out, w))

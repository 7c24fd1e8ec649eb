"""Calls of the dense layer that launch the same kernel with different amounts
of shared memory, from two host threads and from one captured graph (needs a
B200)."""
import ctypes
import threading

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def make(n, d_in, d_out, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(n, d_in).to(dtype), (r(d_out, d_in) / d_in ** 0.5).to(dtype), r(n, d_out).to(dtype)


class Forward:
    """y = x W^T of a few tokens, through the C call with buffers of its own."""

    def __init__(self, n, d_in, d_out, dtype):
        self.x, self.W, _ = make(n, d_in, d_out, dtype, seed=n)
        self.dims = n, d_in, d_out
        self.dt = moe._dt(self.x)
        need = moe.load_library().moe_linear_workspace_size(n, d_in, d_out, self.dt)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        self.out = [torch.empty(n, d_out, dtype=dtype, device="cuda")]

    def bind(self, stream):
        L, p = moe.load_library(), moe._p
        args = (p(self.x), self.dt, p(self.W), None, 0, None, *self.dims, p(self.out[0]), None, p(self.ws),
                self.ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        return lambda: L.moe_linear(*args)


class Backward:
    """dx and dW, through the C call with buffers of its own."""

    def __init__(self, n, d_in, d_out, dtype):
        self.x, self.W, self.dy = make(n, d_in, d_out, dtype, seed=n + 1)
        self.dims = n, d_in, d_out
        self.dt = moe._dt(self.x)
        need = moe.load_library().moe_linear_backward_workspace_size(n, d_in, d_out, 0, self.dt)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        self.out = [torch.empty_like(self.x), torch.empty_like(self.W)]

    def bind(self, stream):
        L, p = moe.load_library(), moe._p
        args = (p(self.dy), p(self.x), self.dt, p(self.W), None, 0, *self.dims, p(self.out[0]), p(self.out[1]), None,
                p(self.ws), self.ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        return lambda: L.moe_linear_backward(*args)


# Each pair runs one kernel with operands in both orders: tiles of 16 rows (a
# forward, or a dx, of a few tokens; a dW of a few columns) and of 32.
BF16, F32 = torch.bfloat16, torch.float32
PAIRS = {
    "bf16, 16 rows": (Forward, (12, 512, 2048), Backward, (14, 512, 16), BF16),
    "bf16, 32 rows": (Forward, (20, 512, 1024), Backward, (300, 256, 264), BF16),
    "f32, 16 rows": (Backward, (9, 272, 5696), Backward, (14, 512, 16), F32),
    "f32, 32 rows": (Forward, (20, 512, 1024), Backward, (300, 256, 264), F32),
}


def calls_of(name):
    f, a, g, b, dtype = PAIRS[name]
    return [f(*a, dtype), g(*b, dtype)]


def expected(calls):
    """Each call's outputs when it runs alone; the buffers are cleared again."""
    want = []
    for c in calls:
        assert c.bind(torch.cuda.current_stream())() == 0
        torch.cuda.synchronize()
        want.append([o.clone() for o in c.out])
        for o in c.out:
            o.zero_()
    torch.cuda.synchronize()
    return want


def same(call, want):
    return all(torch.equal(a, b) for a, b in zip(call.out, want))


@pytest.mark.parametrize("name", PAIRS)
def test_two_threads_of_one_type(name):
    """Calls as fast as two threads can make them, on two streams: no error, the bits of a call alone."""
    require_gpu()
    calls = calls_of(name)
    want = expected(calls)
    said = [set(), set()]
    start = threading.Barrier(2)

    def work(k):
        s = torch.cuda.Stream()
        call = calls[k].bind(s)
        start.wait()
        for _ in range(40):
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
    assert all(same(c, w) for c, w in zip(calls, want))
    assert moe.check_linear_status() == (0, 0)


@pytest.mark.parametrize("name", PAIRS)
def test_both_in_one_graph(name):
    require_gpu()
    calls = calls_of(name)
    want = expected(calls)
    for order in ((0, 1, 0), (1, 0, 1)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for k in order:
                assert calls[k].bind(torch.cuda.current_stream())() == 0
        for _ in range(3):
            for c in calls:
                for o in c.out:
                    o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(same(c, w) for c, w in zip(calls, want))
    assert moe.check_linear_status() == (0, 0)

"""The first call that a host thread makes is one of the library's: no other
CUDA call has made the device's context current in that thread (needs a B200)."""
import ctypes
import threading

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

N, D, E, F = 64, 256, 8, 512


def buffers():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    b = dict(x=r(N, D).bfloat16(), W_g=r(E, D), W_up=(r(E, F, D) / 16).bfloat16(), W_down=(r(E, D, F) / 16).bfloat16(),
             W=(r(F, D) / 16).bfloat16(), y=torch.zeros(N, D, device="cuda").bfloat16(),
             u=torch.zeros(N, F, device="cuda").bfloat16(), dW=torch.zeros(F, D, device="cuda").bfloat16(),
             topk=torch.zeros(N, 2, dtype=torch.int32, device="cuda"), gates=torch.zeros(N, 2, device="cuda"))
    b["dy"] = r(N, F).bfloat16()
    return b, moe.new_workspace(1 << 26, "cuda")


def calls(b, ws, s):
    L, p, n = moe.load_library(), moe._p, ws.numel()
    return {
        "linear": (lambda: L.moe_linear(p(b["x"]), 1, p(b["W"]), None, 0, None, N, D, F, p(b["u"]), None, p(ws), n, s),
                   ("u",)),
        "linear_backward": (lambda: L.moe_linear_backward(p(b["dy"]), p(b["x"]), 1, p(b["W"]), None, 0, N, D, F,
                                                          p(b["y"]), p(b["dW"]), None, p(ws), n, s), ("y", "dW")),
        "layer_norm": (lambda: L.moe_layer_norm(p(b["x"]), None, 1, None, None, 1e-5, N, D, p(b["y"]), None, None, None,
                                                s), ("y",)),
        "route": (lambda: L.moe_route(p(b["x"]), 1, p(b["W_g"]), None, None, 0.0, N, D, E, 2, None, p(b["topk"]),
                                      p(b["gates"]), s), ("topk", "gates")),
        "forward": (lambda: L.moe_forward(p(b["x"]), 1, p(b["W_g"]), None, None, 0.0, N, D, E, F, 2, float("inf"),
                                          p(b["W_up"]), p(b["W_down"]), p(b["y"]), None, None, None, None, None, p(ws), n,
                                          s), ("y",)),
    }


@pytest.mark.parametrize("name", ["linear", "linear_backward", "layer_norm", "route", "forward"])
def test_first_call_of_a_thread(name):
    require_gpu()
    b, ws = buffers()
    call, outs = calls(b, ws, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))[name]
    torch.cuda.synchronize()
    said = []

    def work():
        code = call()
        said.append((code, moe.load_library().moe_last_error().decode() if code else ""))

    th = threading.Thread(target=work)
    th.start()
    th.join()
    assert said == [(0, "")]
    torch.cuda.synchronize()
    got = [b[o].clone() for o in outs]
    assert call() == 0
    torch.cuda.synchronize()
    assert all(torch.equal(g, b[o]) for g, o in zip(got, outs)) and any(bool(g.any()) for g in got)

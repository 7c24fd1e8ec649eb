"""What callers of the layer norm and the dense layer may and may not pass, and
calls from two host threads at once (needs a B200)."""
import threading

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def t(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


def test_refusals():
    require_gpu()
    x, W, f = t(12, 64), t(40, 64), torch.ones(64, device="cuda")
    wide = t(12, 128)
    cases = [
        (lambda: moe.moe_layer_norm(wide[:, :64]), ValueError),                        # rows apart
        (lambda: moe.moe_layer_norm(x.half()), TypeError),
        (lambda: moe.moe_layer_norm(x, f.bfloat16()), ValueError),                     # gamma is fp32
        (lambda: moe.moe_layer_norm(x, f[:63].contiguous()), ValueError),
        (lambda: moe.moe_layer_norm(x, residual=x.float()), ValueError),
        (lambda: moe.moe_layer_norm(x, residual=x[:11]), ValueError),
        (lambda: moe.moe_layer_norm(x, sum_out=x), ValueError),                        # no residual
        (lambda: moe.moe_layer_norm(x, eps=0.0), moe.MoeError),
        (lambda: moe.moe_layer_norm(x.flatten()[1:1 + 11 * 64].view(11, 64)), moe.MoeError),  # 16-byte alignment
        (lambda: moe.moe_layer_norm(x, residual=x, y=wide.view(24, 64)[:12], sum_out=wide.view(24, 64)[:12]),
         moe.MoeError),
        (lambda: moe.moe_layer_norm(x[0]), ValueError),
        (lambda: moe.moe_layer_norm_backward(x, x, None, None), ValueError),
        (lambda: moe.moe_layer_norm_backward(x, x, f[:12].contiguous(), f[:11].contiguous()), ValueError),
        (lambda: moe.moe_layer_norm_backward(x, x, f[:12].contiguous(), f[:12].contiguous(),
                                             ws=torch.empty(16, dtype=torch.uint8, device="cuda")), moe.MoeError),
        (lambda: moe.moe_linear(x, W.float()), ValueError),                            # one type
        (lambda: moe.moe_linear(x, W.t()), ValueError),
        (lambda: moe.moe_linear(x, t(40, 63)), ValueError),
        (lambda: moe.moe_linear(x, W, b=f), ValueError),
        (lambda: moe.moe_linear(x, W, residual=x), ValueError),
        (lambda: moe.moe_linear(x, W, act=3), moe.MoeError),
        (lambda: moe.moe_linear(x, W, y=t(12, 41)), ValueError),
        (lambda: moe.moe_linear(x, W.cpu()), ValueError),
        (lambda: moe.moe_linear(x, W, ws=torch.empty(64, device="cuda")), ValueError),  # uint8
        (lambda: moe.moe_linear_backward(t(12, 40), x, W, act=moe.ACT_GELU), moe.MoeError),   # no z
        (lambda: moe.moe_linear_backward(t(12, 41), x, W), ValueError),
        (lambda: moe.moe_linear_backward(t(12, 40), x, W, act=moe.ACT_RELU, z=t(11, 40)), ValueError),
        (lambda: moe.moe_linear_backward(t(12, 40).cpu(), x, W), ValueError),
    ]
    for i, (call, error) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"case {i} was not refused")


def test_two_threads_at_once():
    """Each thread on its own stream; every result equals the one computed alone."""
    require_gpu()
    ins = [(t(500, 1001, dtype=d), t(700, 1001, dtype=d), t(500, 700, dtype=d)) for d in (torch.bfloat16, torch.float32)]

    def run(x, W, dy, stream=None):
        n, h, mean, rstd = moe.moe_layer_norm(x, residual=x, want_stats=True, stream=stream)
        y, z = moe.moe_linear(n, W, act=moe.ACT_GELU, keep_z=True, stream=stream)
        g = moe.moe_linear_backward(dy, n, W, act=moe.ACT_GELU, z=z, stream=stream)
        b = moe.moe_layer_norm_backward(g["dx"], h, mean, rstd, stream=stream)
        return [n, h, y, z, g["dW"], g["db"], b["dx"], b["dgamma"], b["dbeta"]]

    want = [run(*i) for i in ins]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[k].append(run(*ins[k], stream=s))
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for k in (0, 1):
        for r in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[k]))
    assert moe.check_linear_status() == (0, 0)

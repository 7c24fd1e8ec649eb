"""The dense layer's status word (needs a B200): a wait that ran out is reported
by check_linear_status, once, whatever clean calls lie between."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

TIMEOUT = 6


def step(n, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x = torch.randn(n, 256, generator=g, device="cuda").to(dtype)
    W = (torch.randn(264, 256, generator=g, device="cuda") / 16).to(dtype)
    y, z = moe.moe_linear(x, W, act=moe.ACT_GELU, keep_z=True)
    return [y, z, *moe.moe_linear_backward(y, x, W, act=moe.ACT_GELU, z=z).values()]


@pytest.mark.parametrize("n", [1, 40, 300, 6000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_report_survives_clean_calls(n, dtype):
    require_gpu()
    assert moe.check_linear_status() == (0, 0)
    want = step(n, dtype)
    moe.debug_linear_wait_timeout(5000)
    got = step(n, dtype)
    assert all(torch.equal(a, b) for a, b in zip(got, want))   # the report stops no later call
    code, word = moe.check_linear_status()
    assert code == TIMEOUT and word & 1 and not word & 2, (code, hex(word))
    assert moe.check_linear_status() == (0, 0)                 # read once, then cleared


def test_words_are_apart():
    """The report is in the dense layer's word alone, and another stream's read finds it."""
    require_gpu()
    ws = moe.new_workspace(256, "cuda")
    moe.check_route_status()
    side = torch.cuda.Stream()
    moe.debug_linear_wait_timeout(5000, stream=side)
    side.synchronize()
    assert moe.check_status(ws) == (0, 0) and moe.check_route_status() == (0, 0)
    assert moe.check_linear_status()[0] == TIMEOUT
    moe.debug_wait_timeout(5000, ws)
    assert moe.check_linear_status() == (0, 0) and moe.check_status(ws)[0] == TIMEOUT


def test_refusals():
    require_gpu()
    for us in (0, 2000001):
        with pytest.raises(moe.MoeError, match="timeout_us"):
            moe.debug_linear_wait_timeout(us)


def test_reports_made_while_another_stream_reads():
    """Reads on one stream while reports arrive from another: each is found by one of the reads."""
    require_gpu()
    assert moe.check_linear_status() == (0, 0)
    side = torch.cuda.Stream()
    for _ in range(50):
        moe.debug_linear_wait_timeout(200, stream=side)
        done, found = False, 0
        while not done:
            done = side.query()          # asked first: the last read comes after the report
            found += moe.check_linear_status()[0] == TIMEOUT
        assert found == 1

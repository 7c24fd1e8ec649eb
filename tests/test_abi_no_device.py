"""A valid call in a process without a GPU returns MOE_ERR_CUDA with a message
and leaves the process alive (CPU only: the device is hidden)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = {
    "linear": "L.moe_linear(A, DT, B, None, 2, None, N, 64, 64, C, None, W, BIG, None)",
    "linear_backward": "L.moe_linear_backward(A, B, DT, C, D, 2, N, 64, 64, E, F, G, W, BIG, None)",
    # no pass over dy in front of the products
    "linear_backward_products": "L.moe_linear_backward(A, B, DT, C, None, 0, N, 64, 64, E, F, None, W, BIG, None)",
    "layer_norm": "L.moe_layer_norm(A, None, DT, None, None, 1e-5, N, 64, B, None, C, D, None)",
    "layer_norm_backward": "L.moe_layer_norm_backward(A, B, DT, None, C, D, None, N, 64, E, F, G, W, BIG, None)",
    "route": "L.moe_route(A, DT, B, None, None, 0.0, N, 64, 8, 2, None, C, D, None)",
    "expert_ffn": "L.moe_expert_ffn(A, B, C, D, E, DT, 128, 64, 64, 8, F, W, BIG, None)",
    "forward": "L.moe_forward(A, DT, B, None, None, 0.0, N, 64, 8, 64, 2, 1.0, C, D, E, None, None, None, None, None,"
               " W, BIG, None)",
    "debug_linear_wait_timeout": "L.moe_debug_linear_wait_timeout(10, None)",
    "check_linear_status": "L.moe_check_linear_status(None, None)",
}

SCRIPT = """
import ctypes, sys
sys.path.insert(0, {root!r})
from sparse_mixture_experts_noisy_b200 import moe
from sparse_mixture_experts_noisy_b200.build import build
build()
L = moe.load_library()
assert L.moe_num_sms() == 0   # the addresses below must never reach a GPU
P, BIG = ctypes.c_void_p, 1 << 40
A, B, C, D, E, F, G, W = (P(i << 32) for i in range(1, 9))
for DT in (0, 1):
    for N in (1, 4, 40, 5000):
        code = {call}
        assert code == 4, (DT, N, code)
        assert L.moe_last_error()
print("refused")
"""


def test_wait_diagnostic_limits():
    from sparse_mixture_experts_noisy_b200 import moe
    from sparse_mixture_experts_noisy_b200.build import build
    build()
    for us in (0, 2000001):
        assert moe.load_library().moe_debug_linear_wait_timeout(us, None) == 1


@pytest.mark.parametrize("name", sorted(CALLS))
def test_error_code_without_a_device(name):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, call=CALLS[name])], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", (r.returncode, r.stdout[-500:], r.stderr[-2000:])

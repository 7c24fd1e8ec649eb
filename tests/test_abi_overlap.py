"""moe_layer_norm, moe_linear and their backward passes refuse outputs that
overlap an input or one another, in part too, and accept the overlaps that
include/moe.h allows (CPU only: the device is hidden, so an accepted call ends
with MOE_ERR_CUDA)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import ctypes, itertools, sys
sys.path.insert(0, {root!r})
from sparse_mixture_experts_noisy_b200 import moe
from sparse_mixture_experts_noisy_b200.build import build
build()
L = moe.load_library()
assert L.moe_num_sms() == 0   # the addresses below must never reach a GPU
N, D, O = {N}, {D}, {O}
V = lambda a: None if a is None else ctypes.c_void_p(a)

def norm(p, es, dt):
    size = dict(x=N * D * es, residual=N * D * es, gamma=4 * D, beta=4 * D, y=N * D * es, sum_out=N * D * es, mean=4 * N,
                rstd=4 * N)
    call = lambda a: L.moe_layer_norm(V(a["x"]), V(a["residual"]), dt, V(a["gamma"]), V(a["beta"]), 1e-5, N, D, V(a["y"]),
                                      V(a["sum_out"]), V(a["mean"]), V(a["rstd"]), None)
    return size, ("y", "sum_out", "mean", "rstd"), {{(a, b) for a in ("y", "sum_out") for b in ("x", "residual")}}, call

def norm_bwd(p, es, dt):
    need = L.moe_layer_norm_backward_workspace_size(N, D, dt)
    size = dict(dy=N * D * es, h=N * D * es, dres=N * D * es, gamma=4 * D, mean=4 * N, rstd=4 * N, dx=N * D * es,
                dgamma=4 * D, dbeta=4 * D, ws=need)
    call = lambda a: L.moe_layer_norm_backward(V(a["dy"]), V(a["h"]), dt, V(a["gamma"]), V(a["mean"]), V(a["rstd"]),
                                               V(a["dres"]), N, D, V(a["dx"]), V(a["dgamma"]), V(a["dbeta"]), V(a["ws"]),
                                               need, None)
    return size, ("dx", "dgamma", "dbeta", "ws"), {{("dx", b) for b in ("dy", "h", "dres")}}, call

def linear(p, es, dt):
    need = L.moe_linear_workspace_size(N, D, O, dt)
    size = dict(x=N * D * es, W=O * D * es, b=4 * O, residual=N * O * es, y=N * O * es, z_out=N * O * es, ws=need)
    call = lambda a: L.moe_linear(V(a["x"]), dt, V(a["W"]), V(a["b"]), 2, V(a["residual"]), N, D, O, V(a["y"]),
                                  V(a["z_out"]), V(a["ws"]), need, None)
    return size, ("y", "z_out", "ws"), {{("y", "residual")}}, call

def linear_bwd(p, es, dt):
    need = L.moe_linear_backward_workspace_size(N, D, O, 2, dt)
    size = dict(dy=N * O * es, x=N * D * es, W=O * D * es, z=N * O * es, dx=N * D * es, dW=O * D * es, db=4 * O, ws=need)
    call = lambda a: L.moe_linear_backward(V(a["dy"]), V(a["x"]), dt, V(a["W"]), V(a["z"]), 2, N, D, O, V(a["dx"]),
                                           V(a["dW"]), V(a["db"]), V(a["ws"]), need, None)
    return size, ("dx", "dW", "db", "ws"), set(), call

tried = 0
for make in (norm, norm_bwd, linear, linear_bwd):
    for dt, es in ((0, 4), (1, 2)):
        size, outs, same, call = make(None, es, dt)
        apart = {{q: (i + 1) << 32 for i, q in enumerate(size)}}
        assert call(apart) == 4, (make.__name__, L.moe_last_error())
        for o in outs:
            for q in size:
                if q == o or size[o] == 0 or size[q] == 0:
                    continue
                step = -(-max(size[o], size[q]) // 16) * 16
                for by in (0, 16, -16, step, -step):
                    inside = by < size[q] if by >= 0 else -by < size[o]
                    a = dict(apart)
                    a[o] = a[q] + by
                    fine = not inside or (by == 0 and (o, q) in same)
                    code = call(a)
                    tried += 1
                    assert code == (4 if fine else 1), (make.__name__, dt, o, q, by, code, L.moe_last_error())
                    assert fine or b"overlap" in L.moe_last_error() or b"input" in L.moe_last_error() or \\
                        b"different arrays" in L.moe_last_error()
assert tried > 300
print("refused")
"""


@pytest.mark.parametrize("N,D,O", [(40, 64, 64), (3, 200, 72), (100, 101, 7)], ids=lambda v: str(v))
def test_overlaps(N, D, O):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, N=N, D=D, O=O)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", (r.returncode, r.stdout[-500:], r.stderr[-2000:])


def test_no_rows_keep_the_weights():
    """Without rows the gradients of the weights are still written, so they must not be the weights."""
    script = SCRIPT[:SCRIPT.index("N, D, O =")].format(root=ROOT) + """
P = ctypes.c_void_p
W, G = P(1 << 32), P(2 << 32)
assert L.moe_linear_backward(None, None, 1, W, None, 0, 0, 64, 64, None, W, None, G, 1 << 30, None) == 1
assert b"overlap" in L.moe_last_error() or b"input" in L.moe_last_error()
assert L.moe_layer_norm_backward(None, None, 1, W, None, None, None, 0, 64, None, W, None, G, 1 << 30, None) == 1
assert b"overlap" in L.moe_last_error()
print("refused")
"""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", (r.returncode, r.stdout[-500:], r.stderr[-2000:])

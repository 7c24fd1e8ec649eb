"""moe_layer_norm, moe_linear and their backward passes refuse bad arguments on
the host, before anything is launched (CPU only), in C and in the binding."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe

P = ctypes.c_void_p
A, B = P(0x10000), P(0x20000)
ODD = P(0x10004)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from sparse_mixture_experts_noisy_b200.build import build
    build()
    return moe.load_library()


def _err(L):
    return L.moe_last_error().decode()


def test_layer_norm_arguments(L):
    def call(x=A, res=None, dt=1, gamma=A, beta=A, eps=1e-5, N=4, d=8, y=B, s=None, mean=A, rstd=A):
        return L.moe_layer_norm(x, res, dt, gamma, beta, eps, N, d, y, s, mean, rstd, None)

    for bad in (dict(dt=2), dict(N=-1), dict(d=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(y=None), dict(x=ODD), dict(gamma=ODD), dict(beta=ODD),
                dict(mean=ODD), dict(rstd=ODD), dict(res=ODD, s=A), dict(N=1 << 31)):
        assert call(**bad) == 1, bad
    assert call(d=(1 << 30) + 1, N=1) == 1 and "2^30" in _err(L)
    assert call(res=A) == 1 and "sum_out" in _err(L)
    assert call(s=A) == 1 and "sum_out must be NULL" in _err(L)
    assert call(res=A, s=B) == 1 and "different arrays" in _err(L)
    assert call(N=0, x=None, y=None) == 0


def test_layer_norm_backward_arguments(L):
    need = L.moe_layer_norm_backward_workspace_size(100, 64, 1)
    assert need > 0
    assert L.moe_layer_norm_backward_workspace_size(-1, 64, 1) == 0
    assert L.moe_layer_norm_backward_workspace_size(1, 0, 1) == 0

    def call(dy=A, h=A, dt=1, gamma=A, mean=A, rstd=A, dres=None, N=100, d=64, dx=B, dg=B, db=B, ws=A, n=need):
        return L.moe_layer_norm_backward(dy, h, dt, gamma, mean, rstd, dres, N, d, dx, dg, db, ws, n, None)

    for bad in (dict(dt=-1), dict(N=-1), dict(d=0), dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None),
                dict(dx=None), dict(dx=ODD), dict(dg=ODD), dict(db=ODD), dict(dres=ODD), dict(gamma=ODD)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 3 and call(n=need - 1) == 3 and "workspace" in _err(L)
    assert call(ws=ODD) == 1


def test_linear_arguments(L):
    need = L.moe_linear_workspace_size(100, 64, 48, 0)

    def call(x=A, dt=0, W=A, b=None, act=0, res=None, N=100, d_in=64, d_out=48, y=B, z=None, ws=A, n=BIG):
        return L.moe_linear(x, dt, W, b, act, res, N, d_in, d_out, y, z, ws, n, None)

    for bad in (dict(dt=3), dict(N=-1), dict(d_in=0), dict(d_out=0), dict(act=3), dict(act=-1), dict(x=None),
                dict(W=None), dict(y=None), dict(x=ODD), dict(W=ODD), dict(y=ODD), dict(z=ODD), dict(b=ODD),
                dict(res=ODD), dict(ws=ODD)):
        assert call(**bad) == 1, bad
    assert call(z=B) == 1 and "different arrays" in _err(L)
    for wide in (dict(d_in=(1 << 30) + 1), dict(d_out=(1 << 30) + 1)):
        assert call(N=1, **wide) == 1 and "2^30" in _err(L)
        assert L.moe_linear_workspace_size(1, wide.get("d_in", 8), wide.get("d_out", 8), 0) == 0
    if need:
        assert call(ws=None) == 3 and call(n=need - 1) == 3
    assert call(N=0, x=None, y=None) == 0
    assert L.moe_linear_workspace_size(-1, 64, 48, 0) == 0 and L.moe_linear_workspace_size(1, 64, 0, 0) == 0


def test_linear_backward_arguments(L):
    need = L.moe_linear_backward_workspace_size(100, 64, 48, 2, 0)
    assert need > 0

    def call(dy=A, x=A, dt=0, W=A, z=A, act=2, N=100, d_in=64, d_out=48, dx=B, dW=B, db=B, ws=A, n=need):
        return L.moe_linear_backward(dy, x, dt, W, z, act, N, d_in, d_out, dx, dW, db, ws, n, None)

    for bad in (dict(dt=3), dict(N=-1), dict(d_in=0), dict(d_out=0), dict(act=3), dict(dy=None), dict(x=None),
                dict(W=None), dict(z=None), dict(z=ODD), dict(dx=ODD), dict(dW=ODD), dict(db=ODD), dict(x=ODD),
                dict(ws=ODD)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 3 and call(n=need - 1) == 3 and "workspace" in _err(L)
    assert L.moe_linear_backward_workspace_size(100, 64, 48, 9, 0) == 0


def test_linear_outputs_are_not_inputs(L):
    X, W, Z = 0x500000, 0x600000, 0x700000
    for y, z in ((X, None), (W, None), (B, X), (B, W), (B, Z)):
        assert L.moe_linear(X, 1, W, None, 0, Z, 4, 64, 64, y, z, None, 0, None) == 1 and "input" in _err(L)
    for out in (A, X, W, Z):
        for dx, dW in ((out, None), (None, out)):
            assert L.moe_linear_backward(A, X, 1, W, Z, 2, 4, 64, 64, dx, dW, None, A, BIG, None) == 1
            assert "must not be an input" in _err(L)


def test_binding_refuses_what_it_cannot_pass(L):
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    for f in (lambda: moe.moe_layer_norm(x), lambda: moe.moe_linear(x, W),
              lambda: moe.moe_layer_norm_backward(x, x, x[:, 0], x[:, 0]),
              lambda: moe.moe_linear_backward(torch.zeros(4, 6), x, W)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    with pytest.raises(ValueError, match="2-D"):
        moe.moe_layer_norm(torch.zeros(8))

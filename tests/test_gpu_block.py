"""MoEBlock (layer norm, shared expert, the layer, their backward passes run
together) against 64-bit autograd with the kernels' routing (needs a B200).

Tolerances in the 2-norm, relative.  bf16: a value passes through at most ten
roundings of half a step (2^-8 each at most, h, n, H, the experts' output, y, z,
u, s and their gradients), and the maps between them keep relative errors within
a factor of two: 10 * 2 * 2^-8 = 0.08.  fp32: the products' bound of 1e-5 (see
test_gpu_linear) over two products in a row: 2e-5."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

EPS = 1e-5
TOL = {torch.bfloat16: 0.08, torch.float32: 2e-5}


def make(N, d, E, d_ff, k, cf, d_s, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    layer = moe.MoELayer(r(E, d) / d ** 0.5, (r(E, d_ff, d) / d ** 0.5).to(dtype), (r(E, d, d_ff) / d_ff ** 0.5).to(dtype),
                         k, cf, b_g=0.1 * r(E))
    shared = ((r(d_s, d) / d ** 0.5).to(dtype), 0.1 * r(d_s), (r(d, d_s) / d_s ** 0.5).to(dtype), 0.1 * r(d)) if d_s else None
    block = moe.MoEBlock(layer, 1 + 0.2 * r(d), 0.1 * r(d), EPS, shared=shared, shared_act=moe.ACT_GELU)
    return block, r(N, d).to(dtype), r(N, d).to(dtype), r(N, d).to(dtype), r(N, d).to(dtype)


def rel(got, want):
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-30))


def reference(block, x, delta, saved, ds, dm):
    """The same block in 64 bits, the routing (indices and slots) as the kernels chose it."""
    L = block.layer
    leaf = {q: v.double().requires_grad_() for q, v in
            dict(x=x, delta=delta, gamma=block.gamma, beta=block.beta, W_g=L.W_g, b_g=L.b_g, W_up=L.W_up,
                 W_down=L.W_down).items()}
    h = leaf["x"] + leaf["delta"]
    n = torch.nn.functional.layer_norm(h, (x.shape[1],), leaf["gamma"], leaf["beta"], EPS)
    logits = n @ leaf["W_g"].t() + leaf["b_g"]
    idx = saved["topk"].long()
    gates = torch.softmax(logits.gather(1, idx), dim=1) * (saved["dispatch"]["slot"] >= 0)
    m = torch.zeros_like(n)
    for e in range(L.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        y = torch.relu(n[t] @ leaf["W_up"][e].t()) @ leaf["W_down"][e].t()
        m = m.index_add(0, t, gates[t, j][:, None] * y)
    s = h
    if block.shared is not None:
        for q, v in zip(("W1", "b1", "W2", "b2"), block.shared):
            leaf[q] = v.double().requires_grad_()
        s = h + torch.nn.functional.gelu(n @ leaf["W1"].t() + leaf["b1"]) @ leaf["W2"].t() + leaf["b2"]
    grads = torch.autograd.grad((s * ds.double()).sum() + (m * dm.double()).sum(), list(leaf.values()))
    return s.detach(), m.detach(), dict(zip(leaf, grads))


NAMES = dict(dx="x", dgamma="gamma", dbeta="beta", dW_g="W_g", db_g="b_g", dW_up="W_up", dW_down="W_down", dW1="W1",
             db1="b1", dW2="W2", db2="b2")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,d,E,d_ff,k,cf,d_s", [(200, 256, 4, 320, 2, None, 384), (1, 128, 4, 64, 2, None, 72),
                                                 (333, 136, 8, 96, 2, 1.0, 0), (700, 96, 3, 200, 1, 1.25, 264)])
def test_block_and_gradients(N, d, E, d_ff, k, cf, d_s, dtype):
    require_gpu()
    block, x, delta, ds, dm = make(N, d, E, d_ff, k, cf, d_s, dtype, seed=N)
    s, m, saved = block.train(x, delta)
    g = block.backward(ds.clone(), dm, saved)
    want_s, want_m, want = reference(block, x, delta, saved, ds, dm)
    tol = TOL[dtype]
    assert rel(s, want_s) <= tol and rel(m, want_m) <= tol
    assert set(g) == set(NAMES) - (set() if d_s else {"dW1", "db1", "dW2", "db2"})
    for q, v in g.items():
        if k == 1 and NAMES[q] in ("W_g", "b_g"):   # one choice: its gate is 1, the router has no gradient
            assert float(v.abs().max()) <= tol
        else:
            assert rel(v, want[NAMES[q]]) <= tol, q
    assert rel(g["dx"], want["delta"]) <= tol
    assert moe.check_linear_status() == (0, 0)


@pytest.mark.parametrize("N", [1, 64, 500])
def test_blocks_chain_and_replay(N):
    """Two blocks and the last norm, eager and as one captured graph replayed with
    new inputs, give the same bits; the forward agrees with train()'s."""
    require_gpu()
    b1, x, delta, x2, _ = make(N, 256, 4, 320, 2, None, 384, torch.bfloat16, seed=1)
    b2 = make(N, 256, 4, 192, 2, 1.25, 0, torch.bfloat16, seed=2)[0]

    def run(x):
        s, m = b2(*b1(x))
        return moe.moe_layer_norm(s, b2.gamma, b2.beta, EPS, residual=m)[:2]

    want = [run(x), run(x2)]
    s, m, _ = b1.train(x)
    s0, m0 = b1(x)
    assert torch.equal(s, s0) and rel(m, m0.double()) <= TOL[torch.bfloat16]   # the decode plan sums K in other parts
    torch.cuda.synchronize()
    buf = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(buf)
    for v, w in ((x2, want[1]), (x, want[0])):
        buf.copy_(v)
        graph.replay()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])


def test_train_refuses_what_the_layer_cannot_train():
    require_gpu()
    block, x, _, _, _ = make(8, 64, 2, 64, 1, None, 0, torch.bfloat16, seed=0)
    block.layer.act = moe.ACT_GELU
    with pytest.raises(ValueError, match="ReLU"):
        block.train(x)

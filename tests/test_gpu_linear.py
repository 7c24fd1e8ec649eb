"""moe_linear and moe_linear_backward on the GPU against the formulas in 64
bits (needs a B200).

Tolerances, with u = 2^-24: a product sum of K terms in fp32, in any order and
with each addition off by at most 2 u (an accumulator that truncates), is off by
at most (K + 4) 2 u sum|a||b|; the fp32 products of fp32 storage may themselves
be off by 4 u relative, which the 4 covers.  GELU and its derivative have slopes
up to 1.13 and 0.8 and add at most 8 u (|z| + 1).  Then half a step of the
storage type, finfo.eps / 2, for each rounding: one for y and z, two (dZ, then
the output) for dx and dW.  db sums the unrounded dZ: N additions at most."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu
from tests.test_gpu_norm import close

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "gelu": moe.ACT_GELU}


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    return z * 0.5 * torch.erfc(-z * 0.5 ** 0.5) if act == "gelu" else z


def grad64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z * torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5
    return torch.ones_like(z)


def make(n, d_in, d_out, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=r(n, d_in).to(dtype), W=(r(d_out, d_in) / d_in ** 0.5).to(dtype), b=0.3 * r(d_out),
                res=r(n, d_out).to(dtype), dy=r(n, d_out).to(dtype))


def check_forward(t, act, bias=True, residual=True, **kw):
    dtype = t["x"].dtype
    half = torch.finfo(dtype).eps / 2
    x, W = t["x"].double(), t["W"].double()
    y, z = moe.moe_linear(t["x"], t["W"], b=t["b"] if bias else None, act=ACTS[act],
                          residual=t["res"] if residual else None, keep_z=True, **kw)
    want_z = x @ W.t()
    zt = (x.shape[1] + 4) * 2 * U * (x.abs() @ W.abs().t())
    if bias:
        want_z += t["b"].double()
        zt += U * want_z.abs()
    close(z, want_z, zt + half * (want_z.abs() + zt), "z")
    want = act64(want_z, act)
    yt = 1.13 * zt + (8 * U * (want_z.abs() + 1) if act == "gelu" else 0.0)
    if residual:
        want = want + t["res"].double()
        yt = yt + U * want.abs()
    close(y, want, yt + half * (want.abs() + yt), "y")
    return y, z


def check_backward(t, z, act, **kw):
    dtype = t["x"].dtype
    half = torch.finfo(dtype).eps / 2
    x, W, dy = t["x"].double(), t["W"].double(), t["dy"].double()
    n, d_out = dy.shape
    got = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=ACTS[act], z=None if act == "none" else z, **kw)
    dz = dy if act == "none" else dy * grad64(z.double(), act)
    dzt = torch.zeros_like(dy) if act != "gelu" else 8 * U * (z.double().abs() + 1) * dy.abs()
    close(got["db"], dz.sum(0), dzt.sum(0) + (n + 4) * U * (dz.abs() + dzt).sum(0), "db")
    if act != "none":
        dzt = dzt + half * (dz.abs() + dzt)   # the rounding of dZ
    m = dz.abs() + dzt
    for name, want, tol in (("dx", dz @ W, dzt @ W.abs() + (d_out + 4) * 2 * U * (m @ W.abs())),
                            ("dW", dz.t() @ x, dzt.t() @ x.abs() + (n + 4) * 2 * U * (m.t() @ x.abs()))):
        close(got[name], want, tol + half * (want.abs() + tol), name)
    return got


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 3, 5), (3, 17, 33), (7, 64, 64), (1, 2048, 1408), (1, 1001, 1337), (5, 256, 130),
          (8, 4096, 512), (13, 200, 4096), (16, 768, 768), (17, 8, 1000), (31, 1000, 8), (33, 72, 264), (63, 520, 2056),
          (64, 4096, 1024), (65, 136, 128), (100, 100, 100), (127, 128, 129), (128, 128, 128), (129, 64, 257),
          (130, 1408, 2048), (200, 4104, 24), (255, 512, 256), (256, 256, 256), (257, 264, 520), (300, 63, 65),
          (511, 768, 2048), (600, 1001, 77), (1000, 40, 72), (1025, 2048, 1408), (2047, 1001, 1337), (4097, 768, 130),
          (5000, 16, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    require_gpu()
    t = make(*shape, dtype, seed=sum(shape))
    for act in ("gelu", "none"):
        _, z = check_forward(t, act)
        check_backward(t, z, act)
    assert moe.check_linear_status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 24, 40), (64, 512, 384), (70, 77, 91), (600, 512, 1408), (2100, 768, 1024)],
                         ids=lambda s: "x".join(map(str, s)))
def test_epilogues(shape, dtype):
    """Every activation with and without bias and residual; repeated calls give the same bits."""
    require_gpu()
    t = make(*shape, dtype, seed=3)
    for act in ACTS:
        for bias in (False, True):
            for residual in (False, True):
                y, z = check_forward(t, act, bias, residual)
                kw = dict(b=t["b"] if bias else None, act=ACTS[act], residual=t["res"] if residual else None)
                assert torch.equal(moe.moe_linear(t["x"], t["W"], **kw), y)   # without z
                over = t["res"].clone()
                if residual:   # in place over the residual
                    kw["residual"] = over
                assert torch.equal(moe.moe_linear(t["x"], t["W"], **kw, y=over), y)
        a, b = check_backward(t, z, act), check_backward(t, z, act)
        assert all(torch.equal(a[q], b[q]) for q in a)
        for one in ("dx", "dW", "db"):
            c = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=ACTS[act], z=z, want_dx=one == "dx",
                                        want_dW=one == "dW", want_db=one == "db")
            assert torch.equal(c[one], a[one]) and sum(v is not None for v in c.values()) == 1


@pytest.mark.parametrize("shape", [(1500, 4096, 1408), (3000, 2048, 2048), (64, 14336, 1024)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fp32_is_fp32(shape):
    """fp32 storage keeps fp32's precision: the 2-norm of the error is at most
    1e-5 of the result's, 170 u, although a single product of bf16 parts is exact
    to 2^-8 only."""
    require_gpu()
    t = make(*shape, torch.float32, seed=4)
    x, W, dy = t["x"].double(), t["W"].double(), t["dy"].double()
    y = moe.moe_linear(t["x"], t["W"])
    g = moe.moe_linear_backward(t["dy"], t["x"], t["W"])
    for got, want in ((y, x @ W.t()), (g["dx"], dy @ W), (g["dW"], dy.t() @ x)):
        assert float((got.double() - want).norm() / want.norm()) <= 1e-5


def test_fp32_scales():
    """Rows and columns of very different magnitude keep their own relative precision."""
    require_gpu()
    for n, d_in, d_out in ((40, 96, 72), (700, 512, 384)):
        t = make(n, d_in, d_out, torch.float32, seed=6)
        t["x"] *= torch.logspace(-12, 12, n, device="cuda")[:, None]
        t["W"] *= torch.logspace(-9, 9, d_out, device="cuda")[:, None]
        check_forward(t, "none", bias=False, residual=False)


def test_gradients_against_differences():
    """Central differences of the fp32 forward: rounding over the step, and the
    cubic term (GELU's third derivative is below 2)."""
    require_gpu()
    n, d_in, d_out, step = 4, 10, 12, 1e-2
    t = make(n, d_in, d_out, torch.float32, seed=8)
    _, z = moe.moe_linear(t["x"], t["W"], b=t["b"], act=moe.ACT_GELU, keep_z=True)
    got = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=moe.ACT_GELU, z=z)

    def loss(x, W, b):
        y = moe.moe_linear(x, W, b=b, act=moe.ACT_GELU, residual=t["res"])
        return float((y.double() * t["dy"].double()).sum())

    def diff(name, i):
        v = {q: t[q].clone() for q in ("x", "W", "b")}
        flat = v[name].view(-1)
        at = float(flat[i])
        flat[i] = at + step
        up, hi = float(flat[i]), loss(**v)
        flat[i] = at - step
        lo = float(flat[i])
        return (hi - loss(**v)) / (up - lo)

    tol = n * d_out * 3 * 3 * 30 * U / (2 * step) + 1e-4 * 2 * 10
    for name, g in (("x", got["dx"]), ("W", got["dW"]), ("b", got["db"])):
        for i in range(t[name].numel()):
            assert abs(diff(name, i) - float(g.view(-1)[i])) <= tol, (name, i)


def test_no_rows():
    require_gpu()
    for dtype in (torch.bfloat16, torch.float32):
        t = make(0, 64, 48, dtype, seed=0)
        y, z = moe.moe_linear(t["x"], t["W"], b=t["b"], act=moe.ACT_GELU, residual=t["res"], keep_z=True)
        assert y.shape == z.shape == (0, 48)
        g = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=moe.ACT_GELU, z=z)
        assert g["dx"].shape == (0, 64) and not g["dW"].any() and not g["db"].any()


def test_relu_masks_even_infinite_gradients():
    require_gpu()
    t = make(70, 64, 128, torch.bfloat16, seed=2)
    _, z = moe.moe_linear(t["x"], t["W"], act=moe.ACT_RELU, keep_z=True)
    t["dy"][(z <= 0) & (torch.arange(128, device="cuda") % 5 == 0)] = float("inf")
    check = dict(t, dy=torch.where(z > 0, t["dy"], torch.zeros_like(t["dy"])))
    a = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=moe.ACT_RELU, z=z)
    b = moe.moe_linear_backward(check["dy"], t["x"], t["W"], act=moe.ACT_RELU, z=z)
    assert all(torch.equal(a[q], b[q]) and bool(a[q].isfinite().all()) for q in a)


@pytest.mark.parametrize("shape", [(5, 64, 136), (64, 512, 136), (300, 256, 264), (70, 30, 50)],
                         ids=lambda s: "x".join(map(str, s)))
def test_rows_beside_the_batch_stay(shape):
    """Outputs inside larger arrays; NaN rows around the inputs are not read into the result."""
    require_gpu()
    n, d_in, d_out = shape
    for dtype in (torch.bfloat16, torch.float32):
        t = make(n, d_in, d_out, dtype, seed=12)
        want, z = moe.moe_linear(t["x"], t["W"], b=t["b"], act=moe.ACT_GELU, residual=t["res"], keep_z=True)
        ref = moe.moe_linear_backward(t["dy"], t["x"], t["W"], act=moe.ACT_GELU, z=z)
        pad = lambda a: torch.cat([torch.full_like(a[:1].expand(8, -1), float("nan")), a,  # noqa: E731
                                   torch.full_like(a[:1].expand(130, -1), float("nan"))])[8:8 + a.shape[0]]
        p = {q: pad(t[q]) for q in ("x", "W", "res", "dy")}
        zp = pad(z)
        big = torch.full((n + 16, d_out), 7.0, dtype=dtype, device="cuda")
        moe.moe_linear(p["x"], p["W"], b=t["b"], act=moe.ACT_GELU, residual=p["res"], y=big[8:8 + n])
        assert torch.equal(big[8:8 + n], want)
        assert bool((big[:8] == 7).all()) and bool((big[8 + n:] == 7).all())
        got = moe.moe_linear_backward(p["dy"], p["x"], p["W"], act=moe.ACT_GELU, z=zp)
        assert all(torch.equal(got[q], ref[q]) for q in ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_streams_and_graphs(dtype):
    """Two streams at once, and two captured graphs sharing one workspace and
    replayed in turn with new inputs, give the eager bits."""
    require_gpu()
    n, d_in, d_out = 333, 260, 520
    ins = [make(n, d_in, d_out, dtype, seed=s) for s in (1, 2)]
    W, b = ins[0]["W"], ins[0]["b"]

    def step(t, ws=None, wsb=None, stream=None):
        y, z = moe.moe_linear(t["x"], W, b=b, act=moe.ACT_GELU, residual=t["res"], keep_z=True, ws=ws, stream=stream)
        return y, z, moe.moe_linear_backward(t["dy"], t["x"], W, act=moe.ACT_GELU, z=z, ws=wsb, stream=stream)

    def same(p, q):
        return torch.equal(p[0], q[0]) and torch.equal(p[1], q[1]) and all(torch.equal(p[2][k], q[2][k]) for k in q[2])

    ref = [step(t) for t in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[step(t, stream=s) for t, s in zip(ins, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(same(g, r) for turn in got for g, r in zip(turn, ref))
    L = moe.load_library()
    dt = moe._dt(W)
    ws = torch.empty(max(256, L.moe_linear_workspace_size(n, d_in, d_out, dt)), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(max(256, L.moe_linear_backward_workspace_size(n, d_in, d_out, moe.ACT_GELU, dt)),
                      dtype=torch.uint8, device="cuda")
    buf = {q: v.clone() for q, v in ins[0].items()}
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(buf, ws, wsb))
        graphs.append(g)
    for i in (1, 0, 1):
        for q in ("x", "res", "dy"):
            buf[q].copy_(ins[i][q])
        for g, o in zip(graphs, outs):
            g.replay()
            assert same(o, ref[i])
    assert moe.check_linear_status() == (0, 0)


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements: its last rows equal the same rows alone."""
    require_gpu()
    n, d_in, d_out = 150100, 64, 14336
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(n, d_in, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(d_out, d_in, generator=g, device="cuda").to(torch.bfloat16)
    y = moe.moe_linear(x, W, act=moe.ACT_RELU)
    want = (x[-200:].double() @ W.double().t()).clamp(min=0)
    close(y[-200:], want, 2 ** -8 * want.abs() + 68 * 2 * U * (x[-200:].double().abs() @ W.double().abs().t()), "y")


def test_few_tokens_of_wide_rows():
    """Around the token counts and weight sizes where another kernel takes over."""
    require_gpu()
    for n in (1, 4, 5, 8, 9, 16, 17, 33, 64, 65):
        for d_in, d_out in ((1001, 1337), (1031, 1033), (2048, 1029), (1027, 1032), (300, 700), (140, 2000),
                            (192, 4432)):
            for dtype in (torch.bfloat16, torch.float32):
                t = make(n, d_in, d_out, dtype, seed=n)
                _, z = check_forward(t, "gelu")
                check_backward(t, z, "gelu")

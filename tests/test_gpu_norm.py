"""moe_layer_norm and moe_layer_norm_backward on the GPU against the formulas
in 64 bits (needs a B200).

Tolerances, with u = 2^-24 (half a step of fp32) and k = d / 32 + 16, an upper
bound on the additions any one value passes through in a row sum (a lane sums
at most every 32nd element, then a tree):
  mean: k u mean|h|;  rstd: (k / 2 + 4) u relative (plus the mean's error, which
  enters the variance squared);
  xh: X (k + 8) u with X = |xh| + rstd (|h| + |mu| + mean|h|);
  y: |gamma| times that plus 2 u (|y| + |beta|), and half a step of the storage
  type, finfo.eps / 2 * |y|.
Backward, given mean and rstd: (k + 10) u rstd (|g| + mean|g| + X mean(|g| X)),
then the dres add (u of the sum) and half a step.  A column sum over N rows
passes through at most N / 32 + 64 additions: (N / 32 + 64 + 4) u sum|dy| X.
A bf16 output below the normal range would be off by an absolute half step of
2^-134; no test has values near it."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def make(n, d, dtype, seed, offset=0.25, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=(r(n, d) * std + offset).to(dtype), res=r(n, d).to(dtype), dy=r(n, d).to(dtype),
                dres=r(n, d).to(dtype), gamma=1 + 0.3 * r(d), beta=0.2 * r(d))


def close(got, want, tol, what):
    assert got.shape == want.shape, what
    bad = ~((got.double() - want).abs() <= tol)   # a NaN is bad
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(got.double()[bad][0]), float(want[bad][0]))


def stats(h):
    hd = h.double()
    mu = hd.mean(1)
    var = ((hd - mu[:, None]) ** 2).mean(1)
    return hd, mu, 1 / torch.sqrt(var + EPS)


def check_forward(t, n, d, dtype, gamma, beta, residual, **kw):
    y, h, mean, rstd = moe.moe_layer_norm(t["x"], gamma, beta, EPS, residual=t["res"] if residual else None,
                                          want_stats=True, **kw)
    want_h = (t["x"].float() + t["res"].float()).to(dtype) if residual else t["x"]
    assert torch.equal(h, want_h)
    hd, mu, rs = stats(want_h)
    k = d / 32 + 16
    a = hd.abs().mean(1)
    close(mean, mu, k * U * a + U * mu.abs(), "mean")
    close(rstd, rs, ((k / 2 + 4) * U + (k * U * a * rs) ** 2) * rs, "rstd")
    xh = (hd - mu[:, None]) * rs[:, None]
    X = xh.abs() + rs[:, None] * (hd.abs() + (mu.abs() + a)[:, None])
    ga = 1.0 if gamma is None else gamma.double()
    be = torch.zeros(d, device="cuda").double() if beta is None else beta.double()
    want = xh * ga + be
    tol = (X * ga if gamma is None else X * ga.abs()) * (k + 8) * U + 2 * U * (want.abs() + be.abs())
    close(y, want, tol * (1 + 2 ** -7) + torch.finfo(dtype).eps / 2 * want.abs(), "y")
    return y, h, mean, rstd


def check_backward(t, h, mean, rstd, n, d, dtype, gamma, dres, **kw):
    hd, mu, rs = h.double(), mean.double()[:, None], rstd.double()[:, None]
    dy = t["dy"].double()
    want_dres = t["dres"].double() if dres else 0.0
    out = moe.moe_layer_norm_backward(t["dy"], h, mean, rstd, gamma=gamma, dres=t["dres"] if dres else None, **kw)
    k = d / 32 + 16
    xh = (hd - mu) * rs
    X = xh.abs() + rs * (hd.abs() + mu.abs())
    g = dy if gamma is None else dy * gamma.double()
    core = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    want = core + want_dres
    tol = (k + 10) * U * rs * (g.abs() + g.abs().mean(1, keepdim=True) + X * (g.abs() * X).mean(1, keepdim=True))
    close(out["dx"], want, (tol + U * want.abs()) * (1 + 2 ** -7) + torch.finfo(dtype).eps / 2 * want.abs(), "dx")
    k2 = (n / 32 + 68) * U
    close(out["dgamma"], (dy * xh).sum(0), k2 * (dy.abs() * X).sum(0), "dgamma")
    close(out["dbeta"], dy.sum(0), k2 * dy.abs().sum(0), "dbeta")
    return out


WIDTHS = [1, 2, 3, 7, 8, 9, 31, 33, 64, 100, 127, 256, 511, 513, 768, 1001, 1024, 1337, 2040, 2048, 2050, 3000, 4090,
          4096, 4100, 8185, 8192, 8200, 16377, 16384, 16390, 20000, 33000]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dtype):
    require_gpu()
    for n in (1, 9, 130):
        t = make(n, d, dtype, seed=d * 3 + n)
        for residual in (False, True):
            y, h, mean, rstd = check_forward(t, n, d, dtype, t["gamma"], t["beta"], residual)
            check_backward(t, h, mean, rstd, n, d, dtype, t["gamma"], residual)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(2, 768), (3, 1001), (7, 4096), (8, 4099), (64, 4096), (1000, 1337), (4099, 768),
                                 (2500, 2048), (1300, 4096), (700, 8191), (20000, 64), (9001, 33), (3001, 520)])
def test_batches(n, d, dtype):
    require_gpu()
    t = make(n, d, dtype, seed=n + d)
    y, h, mean, rstd = check_forward(t, n, d, dtype, t["gamma"], t["beta"], True)
    check_backward(t, h, mean, rstd, n, d, dtype, t["gamma"], True)
    # no gamma, no beta, no residual; the same bits on a second call
    y, h, mean, rstd = check_forward(t, n, d, dtype, None, None, False)
    a = check_backward(t, h, mean, rstd, n, d, dtype, None, False)
    b = check_backward(t, h, mean, rstd, n, d, dtype, None, False)
    assert all(torch.equal(a[q], b[q]) for q in a)
    assert torch.equal(y, moe.moe_layer_norm(t["x"], eps=EPS)[0])


def test_large_offset_keeps_the_variance():
    """A common offset of 1000 spreads: the variance is taken from centred values."""
    require_gpu()
    t = make(64, 4096, torch.float32, seed=5, offset=1000.0)
    y, h, mean, rstd = check_forward(t, 64, 4096, torch.float32, t["gamma"], t["beta"], False)
    check_backward(t, h, mean, rstd, 64, 4096, torch.float32, t["gamma"], True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_constant_rows_and_rows_apart(dtype):
    """A constant row normalises to beta; a NaN or infinite row stays in its row
    of y and dx (it does reach the column sums)."""
    require_gpu()
    for d in (40, 1001, 4096, 9000, 40000):
        t = make(6, d, dtype, seed=d)
        t["x"][1] = 3.0
        y, _, mean, rstd = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS, want_stats=True)
        assert torch.equal(y[1], t["beta"].to(dtype)) and float(mean[1]) == 3.0
        x = t["x"].clone()
        x[2, d // 2] = float("nan")
        x[4, 0] = float("inf")
        y2, _, m2, r2 = moe.moe_layer_norm(x, t["gamma"], t["beta"], EPS, want_stats=True)
        keep = [0, 1, 3, 5]
        assert torch.equal(y2[keep], y[keep]) and bool(y2[2].isnan().all()) and bool(y2[4].isnan().all())
        a = moe.moe_layer_norm_backward(t["dy"], t["x"], mean, rstd, gamma=t["gamma"])
        b = moe.moe_layer_norm_backward(t["dy"], x, m2, r2, gamma=t["gamma"])
        assert torch.equal(a["dx"][keep], b["dx"][keep]) and bool(b["dx"][2].isnan().all())


@pytest.mark.parametrize("d", [768, 1001, 4096, 9000, 40000])
def test_in_place(d):
    """y over x; the sum over x or the residual; dx over dy, h or dres."""
    require_gpu()
    for dtype in (torch.bfloat16, torch.float32):
        t = make(300, d, dtype, seed=d + 1)
        y, h, mean, rstd = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS, residual=t["res"], want_stats=True)
        want = moe.moe_layer_norm_backward(t["dy"], h, mean, rstd, gamma=t["gamma"], dres=t["dres"])
        for over in ("x", "res"):
            c = {q: v.clone() for q, v in t.items()}
            y2, h2, _, _ = moe.moe_layer_norm(c["x"], t["gamma"], t["beta"], EPS, residual=c["res"], sum_out=c[over])
            assert h2 is c[over] and torch.equal(h2, h) and torch.equal(y2, y)
            c = {q: v.clone() for q, v in t.items()}
            y2, h2, _, _ = moe.moe_layer_norm(c["x"], t["gamma"], t["beta"], EPS, residual=c["res"], y=c[over])
            assert y2 is c[over] and torch.equal(h2, h) and torch.equal(y2, y)
        x = t["x"].clone()
        assert torch.equal(moe.moe_layer_norm(x, t["gamma"], t["beta"], EPS, y=x)[0],
                           moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS)[0])
        for over in ("dy", "h", "dres"):
            c = dict(dy=t["dy"].clone(), h=h.clone(), dres=t["dres"].clone())
            got = moe.moe_layer_norm_backward(c["dy"], c["h"], mean, rstd, gamma=t["gamma"], dres=c["dres"],
                                              dx=c[over])
            assert all(torch.equal(got[q], want[q]) for q in want), over


def test_gradients_against_differences():
    """Central differences of the forward in fp32 storage: the error of a
    difference is the cubic term, step^2 times third derivatives of order 1,
    and the forward's rounding over the step."""
    require_gpu()
    n, d, step = 5, 24, 1e-2
    t = make(n, d, torch.float32, seed=9)
    _, h, mean, rstd = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS, residual=t["res"], want_stats=True)
    got = moe.moe_layer_norm_backward(t["dy"], h, mean, rstd, gamma=t["gamma"])

    def loss(x, gamma, beta):
        return float((moe.moe_layer_norm(x, gamma, beta, EPS, residual=t["res"])[0].double() * t["dy"].double()).sum())

    def diff(name, i):
        v = {q: t[q].clone() for q in ("x", "gamma", "beta")}
        flat = v[name].view(-1)
        at = float(flat[i])
        flat[i] = at + step
        up, hi = float(flat[i]), loss(**v)
        flat[i] = at - step
        lo = float(flat[i])
        return (hi - loss(**v)) / (up - lo)

    # rounding: d values of about 3 with 40 u each, over 2 steps; cubic: 1e-4 * 10
    tol = d * 3 * 3 * 40 * U / (2 * step) + 1e-3
    for i in range(0, n * d, 7):
        assert abs(diff("x", i) - float(got["dx"].view(-1)[i])) <= tol
    for i in range(d):
        assert abs(diff("gamma", i) - float(got["dgamma"][i])) <= tol
        assert abs(diff("beta", i) - float(got["dbeta"][i])) <= tol


def test_no_rows():
    require_gpu()
    x = torch.empty((0, 768), dtype=torch.bfloat16, device="cuda")
    y, h, mean, rstd = moe.moe_layer_norm(x, residual=x, want_stats=True)
    assert y.shape == h.shape == (0, 768) and mean.shape == (0,)
    out = moe.moe_layer_norm_backward(x, x, mean, rstd)
    assert not out["dgamma"].any() and not out["dbeta"].any() and out["dx"].shape == (0, 768)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows equal the same rows alone."""
    require_gpu()
    n, d = 65600, 32768
    x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    last = torch.randn(70, d, device="cuda").to(torch.bfloat16)
    x[-70:] = last
    gamma = torch.rand(d, device="cuda")
    y, _, mean, rstd = moe.moe_layer_norm(x, gamma, None, EPS, want_stats=True)
    y1, _, m1, r1 = moe.moe_layer_norm(last, gamma, None, EPS, want_stats=True)
    assert torch.equal(y[-70:], y1) and torch.equal(mean[-70:], m1) and torch.equal(rstd[-70:], r1)
    out = moe.moe_layer_norm_backward(y, x, mean, rstd, gamma=gamma, want_params=False)
    one = moe.moe_layer_norm_backward(y1, last, m1, r1, gamma=gamma, want_params=False)
    assert out["dgamma"] is None and torch.equal(out["dx"][-70:], one["dx"])
    assert not out["dx"][:100].any()


def test_rows_beside_the_batch_stay():
    """Outputs inside larger arrays: nothing before or behind them is written."""
    require_gpu()
    for n, d in [(5, 1001), (64, 768), (3, 16391)]:
        t = make(n, d, torch.bfloat16, seed=n)
        step = 8 // __import__("math").gcd(d, 8)   # rows whose start is 16-byte aligned
        big = [torch.full((n + 2 * step, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        y, s, dx = (b[step:step + n] for b in big)
        _, h, mean, rstd = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS, residual=t["res"], want_stats=True,
                                              y=y, sum_out=s)
        moe.moe_layer_norm_backward(t["dy"], h, mean, rstd, gamma=t["gamma"], dx=dx)
        torch.cuda.synchronize()
        for b in big:
            assert bool((b[:step] == 7).all()) and bool((b[step + n:] == 7).all())


def test_streams_and_graphs():
    """A side stream, and two captured graphs that share a workspace, replayed in
    turn with new inputs, give the eager bits."""
    require_gpu()
    n, d = 777, 1001
    t = make(n, d, torch.bfloat16, seed=1)
    u = make(n, d, torch.bfloat16, seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, mean, rstd = moe.moe_layer_norm(t["x"], t["gamma"], t["beta"], EPS, residual=t["res"], want_stats=True,
                                          stream=side)
    out = moe.moe_layer_norm_backward(t["dy"], h, mean, rstd, gamma=t["gamma"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref = {}
    for q, v in (("t", t), ("u", u)):
        y0, h0, m0, r0 = moe.moe_layer_norm(v["x"], t["gamma"], t["beta"], EPS, residual=v["res"], want_stats=True)
        ref[q] = (y0, moe.moe_layer_norm_backward(v["dy"], h0, m0, r0, gamma=t["gamma"]))
    assert torch.equal(y, ref["t"][0]) and all(torch.equal(out[q], ref["t"][1][q]) for q in out)
    buf = {q: v.clone() for q, v in t.items()}
    ws = torch.empty(moe.load_library().moe_layer_norm_backward_workspace_size(n, d, moe.MOE_BF16),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y1, h1, m1, r1 = moe.moe_layer_norm(buf["x"], t["gamma"], t["beta"], EPS, residual=buf["res"],
                                                want_stats=True)
            o1 = moe.moe_layer_norm_backward(buf["dy"], h1, m1, r1, gamma=t["gamma"], ws=ws)
        graphs.append(g)
        got.append((y1, o1))
    for v, q in ((u, "u"), (t, "t"), (u, "u")):
        for name in ("x", "res", "dy"):
            buf[name].copy_(v[name])
        for g, (y1, o1) in zip(graphs, got):
            g.replay()
            assert torch.equal(y1, ref[q][0]) and all(torch.equal(o1[p], ref[q][1][p]) for p in o1)

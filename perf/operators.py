"""The operators around the expert layer, as cases: layer norm with the residual
add (forward, backward) and the dense layer with bias, activation and residual
(forward, backward).

`run` computes a case in elementary torch operations, or, where `own` is true,
through the framework's entry points.  `exact` gives the same outputs in 64
bits.  Shapes: x [n, d_in] row-major in bf16 or fp32, W [d_out, d_in] of the
same type; gamma, beta, the bias and their gradients are fp32.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = {"none": 0, "relu": 1, "gelu": 2}
# work of the largest listed case, which a drawn one never exceeds
MOST_NORM = 16384 * 4096
MOST_LINEAR = 16384 * 4096 * 14336


def _norm(name, n, d, dtype, residual):
    return {"name": name, "op": "norm", "n": n, "d": d, "dtype": dtype, "residual": residual}


def _norm_bwd(name, n, d, dtype, residual):
    return {"name": name, "op": "norm_bwd", "n": n, "d": d, "dtype": dtype, "residual": residual}


def _linear(name, n, d_in, d_out, dtype, act, residual):
    return {"name": name, "op": "linear", "n": n, "d_in": d_in, "d_out": d_out, "dtype": dtype, "act": act,
            "residual": residual}


def _linear_bwd(name, n, d_in, d_out, dtype, act):
    return {"name": name, "op": "linear_bwd", "n": n, "d_in": d_in, "d_out": d_out, "dtype": dtype, "act": act}


def listed():
    return [
        # one decode step of a 64-sequence batch: the norm in front of the expert layer, launch-bound
        _norm("norm decode 64x4096", 64, 4096, "bf16", True),
        # a prefill or training batch of the fine-grained workload: bandwidth-bound
        _norm("norm fine 32768x2048", 32768, 2048, "bf16", True),
        # rows of an odd width, whose starts have no common alignment
        _norm("norm odd 8191x1001", 8191, 1001, "bf16", False),
        # training batch of the small GPT-sized workload, with the skip path's gradient
        _norm_bwd("norm bwd nano 8192x768", 8192, 768, "bf16", True),
        # training batch of the large workload
        _norm_bwd("norm bwd wide 16384x4096", 16384, 4096, "bf16", True),
        # an fp32 model of an odd width
        _norm_bwd("norm bwd odd 1000x1337", 1000, 1337, "f32", False),
        # a shared expert's up projection for one token: streams W once, latency counts
        _linear("linear token 1x2048x1408", 1, 2048, 1408, "bf16", "gelu", False),
        # a dense down projection in a 64-sequence decode step, the skip path added: bound by W's bytes
        _linear("linear decode 64x14336x4096", 64, 14336, 4096, "bf16", "none", True),
        # a dense up projection in prefill: bound by the tensor cores
        _linear("linear prefill 16384x4096x14336", 16384, 4096, 14336, "bf16", "gelu", False),
        # an fp32 model with odd widths
        _linear("linear odd 2047x1001x1337", 2047, 1001, 1337, "f32", "relu", True),
        # a shared expert's up projection in training
        _linear_bwd("linear bwd fine 32768x2048x1408", 32768, 2048, 1408, "bf16", "gelu"),
        # an fp32 projection in training, sizes off the tiles
        _linear_bwd("linear bwd f32 4097x768x2050", 4097, 768, 2050, "f32", "none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over the range: half of them multiples of 64, a quarter of 8, the others any."""
    v = _log(rng, lo, hi)
    to = rng.choice((64, 64, 8, 1))
    return min(hi, max(lo, (v + to - 1) // to * to))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if rng.random() < 0.5:
        op = rng.choice(("norm", "norm_bwd"))
        d = _width(rng, 16, 16384)
        n = _log(rng, 1, max(1, min(65536, MOST_NORM // (2 * d))))
        return {"op": op, "n": n, "d": d, "dtype": dtype, "residual": rng.random() < 0.6}
    op = rng.choice(("linear", "linear_bwd"))
    d_in, d_out = _width(rng, 8, 14336), _width(rng, 8, 14336)
    most = MOST_LINEAR // (2 if op == "linear_bwd" else 1) // (16 if dtype == "f32" else 1)
    n = _log(rng, 1, max(1, min(16384, most // (d_in * d_out))))
    case = {"op": op, "n": n, "d_in": d_in, "d_out": d_out, "dtype": dtype, "act": rng.choice(tuple(ACTS))}
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    n = case["n"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    s = {"case": case}
    if case["op"] in ("norm", "norm_bwd"):
        d = case["d"]
        # hidden states: a common offset and a spread that differs from row to row
        spread = torch.rand(n, 1, generator=g, device="cuda") * 2 + 0.5
        x = (torch.randn(n, d, generator=g, device="cuda") * spread + 0.25).to(dt)
        s["gamma"] = normal(d, std=0.2, mean=1.0, dtype=torch.float32)
        s["beta"] = normal(d, std=0.1, dtype=torch.float32)
        if case["op"] == "norm":
            s["x"] = x
            s["residual"] = normal(n, d, std=0.5) if case["residual"] else None
            return s
        s["h"] = x
        s["mean"] = x.float().mean(1)
        s["rstd"] = (x.float().var(1, unbiased=False) + EPS).rsqrt()
        s["dy"] = normal(n, d)
        s["dres"] = normal(n, d) if case["residual"] else None
        return s
    d_in, d_out = case["d_in"], case["d_out"]
    s["x"] = normal(n, d_in)
    s["W"] = normal(d_out, d_in, std=1.0 / math.sqrt(d_in))
    if case["op"] == "linear":
        s["b"] = normal(d_out, std=0.1, dtype=torch.float32)
        s["residual"] = normal(n, d_out) if case["residual"] else None
        return s
    s["dy"] = normal(n, d_out)
    # the forward's pre-activations, as it stored them
    s["z"] = torch.matmul(s["x"], s["W"].t()) if case["act"] != "none" else None
    return s


def _own(s):
    from sparse_mixture_experts_noisy_b200 import moe
    case = s["case"]
    if case["op"] == "norm":
        return moe.moe_layer_norm(s["x"], s["gamma"], s["beta"], EPS, residual=s["residual"], want_stats=True)
    if case["op"] == "norm_bwd":
        return moe.moe_layer_norm_backward(s["dy"], s["h"], s["mean"], s["rstd"], gamma=s["gamma"], dres=s["dres"])
    if case["op"] == "linear":
        return moe.moe_linear(s["x"], s["W"], b=s["b"], act=ACTS[case["act"]], residual=s["residual"])
    return moe.moe_linear_backward(s["dy"], s["x"], s["W"], act=ACTS[case["act"]], z=s["z"])


def _plain_norm(x, residual, gamma, beta):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hf = h.float()
    mean = hf.sum(1) / hf.shape[1]
    c = hf - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).sum(1) / hf.shape[1] + EPS)
    y = c * rstd[:, None] * gamma + beta
    return y.to(x.dtype), h, mean, rstd


def _plain_norm_bwd(dy, h, mean, rstd, gamma, dres):
    d = h.shape[1]
    dyf = dy.float()
    xh = (h.float() - mean[:, None]) * rstd[:, None]
    gdy = dyf * gamma
    dx = rstd[:, None] * (gdy - gdy.sum(1, keepdim=True) / d - xh * ((gdy * xh).sum(1, keepdim=True) / d))
    if dres is not None:
        dx = dx + dres.float()
    return {"dx": dx.to(dy.dtype), "dgamma": (dyf * xh).sum(0), "dbeta": dyf.sum(0)}


def _plain_linear(x, W, b, act, residual):
    z = x.float() @ W.float().t() + b
    if act == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif act == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if residual is not None:
        z = z + residual.float()
    return z.to(x.dtype)


def _plain_linear_bwd(dy, x, W, act, z):
    dz = dy.float()
    if act == "relu":
        dz = dz * (z > 0)
    elif act == "gelu":
        zf = z.float()
        cdf = 0.5 * (1 + torch.erf(zf * math.sqrt(0.5)))
        dz = dz * (cdf + zf * torch.exp(-0.5 * zf * zf) * (1 / math.sqrt(2 * math.pi)))
    return {"dx": (dz @ W.float()).to(x.dtype), "dW": (dz.t() @ x.float()).to(W.dtype), "db": dz.sum(0)}


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    if case["op"] == "norm":
        return _plain_norm(s["x"], s["residual"], s["gamma"], s["beta"])
    if case["op"] == "norm_bwd":
        return _plain_norm_bwd(s["dy"], s["h"], s["mean"], s["rstd"], s["gamma"], s["dres"])
    if case["op"] == "linear":
        return _plain_linear(s["x"], s["W"], s["b"], case["act"], s["residual"])
    return _plain_linear_bwd(s["dy"], s["x"], s["W"], case["act"], s["z"])


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "norm":
        d = case["d"]  # x and y, the residual and the sum; gamma, beta; the two statistics
        return {"bytes": n * d * es * (4 if case["residual"] else 2) + 8 * d + 8 * n, "flops": 8 * n * d}
    if case["op"] == "norm_bwd":
        d = case["d"]  # dy, h and dx, the skip path's gradient; gamma, dgamma, dbeta; the two statistics
        return {"bytes": n * d * es * (4 if case["residual"] else 3) + 12 * d + 8 * n, "flops": 14 * n * d}
    d_in, d_out = case["d_in"], case["d_out"]
    if case["op"] == "linear":
        return {"bytes": es * (n * d_in + d_in * d_out + n * d_out * (2 if case["residual"] else 1)) + 4 * d_out,
                "flops": 2 * n * d_in * d_out}
    rows = 1 if case["act"] == "none" else 2  # dy, and z
    return {"bytes": es * (n * d_out * rows + 2 * n * d_in + 2 * d_in * d_out) + 4 * d_out,
            "flops": 4 * n * d_in * d_out}


def exact(case, seed):
    s = prepare(case, seed)
    F = torch.nn.functional
    up = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "norm":
        # the operator normalises the sum as it is stored
        h = s["x"] if s["residual"] is None else torch.add(s["x"].float(), s["residual"].float()).to(s["x"].dtype)
        hd = h.double()
        var, mean = torch.var_mean(hd, dim=1, correction=0)
        y = F.layer_norm(hd, (case["d"],), s["gamma"].double(), s["beta"].double(), EPS)
        return y, hd, mean, (var + EPS).pow(-0.5)
    if case["op"] == "norm_bwd":
        h, ga = up(s["h"]).requires_grad_(), up(s["gamma"]).requires_grad_()
        be = torch.zeros_like(ga).requires_grad_()
        dx, dg, db = torch.autograd.grad(F.layer_norm(h, (case["d"],), ga, be, EPS), (h, ga, be), up(s["dy"]))
        return {"dx": dx if s["dres"] is None else dx + up(s["dres"]), "dgamma": dg, "dbeta": db}
    act = {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu}[case["act"]]
    if case["op"] == "linear":
        y = act(F.linear(up(s["x"]), up(s["W"]), up(s["b"])))
        return y if s["residual"] is None else y.add_(up(s["residual"]))
    dz = up(s["dy"])
    if s["z"] is not None:
        z = up(s["z"]).requires_grad_()
        dz, = torch.autograd.grad(act(z), z, dz)
    return {"dx": torch.einsum("no,oi->ni", dz, up(s["W"])), "dW": torch.einsum("no,ni->oi", dz, up(s["x"])),
            "db": torch.einsum("no->o", dz)}

"""fp32 storage of the dense layer over its range of values: what the three bf16
parts of a value keep, and where they stop (needs a B200).

A value v = p0 + p1 + p2 exactly from 2^-110 up to fp32's largest; below, the
parts end at bf16's smallest step 2^-133, so their sum is off by at most
2^-134."""
import pytest
import torch

from sparse_mixture_experts_noisy_b200 import moe
from tests.gpu_util import require_gpu
from tests.test_gpu_norm import close

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FEW, MANY = (8, 256, 128), (700, 512, 384)        # CUDA cores; CTA pairs and split K
SHAPES = [FEW, (100, 256, 128), MANY, (2500, 1024, 1024)]
ids = lambda s: "x".join(map(str, s))  # noqa: E731


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_all_24_bits_of_a_value_arrive(shape):
    """W has a single power of two in each row (and column), so every output is one
    value, scaled.  Its parts are added from the smallest up; each of three
    additions is off by 2 u at most.  Without the third part the error would be up
    to 2^-17, 128 u."""
    require_gpu()
    n, d_in, d_out = shape
    g = gen(n)
    x = torch.randn(n, d_in, generator=g, device="cuda") * torch.logspace(-25, 25, n, device="cuda")[:, None]
    dy = torch.randn(n, d_out, generator=g, device="cuda") * torch.logspace(-25, 25, n, device="cuda")[:, None]
    W = torch.zeros(d_out, d_in, device="cuda")
    cols = torch.randperm(d_in, generator=g, device="cuda")[:d_out] if d_out <= d_in else None
    assert cols is not None
    scale = 2.0 ** torch.randint(-9, 10, (d_out,), generator=g, device="cuda").float()
    W[torch.arange(d_out, device="cuda"), cols] = scale
    want = x.double()[:, cols] * scale.double()
    close(moe.moe_linear(x, W), want, 6 * U * want.abs(), "y")
    got = moe.moe_linear_backward(dy, x, W, want_dW=False, want_db=False)["dx"]
    want = torch.zeros(n, d_in, dtype=torch.float64, device="cuda")
    want[:, cols] = dy.double() * scale.double()
    close(got, want, 6 * U * want.abs(), "dx")


@pytest.mark.parametrize("rows", [200, 3000])
def test_all_24_bits_reach_dW(rows):
    """One row of dy is a power of two and the others zero: dW's row is that row of x, scaled."""
    require_gpu()
    g = gen(rows)
    x = torch.randn(rows, 512, generator=g, device="cuda")
    W = torch.randn(384, 512, generator=g, device="cuda")
    dy = torch.zeros(rows, 384, device="cuda")
    pick = torch.randint(0, rows, (384,), generator=g, device="cuda")
    dy[pick, torch.arange(384, device="cuda")] = 0.25
    got = moe.moe_linear_backward(dy, x, W, want_dx=False, want_db=False)["dW"]
    want = 0.25 * x.double()[pick]
    close(got, want, 6 * U * want.abs(), "dW")


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_small_values(shape):
    """Rows around 1e-36: normal numbers whose parts are cut off at 2^-134 on the
    tensor cores, each in a sum of K products with W."""
    require_gpu()
    n, d_in, d_out = shape
    g = gen(n + 1)
    x = torch.randn(n, d_in, generator=g, device="cuda") * 1e-36
    W = torch.randn(d_out, d_in, generator=g, device="cuda")
    want = x.double() @ W.double().t()
    tol = (d_in + 4) * 2 * U * (x.double().abs() @ W.double().abs().t()) + 2.0 ** -134 * W.double().abs().sum(1)
    close(moe.moe_linear(x, W), want, tol + U * want.abs() + 2.0 ** -149, "y")


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_largest_finite_values(shape):
    """Values up to fp32's largest, beyond bf16's, against small weights."""
    require_gpu()
    n, d_in, d_out = shape
    g = gen(n + 2)
    top = torch.finfo(torch.float32).max
    x = torch.randn(n, d_in, generator=g, device="cuda")
    x[:, ::7] = top
    x[:, 3::7] = -3.4e38
    W = torch.randn(d_out, d_in, generator=g, device="cuda") / 2.0 ** 20
    want = x.double() @ W.double().t()
    tol = (d_in + 4) * 2 * U * (x.double().abs() @ W.double().abs().t())
    close(moe.moe_linear(x, W), want, tol + U * want.abs(), "y")


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_infinite_values_stay_in_their_row(shape):
    """An infinite x: fp32's own infinities from the CUDA cores (a few tokens), NaN
    from the tensor cores, whose parts of it are no numbers; other rows keep their
    bits.  A NaN gives NaN."""
    require_gpu()
    n, d_in, d_out = shape
    g = gen(n + 3)
    x = torch.randn(n, d_in, generator=g, device="cuda")
    W = torch.randn(d_out, d_in, generator=g, device="cuda")
    y = moe.moe_linear(x, W)
    z = x.clone()
    z[1, 5] = float("inf")
    z[3, 7] = float("-inf")
    z[4, d_in - 1] = float("nan")
    got = moe.moe_linear(z, W)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[1, 3, 4]] = False
    assert torch.equal(got[keep], y[keep])
    assert bool(got[4].isnan().all())
    if shape == FEW:
        assert torch.equal(got[1], W[:, 5].sign() * float("inf"))
        assert torch.equal(got[3], -W[:, 7].sign() * float("inf"))
    else:
        assert bool(got[1].isnan().all()) and bool(got[3].isnan().all())

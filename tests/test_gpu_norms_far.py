"""Layer norm of rows that are far from zero and hardly spread: what the mean's rounding leaves must not show.

Bounds, with F = 2^-24 half an fp32 step.  A sum of a row goes through at most K additions and products.  The kernels take a
row's deviations from a pivot that is a mean in fp32, off by e = K F max|x| at most.  With S = max|x - mean|, deviations and
the distances of pivots are at most 2 S + 2 e in size, each rounded by F of itself, and sums of them divided by their number
are off by K F (2 S + 2 e): n / rstd is off by (K + 8) F (4 S + 4 e), a row's mean square by (2 K + 20) F (2 S + 2 e)^2.  The mean
that is stored is rounded once."""
import pytest
import torch

from tests._gpu import require_gpu
from tests._norms import DEPTH, F, RSQRT, half_step
from tests.test_gpu_norms import Norm

pytestmark = pytest.mark.gpu
K = DEPTH + 8


def _check(n, eps):
    x = n.x.t.double()
    w, b = n.weight.double(), n.bias.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    y = d * rstd * w + b
    e, s = K * F * x.abs().amax(1, keepdim=True), d.abs().amax(1, keepdim=True)
    dd, dv = (K + 8) * F * (4 * s + 4 * e), (2 * K + 20) * F * (2 * s + 2 * e).square()
    high, low = ((var - dv).clamp(min=0) + eps).rsqrt() * (1 + RSQRT + 2 * F), (var + dv + eps).rsqrt() * (1 - RSQRT - 2 * F)
    off = high * dd + d.abs() * torch.maximum(high - rstd, rstd - low)
    err = w.abs() * off + 4 * F * ((d * rstd * w).abs() + b.abs())
    half, least = half_step(n.dtype)
    for name, got, ref, tol in (("y", n.out.t, y, err + (half + F) * (y.abs() + err) + least),
                                ("mean", n.mean[:, None], mean, dd + F * (mean.abs() + dd))):
        over = (got.double() - ref).abs() - tol
        assert (over <= 0).all(), f"{name}: off by {float((got.double() - ref).abs().max()):.3g}, {float(over.max()):.3g} over its bound"
    got = n.rstd.double()[:, None]
    assert ((got <= high * (1 + F)) & (got >= low * (1 - F))).all(), f"rstd: {got.min()} {got.max()}, {low.min()} {high.max()}"


WIDTHS = [1, 3, 33, 257, 512, 515, 1000, 1155, 1536, 2560, 4096, 5003, 8192, 10007, 16384]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("value", [100.1, -3000.1, 100000.1, 1e8])
def test_constant_rows(width, value):
    mi = require_gpu()
    for kind in ("f32", "bf16", "f16"):
        if kind == "f16" and abs(value) > 65504:
            continue
        n = Norm(37, width, kind)
        n.x.t[:] = value
        n.x.t[5] = -value
        n.forward(mi)
        _check(n, 1e-6)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_small_spread_far_from_zero(width, kind):
    """A few steps of the type around a value."""
    mi = require_gpu()
    for value in (100.1, -3000.1, 30000.1):
        n = Norm(37, width, kind)
        at = torch.tensor(value).to(n.dtype)
        step = 2.0 ** (torch.frexp(at.float())[1].item() - 1) * torch.finfo(n.dtype).eps
        g = torch.Generator(device="cuda").manual_seed(width)
        n.x.t.copy_(at.double().cuda() + step * torch.randint(-3, 4, (37, width), generator=g, device="cuda"))
        n.forward(mi)
        _check(n, 1e-6)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_the_largest_values_that_are_promised(width, kind):
    """|x| just below 2^66, deviations just below 2^50 (bf16: no smaller ones than steps of 2^58 there, so |x| below 2^50)."""
    mi = require_gpu()
    n = Norm(37, width, kind)
    g = torch.Generator(device="cuda").manual_seed(width)
    at = 2.0 ** 65.9 if kind == "f32" else 0.0
    n.x.t.copy_(at + (2 * torch.rand(37, width, generator=g, device="cuda", dtype=torch.float64) - 1) * 2.0 ** 48.9)
    n.forward(mi)
    _check(n, 1e-6)

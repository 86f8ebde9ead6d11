"""64-bit forms of the norms' forward and backward passes and the error bounds of the kernels, element by element.

F = 2^-24 is half an fp32 step relative to the value, eps(t) / 2 half a step of the output's type.  Inputs are exact.  A
row's sum goes through at most DEPTH additions in a kernel (a thread's own terms, a tree over a warp, one over the warps of
a row), so it is off by at most DEPTH F times the sum of its terms' absolute values; a sum over rows through at most
rows / 100 + 400 (a part's rows, the parts), or as many as there are rows.  rsqrt is good to 2 units of the last place, 2^-22."""
import torch

F = 2.0 ** -24
DEPTH = 96
RSQRT = 2.0 ** -22
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dtype):
    """(half a step relative to the value, half the smallest step) of a type."""
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def row_depth(rows):
    return min(rows, rows // 100 + 400) + 2


def rounded(value, err, dtype):
    """Bound of an output of a type: `err` before its one rounding."""
    u, least = half_step(dtype)
    return err + (u + F) * (value.abs() + err) + least


def layer_norm64(x, weight, bias, eps):
    """x [rows, width] of any type; weight, bias [width] or None.  Returns y, mean, rstd and y_tol, mean_tol, rstd_tol."""
    dtype, x = x.dtype, x.double()
    w = torch.ones_like(x[0]) if weight is None else weight.double()
    b = torch.zeros_like(x[0]) if bias is None else bias.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = d * rstd
    y = n * w + b
    dm = (DEPTH + 2) * F * x.abs().mean(1, keepdim=True)
    # the squares are of x - (mean + dm): var + dm^2 exactly, with roundings of d, of the products and of the sum
    dv = (DEPTH + 6) * F * (var + dm.square()) + dm.square()
    rel = 0.5 * dv / (var + eps) * (1 + 2 * dv / (var + eps)) + RSQRT + 2 * F
    dn = rstd * (dm + F * d.abs()) * (1 + rel) + n.abs() * (rel + 2 * F)
    err = w.abs() * dn + 2 * F * ((w * n).abs() + b.abs())
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "y_tol": rounded(y, err, dtype), "mean_tol": dm[:, 0] + 1e-44,
            "rstd_tol": (rel * rstd)[:, 0]}


def norm_backward64(dy, x, factor, mean, rstd, residual=None, rel=0.0):
    """dy, x [rows, width]; factor [width] (the weight), mean, rstd [rows, 1] in 64 bits; mean None: an rms norm.  rel:
    how far the kernel's own rstd may be off.  Rows whose dy is zero count as x = mean."""
    dtype = x.dtype
    dead = (dy == 0).all(1, keepdim=True)
    dy, x = dy.double(), torch.where(dead, torch.zeros_like(x), x).double()
    rstd = torch.where(dead, torch.ones_like(rstd), rstd)
    m = torch.zeros_like(rstd) if mean is None else torch.where(dead, torch.zeros_like(mean), mean)
    r = torch.zeros_like(x) if residual is None else residual.double()
    n, g = (x - m) * rstd, dy * factor
    c2 = (g * n).mean(1, keepdim=True)
    c1 = torch.zeros_like(c2) if mean is None else g.mean(1, keepdim=True)
    dx = r + rstd * (g - c1 - n * c2)
    dx = torch.where(dead, r, dx)
    n_rel = rel + 3 * F
    e1 = (DEPTH + 3) * F * g.abs().mean(1, keepdim=True)
    e2 = ((DEPTH + 8) * F + n_rel) * (g * n).abs().mean(1, keepdim=True)
    size = rstd * (g.abs() + c1.abs() + (n * c2).abs())
    err = (8 * F + 2 * rel + n_rel) * size + rstd * (e1 + n.abs() * e2) * (1 + 4 * n_rel) + F * r.abs()
    terms, depth = (dy * n).abs(), row_depth(len(x)) * F
    return {"dx": dx, "dx_tol": rounded(dx, err, dtype), "dweight": (dy * n).sum(0),
            "dweight_tol": (depth + n_rel) * terms.sum(0) + 1e-40, "dbias": dy.sum(0), "dbias_tol": depth * dy.abs().sum(0) + 1e-40}


def rms64(x, eps):
    """1 / root mean square [rows, 1] in 64 bits, and how far the kernel's may be off relative to it."""
    return (x.double().square().mean(1, keepdim=True) + eps).rsqrt(), 0.5 * (DEPTH + 4) * F + RSQRT + 2 * F


def within(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - ref).abs() - tol
    assert (off <= 0).all(), f"{what}: off by {float((got - ref).abs().max()):.3g}, at worst {float(off.max()):.3g} over its bound"

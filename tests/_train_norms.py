"""Checks of the training pass that a wrong gradient does not pass: errors in the 2-norm.

U = 2^-8 is half a bf16 step relative to the value.  An output of the pass has two roundings on its way that
count: P or dS as a matrix operand and the output itself, each at most U of the value it rounds.  The
operand's add up over the terms of a sum as the terms do (in quadrature, for terms of either sign), so each
rounding has at most U of the output's 2-norm and both together 2 U; D, lse and the sums add fp32 errors and
the rounding of o, which is averaged over 128 columns.  (A uniform rounding error has about U / sqrt(5) in the
mean square, two of them 0.0025.)  A gradient of a common 2 % too much is 2.5 times that bound."""
import math

import torch

from tests._train import F, HEAD, U

NORM_TOL = 2 * U


def norm_error(got, ref):
    """|got - ref| / |ref| in the 2-norm, not finite where got is not."""
    return float((got.double() - ref).norm() / ref.norm())


def close_in_norm(got, ref, what):
    err = norm_error(got, ref)
    assert err <= NORM_TOL, f"{what}: off by {err:.3g} of its norm, at most {NORM_TOL:.3g}"


def directions(ref, gen, count=3):
    """Unit vectors with a good part along ref: ref's own direction, and that with as much of a random one."""
    along = ref / ref.norm()
    yield along
    for _ in range(count):
        u = torch.randn(ref.shape, generator=gen, device=ref.device, dtype=torch.float64)
        u = along + u / u.norm()
        yield u / u.norm()


def agrees_with_difference(got, u, diff, size, what):
    """got along the unit vector u against a central difference: |(got - g) u| <= |got - g| <= 2 U |g|; the
    difference itself is off by its step squared and by 1e-16 over the step, far below."""
    slope = float((got.double() * u).sum())
    assert abs(slope - diff) <= NORM_TOL * size + 1e-5 * (abs(diff) + 1), f"{what}: {slope} along u, differences give {diff}"


def head64(q, k, v, keys, d_o=None, chunk=2048):
    """One head in 64 bits, some queries at a time: q, k, v, d_o float64 [seq, 128], keys: indices of the valid
    ones.  Returns o, lse and its tolerance, and dq, dk, dv."""
    kk, vv = k[keys], v[keys]
    top = kk.norm(dim=1).max()
    out = {n: torch.zeros_like(q) for n in ("o", "dq", "dk", "dv")}
    out["lse"], out["lse_tol"] = torch.empty_like(q[:, 0]), torch.empty_like(q[:, 0])
    dk, dv = torch.zeros_like(kk), torch.zeros_like(vv)
    sc = 1.0 / math.sqrt(HEAD)
    for i in range(0, len(q), chunk):
        at = slice(i, i + chunk)
        z = q[at] @ kk.T * sc
        lse = torch.logsumexp(z, 1)
        out["lse"][at] = lse
        # a score's terms add up to |q| |k| at most; fp32 sums of them and of the exponentials, as in attention64
        out["lse_tol"][at] = ((HEAD + 4) * F * sc * q[at].norm(dim=1) * top + 8 * F * (1.0 + lse.abs()) + (len(keys) + 8) * F
                              + 2.0 ** -21)
        p = z.sub_(lse[:, None]).exp_()
        out["o"][at] = p @ vv
        if d_o is None:
            continue
        dv += p.T @ d_o[at]
        dp = d_o[at] @ vv.T
        dp.sub_((dp * p).sum(1, keepdim=True)).mul_(p).mul_(sc)
        out["dq"][at] = dp @ kk
        dk += dp.T @ q[at]
    out["dk"][keys], out["dv"][keys] = dk, dv
    return out

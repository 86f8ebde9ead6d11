"""64-bit forms of the training pass and the error bounds of its kernels, element by element.

Roundings counted: U = 2^-8 is half a bf16 step relative to the value, F = 2^-24 half an fp32 step.
The kernels round P and dS to bf16 once (as matrix operands) and each output once; everything else is
fp32.  `A` below is the sum of the absolute values of the terms of a sum: a sum of n fp32 terms in any
order is off by at most n F A."""
import math

import torch

U = 2.0 ** -8
F = 2.0 ** -24
HEAD = 128


def heads_of(t, batch, seq, heads):
    """[batch * seq, heads * 128] -> float64 [batch, heads, seq, 128]"""
    return t.reshape(batch, seq, heads, HEAD).permute(0, 2, 1, 3).double()


def attention64(q, k, v, mask, d_o=None, with_bounds=True):
    """q, k, v, d_o: float64 [batch, heads, seq, 128]; mask uint8 [batch, seq] or None.  Returns a dict of
    values and, under "name_tol", how far a kernel's value may be off."""
    seq = q.shape[2]
    z = q @ k.transpose(2, 3) / math.sqrt(HEAD)
    za = q.abs() @ k.abs().transpose(2, 3) / math.sqrt(HEAD)
    if mask is not None:
        off = (mask == 0)[:, None, None, :]
        z = z.masked_fill(off, -math.inf)
        za = za.masked_fill(off, 0.0)
        keep = (mask != 0)[:, None, :, None]
        k = torch.where(keep, k, torch.zeros_like(k))  # a masked key's row may hold anything
        v = torch.where(keep, v, torch.zeros_like(v))
        z = torch.where(off, torch.full_like(z, -math.inf), z)
        za = torch.where(off, torch.zeros_like(za), za)
    lse = torch.logsumexp(z, 3)
    empty = lse == -math.inf
    p = torch.exp(z - torch.where(empty, torch.zeros_like(lse), lse).unsqueeze(3))
    r = {"lse": lse, "o": p @ v}
    # a score is a sum of 128 products and its exponent in base 2 one more fma; lse adds seq terms
    s_err = (HEAD + 4) * F * za.amax(3) + 8 * F * (1.0 + torch.where(empty, torch.zeros_like(lse), lse.abs()))
    p_rel = s_err + (seq + 8) * F + 2.0 ** -21       # exp2 of the unit: two units of the last place
    r["lse_tol"] = p_rel
    pr = p_rel.unsqueeze(3)
    pa = p @ v.abs()
    r["o_tol"] = (U + 2 * pr + (seq + 8) * F) * pa + U * r["o"].abs() + 1e-30
    if d_o is None:
        return r
    g = d_o
    dp, dpa = g @ v.transpose(2, 3), g.abs() @ v.abs().transpose(2, 3)
    d = (p * dp).sum(3, keepdim=True)
    ds = p * (dp - d)
    sc = 1.0 / math.sqrt(HEAD)
    r["dq"], r["dk"], r["dv"] = ds @ k * sc, ds.transpose(2, 3) @ q * sc, p.transpose(2, 3) @ g
    d_err = (g.abs() * (r["o_tol"] + HEAD * F * r["o"].abs())).sum(3, keepdim=True)
    da = dp.abs() + d.abs()
    ds_err = U * ds.abs() * (1 + U) + p * ((1 + 2 * U) * (d_err + HEAD * F * dpa + 4 * F * da) + 2 * pr * da)
    dsa = ds.abs() + ds_err
    r["dq_tol"] = (ds_err @ k.abs() + (seq + 8) * F * (dsa @ k.abs())) * sc + U * r["dq"].abs() + 1e-30
    r["dk_tol"] = (ds_err.transpose(2, 3) @ q.abs() + (seq + 8) * F * (dsa.transpose(2, 3) @ q.abs())) * sc + U * r["dk"].abs() + 1e-30
    r["dk_tol"] = r["dk_tol"] * (1 + U)
    r["dq_tol"] = r["dq_tol"] * (1 + U)
    dva = p.transpose(2, 3) @ g.abs()
    dvp = (p * (2 * pr)).transpose(2, 3) @ g.abs()
    r["dv_tol"] = (U * dva + dvp + (seq + 8) * F * dva + U * r["dv"].abs()) * (1 + U) + 1e-30
    return r


def qk_backward64(x, gain, cos, sin, dy, eps):
    """x float64 [batch, seq, heads, 128] raw, dy float64 the same, cos/sin float64 [batch or 1, seq, 1, 64].
    Returns dx, dgain and their tolerances."""
    a, b = dy[..., 0::2], dy[..., 1::2]
    dz = torch.stack([a * cos + b * sin, b * cos - a * sin], 4).flatten(3)
    dza = torch.stack([(a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()], 4).flatten(3)
    r = torch.rsqrt(x.square().mean(3, keepdim=True) + eps)
    n = x * r
    t, ta = dz * gain, dza * gain.abs()
    dx = r * (t - n * (t * n).mean(3, keepdim=True))
    dxa = r * (ta + n.abs() * (ta * n.abs()).mean(3, keepdim=True))
    # fp32 up to the one output rounding: chains of at most 8 + 4 adds and a dozen products
    dx_tol = (U * dx.abs() + 32 * F * dxa) * (1 + U) + 1e-30
    dgain = (dz * n).sum((0, 1, 2))
    # a chain adds at most 2^8 terms in a lane, 8 warps and 2^9 CTAs; each term has a few roundings
    dgain_tol = (2 ** 8 + 2 ** 9 + 32) * F * (dza * n.abs()).sum((0, 1, 2)) + 1e-30
    return dx, dx_tol, dgain, dgain_tol


def within(got, ref, tol, what):
    got = got.double()
    err = (got - ref).abs()
    bad = ~(err <= tol) & ~((ref == got) | (ref.isnan() & got.isnan()))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values are off, worst "
                           f"{float((err / tol)[bad].max()):.3g} x its bound")

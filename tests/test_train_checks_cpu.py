"""The checks of tests/_train_norms.py without a GPU: they take a rounded pass, and nothing that is wrong.  Refusals
made before a device is touched."""
import math

import pytest
import torch

from tests._train import attention64
from tests._train_norms import agrees_with_difference, close_in_norm, directions, head64
from tests.test_train_cpu import MB, P, _axes, _refused, lib  # noqa: F401


def _bf(t):
    return t.bfloat16().double()


@pytest.fixture(scope="module")
def rounded():
    """A pass of two elements (padded keys in the last) with the kernels' roundings: the right values, and those
    with P, dS, o and every output in bf16."""
    gen = torch.Generator().manual_seed(11)
    q, k, v, g = (_bf(torch.randn(2, 2, 150, 128, generator=gen, dtype=torch.float64)) for _ in range(4))
    mask = torch.ones(2, 150, dtype=torch.uint8)
    mask[1, 30:80] = 0
    ref = attention64(q, k, v, mask, g)
    z = (q @ k.transpose(2, 3) / math.sqrt(128)).masked_fill((mask == 0)[:, None, None, :], -math.inf)
    p = torch.exp(z - ref["lse"].unsqueeze(3))
    o = _bf(_bf(p) @ v)
    ds = _bf(p * (g @ v.transpose(2, 3) - (g * o).sum(3, keepdim=True))) / math.sqrt(128)
    got = {"o": o, "dq": _bf(ds @ k), "dk": _bf(ds.transpose(2, 3) @ q), "dv": _bf(_bf(p).transpose(2, 3) @ g)}
    return (q, k, v, g, mask), ref, got


WRONG = {"zero": lambda t: t * 0, "negated": lambda t: -t, "2 % too much": lambda t: t * 1.02, "2 % too little": lambda t: t * 0.98,
         "another head's": lambda t: t.flip(1), "not finite": lambda t: t * math.nan}


@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv"])
def test_norms_take_roundings_and_nothing_else(rounded, name):
    _, ref, got = rounded
    close_in_norm(got[name], ref[name], name)
    for what, wrong in WRONG.items():
        with pytest.raises(AssertionError, match=name):
            close_in_norm(wrong(got[name]), ref[name], name)
            pytest.fail(f"passes: {what}")


@pytest.mark.parametrize("name", ["dq", "dk", "dv"])
def test_differences_take_roundings_and_nothing_else(rounded, name):
    (q, k, v, g, mask), ref, got = rounded
    i = ("dq", "dk", "dv").index(name)

    def loss(t, u):
        x = [q, k, v]
        x[i] = x[i] + t * u
        return float((attention64(*x, mask)["o"] * g).sum())

    size = float(ref[name].norm())
    for u in directions(ref[name], torch.Generator().manual_seed(12)):
        diff = (loss(1e-4, u) - loss(-1e-4, u)) / 2e-4
        agrees_with_difference(got[name], u, diff, size, name)
        for what in ("zero", "negated", "not finite"):
            with pytest.raises(AssertionError, match="differences"):
                agrees_with_difference(WRONG[what](got[name]), u, diff, size, name)
        with pytest.raises(AssertionError, match="differences"):
            agrees_with_difference(got[name] * 1.05, u, diff, size, name)


def test_one_head_by_chunks_is_the_whole(rounded):
    (q, k, v, g, mask), ref, _ = rounded
    r = head64(q[1, 0], k[1, 0], v[1, 0], mask[1].nonzero().flatten(), g[1, 0], chunk=64)
    for name in ("o", "lse", "dq", "dk", "dv"):
        assert torch.allclose(r[name], ref[name][1, 0], rtol=1e-10, atol=1e-12), name


@pytest.mark.parametrize("change", [
    dict(cos=P + MB, sin=P + MB), dict(cos=P + MB, sin=P + MB + 10 * 256 - 16), dict(cos=P + MB + 10 * 256 - 16, sin=P + MB),
    dict(pos=P + MB), dict(pos=P + 2 * MB + 10 * 256 - 4), dict(pos=P + 2 * MB - 10 * 12 + 4)])
def test_rope_axes_refuses_tables_that_overlap(lib, change):  # noqa: F811
    _refused(lib, _axes(lib, **change), 1, "overlaps")


@pytest.mark.parametrize("change", [dict(cos=P + MB, sin=P + MB + 10 * 256), dict(pos=P + 2 * MB + 10 * 256), dict(pos=P + 2 * MB - 10 * 12)])
def test_rope_axes_takes_tables_that_touch(lib, change):  # noqa: F811
    """(Only without a GPU, where the call ends at the device it needs.)"""
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not the device's")
    assert _axes(lib, **change) not in (0, 1), lib.mi_last_error()

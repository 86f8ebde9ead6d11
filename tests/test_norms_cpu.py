"""Norms' gradients and gradient clipping without a GPU: the 64-bit forms against autograd, what their bounds let pass,
and the refusals of the calls (all made before a device is touched)."""
import ctypes
import math

import pytest
import torch

from tests._norms import layer_norm64, norm_backward64, rms64

P = 1 << 20  # an aligned address that is never read
MB = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from diffusion_transformer_denoiser_gb300 import _build
    import diffusion_transformer_denoiser_gb300 as mi

    _build.build()
    return mi.lib()


@pytest.mark.parametrize("width", [1, 5, 64])
@pytest.mark.parametrize("rms", [False, True])
def test_formulas_against_autograd(width, rms):
    gen = torch.Generator().manual_seed(width)
    x = torch.randn(7, width, generator=gen, dtype=torch.float64, requires_grad=True)
    w, b = (torch.randn(width, generator=gen, dtype=torch.float64, requires_grad=True) for _ in range(2))
    dy = torch.randn(7, width, generator=gen, dtype=torch.float64)
    if rms:
        r, _ = rms64(x.detach(), 1e-3)
        y = x * (x.square().mean(1, keepdim=True) + 1e-3).rsqrt() * w + b
        ref = norm_backward64(dy, x.detach(), w.detach(), None, r)
    else:
        f = layer_norm64(x.detach(), w.detach(), b.detach(), 1e-3)
        y = torch.nn.functional.layer_norm(x, (width,), w, b, 1e-3)
        assert torch.allclose(f["y"], y, rtol=1e-12, atol=1e-13)
        ref = norm_backward64(dy, x.detach(), w.detach(), f["mean"][:, None], f["rstd"][:, None])
    (y * dy).sum().backward()
    for got, want in ((x.grad, ref["dx"]), (w.grad, ref["dweight"]), (b.grad, ref["dbias"])):
        assert torch.allclose(got, want, rtol=1e-10, atol=1e-12)


def test_the_bounds_do_not_let_a_wrong_gradient_pass():
    """What leaves out the mean's part, the projection or 2 % of a gradient is outside the bounds."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(40, 256, generator=gen).bfloat16()
    dy = (torch.randn(40, 256, generator=gen) + 0.5).bfloat16()
    w = torch.ones(256, dtype=torch.float64)
    f = layer_norm64(x, None, None, 1e-6)
    mean, rstd = f["mean"][:, None], f["rstd"][:, None]
    ref = norm_backward64(dy, x, w, mean, rstd)
    g, n = dy.double(), (x.double() - mean) * rstd
    wrong = {"mean": rstd * (g - n * (g * n).mean(1, keepdim=True)), "projection": rstd * (g - g.mean(1, keepdim=True)),
             "scaled": ref["dx"] * 1.02}
    for name, dx in wrong.items():
        assert ((dx - ref["dx"]).abs() > ref["dx_tol"]).double().mean() > 0.5, name
    assert (0.02 * ref["dweight"].abs() > ref["dweight_tol"]).double().mean() > 0.9
    assert (0.02 * (f["y"].abs()) > f["y_tol"]).double().mean() > 0.9


def _refused(lib, status, want, needle):
    assert status == want, (status, lib.mi_last_error())
    assert needle in lib.mi_last_error().decode(), lib.mi_last_error()


FWD = dict(x=P, x_stride=64, weight=P + MB, bias=P + 2 * MB, out=P + 3 * MB, out_stride=64, mean=P + 4 * MB, rstd=P + 5 * MB,
           rows=10, width=64, eps=1e-6, dtype=0, param_dtype=0, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(x=None), 1, "null"), (dict(out=None), 1, "null"), (dict(x=P + 1), 1, "aligned"), (dict(out=P + 3 * MB + 1), 1, "aligned"),
    (dict(weight=P + MB + 2, param_dtype=2), 1, "aligned"), (dict(mean=P + 4 * MB + 2), 1, "aligned"), (dict(rows=-1), 1, "rows"),
    (dict(width=0), 1, "width"), (dict(width=16385), 2, "16384"), (dict(eps=-1e-6), 1, "eps"), (dict(eps=math.nan), 1, "eps"),
    (dict(dtype=3), 1, "mi_dtype"), (dict(dtype=-1), 1, "mi_dtype"), (dict(param_dtype=1), 2, "param_dtype"),
    (dict(dtype=2, param_dtype=0), 2, "param_dtype"), (dict(x_stride=63), 1, "overlap"), (dict(x_stride=-64), 1, "overlap"),
    (dict(out_stride=0), 1, "overlap"), (dict(rows=1, x_stride=-64), 1, "stride"), (dict(out=P), 1, "overlaps"),
    (dict(out=P + 64 * 19), 1, "overlaps"), (dict(out=P + 128, out_stride=128, x_stride=127), 1, "overlaps"),
    (dict(out=P + 126, out_stride=128, x_stride=128), 1, "overlaps"),
    (dict(mean=P + 5 * MB + 36), 1, "overlaps"), (dict(rstd=P + MB), 1, "overlaps"), (dict(out=P + 2 * MB), 1, "overlaps")])
def test_layer_norm_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_layer_norm(*{**FWD, **change}.values()), want, needle)


def test_layer_norm_takes_what_it_can(lib):
    """Arguments that pass every check but the last one, which is eps's; and no rows are no call."""
    assert lib.mi_layer_norm(*{**FWD, "rows": 0, "x": None, "out": None}.values()) == 0
    for change in (dict(), dict(weight=None, bias=None, mean=None, rstd=None), dict(x_stride=0), dict(x=P + 2),
                   dict(out=P + 128, out_stride=128, x_stride=128), dict(rows=1, x_stride=0)):
        _refused(lib, lib.mi_layer_norm(*{**FWD, **change, "eps": -1.0}.values()), 1, "eps")


BWD = dict(dy=P, dy_stride=64, x=P + MB, x_stride=64, weight=P + 2 * MB, mean=P + 3 * MB, rstd=P + 4 * MB, residual=P + 5 * MB,
           residual_stride=64, dx=P + 6 * MB, dx_stride=64, dweight=P + 7 * MB, dbias=P + 8 * MB, rows=10, width=64, dtype=0,
           param_dtype=0, ws=P + 9 * MB, ws_bytes=MB, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(dy=None), 1, "null"), (dict(x=None), 1, "null"), (dict(dx=None), 1, "null"), (dict(mean=None), 1, "null"),
    (dict(rstd=None), 1, "null"), (dict(dy=P + 1), 1, "aligned"), (dict(dweight=P + 7 * MB + 2), 1, "aligned"),
    (dict(rows=-5), 1, "rows"), (dict(width=-1), 1, "width"), (dict(width=20000), 2, "16384"), (dict(dtype=7), 1, "mi_dtype"),
    (dict(param_dtype=1), 2, "param_dtype"), (dict(dx_stride=10), 1, "overlap"), (dict(dx_stride=0), 1, "overlap"),
    (dict(residual_stride=60), 1, "overlap"), (dict(ws=P + 9 * MB + 16), 3, "256-byte"), (dict(ws=None), 3, "256-byte"),
    (dict(dx=P), 1, "overlaps"), (dict(dx=P + MB), 1, "overlaps"), (dict(dx=P + 5 * MB, dx_stride=65), 1, "overlaps"),
    (dict(dx=P + 5 * MB + 2), 1, "overlaps"), (dict(dweight=P + 8 * MB), 1, "overlaps"), (dict(dbias=P + 3 * MB), 1, "overlaps"),
    (dict(ws=P + 4 * MB), 1, "overlaps")])
def test_layer_norm_backward_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_layer_norm_backward(*{**BWD, **change}.values()), want, needle)


def test_layer_norm_backward_takes_what_it_can(lib):
    """The workspace's address is the last check."""
    for change in (dict(), dict(dx=P + 5 * MB), dict(residual=None), dict(dweight=None, dbias=None, weight=None), dict(dy_stride=0)):
        _refused(lib, lib.mi_layer_norm_backward(*{**BWD, **change, "ws": BWD["ws"] + 64}.values()), 3, "256-byte")


MOD = dict(dy=P, x=P + MB, mod=P + 2 * MB, shift_row=0, scale_row=1, residual=P + 3 * MB, dx=P + 4 * MB, dmod=P + 5 * MB, batch=2,
           seq=10, hidden=256, eps=1e-6, ws=P + 6 * MB, ws_bytes=MB, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(dy=None), 1, "null"), (dict(dmod=None), 1, "null"), (dict(residual=P + 3 * MB + 2), 1, "aligned"),
    (dict(dmod=P + 5 * MB + 4), 1, "aligned"), (dict(batch=0), 1, "positive"), (dict(seq=-3), 1, "positive"),
    (dict(hidden=128), 2, "256"), (dict(hidden=4352), 2, "4096"), (dict(batch=1 << 16, seq=1 << 15), 2, "2^30"),
    (dict(shift_row=6), 1, "0..5"), (dict(scale_row=-1), 1, "0..5"), (dict(eps=-1.0), 1, "eps"), (dict(ws=None), 3, "256-byte"),
    (dict(ws=P + 6 * MB + 128), 3, "256-byte"), (dict(dx=P), 1, "overlaps"), (dict(dx=P + 3 * MB + 16), 1, "overlaps"),
    (dict(dmod=P + 2 * MB), 1, "overlaps"), (dict(ws=P + MB), 1, "overlaps")])
def test_mod_backward_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_mod_rmsnorm_backward(*{**MOD, **change}.values()), want, needle)
    _refused(lib, lib.mi_mod_rmsnorm_backward(*{**MOD, "dx": MOD["residual"], "ws": None}.values()), 3, "256-byte")


def _set(lib, tensors, outs=None, dtypes=None, n=None):
    """tensors: (address, count) of each."""
    n = len(tensors) if n is None else n
    h = ctypes.c_void_p()
    arr = ctypes.c_void_p * max(1, len(tensors))
    st = lib.mi_grads_init(ctypes.byref(h), n, arr(*[a for a, _ in tensors]), None if outs is None else arr(*outs),
                           (ctypes.c_int64 * max(1, len(tensors)))(*[c for _, c in tensors]),
                           (ctypes.c_int * max(1, len(tensors)))(*(dtypes or [2] * len(tensors))))
    return st, h


@pytest.mark.parametrize("tensors,outs,dtypes,needle", [
    ([(None, 3)], None, None, "null"), ([(P, 3)], [None], None, "null"), ([(P + 2, 3)], None, None, "aligned"),
    ([(P + 1, 3)], None, [0], "aligned"), ([(P, -1)], None, None, "count"), ([(P, 1 << 50)], None, None, "count"),
    ([(P, 3)], None, [3], "mi_dtype"), ([(P, 3), (P, 3)], None, None, "overlaps"), ([(P, 3), (P + 8, 3)], None, None, "overlaps"),
    ([(P + 8, 3), (P, 100), (P + 4 * MB, 1)], None, None, "overlaps"), ([(P, 8)], [P + 16], None, "overlaps"),
    ([(P, 4), (P + MB, 4)], [P + MB, P + 2 * MB], None, "overlaps"), ([(P, 4), (P + MB, 4)], [P + 2 * MB] * 2, None, "overlaps"),
    ([(P, 4), (P, 4)], [P, P + MB], None, "overlaps")])
def test_grad_set_refusals(lib, tensors, outs, dtypes, needle):
    st, h = _set(lib, tensors, outs, dtypes)
    _refused(lib, st, 1, needle)
    assert not h.value


def test_grad_set_takes_what_it_can(lib):
    for tensors, outs, dtypes in (([], None, None), ([(None, 0), (P, 3)], None, None), ([(P, 4), (P + 16, 4)], None, None),
                                  ([(P, 4), (P, 4)], [P + 16, P + 32], None), ([(P, 4), (P + 8, 1)], [P, P + 64], [0, 2]),
                                  ([(P + 2, 4)], [P + MB + 6], [1])):
        st, h = _set(lib, tensors, outs, dtypes)
        assert st == 0, lib.mi_last_error()
        lib.mi_grads_destroy(h)
    _refused(lib, _set(lib, [(P, 3)], n=-1)[0], 1, "negative")
    _refused(lib, lib.mi_grads_init(None, 0, None, None, None, None), 1, "null")


def test_grad_call_refusals(lib):
    st, h = _set(lib, [(P, 100), (P + MB, 7)])
    w = P + 2 * MB
    _refused(lib, lib.mi_grad_norm(h, None, w, 4096, None), 1, "null")
    _refused(lib, lib.mi_grad_norm(None, w, w, 4096, None), 1, "null")
    _refused(lib, lib.mi_grad_norm(h, P + 3 * MB + 2, w, 4096, None), 1, "aligned")
    _refused(lib, lib.mi_grad_norm(h, P + 3 * MB, w + 64, 4096, None), 3, "256-byte")
    _refused(lib, lib.mi_grad_norm(h, P + 3 * MB, None, 4096, None), 3, "256-byte")
    for at in (P + 396, P + MB, w + 4092):
        _refused(lib, lib.mi_grad_norm(h, at, w, 4096, None), 1, "overlaps")
    _refused(lib, lib.mi_grad_norm(h, P + 3 * MB, P, 4096, None), 1, "overlaps")
    for limit in (0.0, -2.0, math.inf, math.nan):
        _refused(lib, lib.mi_grad_clip(h, limit, P + 3 * MB, None), 1, "max_norm")
        _refused(lib, lib.mi_grad_clip_norm(h, limit, P + 3 * MB, w, 4096, None), 1, "max_norm")
    n = ctypes.c_size_t(0)
    _refused(lib, lib.mi_grads_workspace_size(None, ctypes.byref(n)), 1, "null")
    _refused(lib, lib.mi_layer_norm_backward_workspace_size(-1, 5, ctypes.byref(n)), 1, "rows")
    _refused(lib, lib.mi_mod_rmsnorm_backward_workspace_size(1, 5, 100, ctypes.byref(n)), 2, "256")
    lib.mi_grads_destroy(h)


def test_binding_refuses_wrong_tensors():
    import diffusion_transformer_denoiser_gb300 as mi

    t = torch.empty(10, 64)
    for call in (lambda: mi.layer_norm(t, None, None, t), lambda: mi.layer_norm_backward(t, t, None, t, t, t, t, t, t),
                 lambda: mi.mod_rmsnorm_backward(t, t, t, 0, 1, t, t, 1, 10, t), lambda: mi.GradSet([t])):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    with pytest.raises(ValueError, match="outs"):
        mi.GradSet([t], [])
    assert mi._rows(t, torch.float32, 10, 64, "x", -1) == (t.data_ptr(), 64)
    assert mi._rows(t[:, 8:24], torch.float32, 10, 16, "x", -1) == (t.data_ptr() + 32, 64)
    assert mi._rows(t.view(2, 5, 64), torch.float32, 10, 64, "x", -1) == (t.data_ptr(), 64)
    for bad, needle in ((t[:, ::2], "contiguous"), (t.T, "contiguous"), (t.view(5, 2, 64)[:, :1], "contiguous"), (t[:5], "rows")):
        with pytest.raises(ValueError, match=needle):
            mi._rows(bad, torch.float32, bad.numel() // bad.shape[-1] if needle != "rows" else 10, bad.shape[-1], "x", -1)
    with pytest.raises(TypeError, match="expected torch.float16"):
        mi._rows(t, torch.float16, 10, 64, "x", -1)

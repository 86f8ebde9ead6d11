"""The training pass without a GPU: the 64-bit forms against differences, and the refusals of its calls
(all made before a device is touched)."""
import ctypes
import math

import pytest
import torch

from tests._train import attention64, qk_backward64

P = 1 << 20  # an aligned address that is never read
MB = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from diffusion_transformer_denoiser_gb300 import _build
    import diffusion_transformer_denoiser_gb300 as mi

    _build.build()
    return mi.lib()


def test_attention_formulas_against_differences():
    gen = torch.Generator().manual_seed(3)
    q, k, v, g = (torch.randn(2, 2, 9, 128, generator=gen, dtype=torch.float64) for _ in range(4))
    mask = torch.ones(2, 9, dtype=torch.uint8)
    mask[0, 2:5] = 0
    r = attention64(q, k, v, mask, g)
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(q.shape, generator=gen, dtype=torch.float64)

        def loss(t):
            x = [q, k, v]
            x[i] = x[i] + t * u
            return float((attention64(*x, mask)["o"] * g).sum())

        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs(diff - float((r[name] * u).sum())) <= 1e-7 * (1 + abs(diff))
    assert (r["dk"][0, :, 2:5] == 0).all() and (r["dv"][0, :, 2:5] == 0).all()


def test_attention_formulas_of_an_empty_row():
    x = torch.ones(1, 1, 3, 128, dtype=torch.float64)
    r = attention64(x, x, x, torch.zeros(1, 3, dtype=torch.uint8), x)
    assert (r["lse"] == -math.inf).all()
    assert all((r[n] == 0).all() for n in ("o", "dq", "dk", "dv"))


def test_qk_formulas_against_autograd():
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(2, 3, 2, 128, generator=gen, dtype=torch.float64, requires_grad=True)
    gain = torch.randn(128, generator=gen, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(2, 3, 2, 128, generator=gen, dtype=torch.float64)
    a = torch.rand(1, 3, 1, 64, generator=gen, dtype=torch.float64) * 9
    z = x * torch.rsqrt(x.square().mean(3, keepdim=True) + 1e-6) * gain
    e, o = z[..., 0::2], z[..., 1::2]
    y = torch.stack([e * a.cos() - o * a.sin(), e * a.sin() + o * a.cos()], 4).flatten(3)
    (y * dy).sum().backward()
    dx, _, dgain, _ = qk_backward64(x.detach(), gain.detach(), a.cos(), a.sin(), dy, 1e-6)
    assert torch.allclose(dx, x.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(dgain, gain.grad, rtol=1e-10, atol=1e-12)


# ------------------------------------------------------------------------------------------ refusals
def _refused(lib, status, want, needle):
    assert status == want, (status, lib.mi_last_error())
    assert needle in lib.mi_last_error().decode(), lib.mi_last_error()


BWD = dict(qp=P, kp=P + MB, qkv=P + 2 * MB, key_mask=None, o=P + 6 * MB, lse=P + 7 * MB, d_o=P + 8 * MB, dqp=P + 9 * MB,
           dkp=P + 10 * MB, dqkv=P + 11 * MB, batch=1, seq=74, n_heads=2, ws=P + 15 * MB, ws_bytes=MB, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(qp=None), 1, "null"), (dict(lse=None), 1, "null"), (dict(dqkv=None), 1, "null"),
    (dict(o=P + 6 * MB + 8), 1, "aligned"), (dict(dkp=P + 10 * MB + 2), 1, "aligned"),
    (dict(batch=0), 1, "positive"), (dict(seq=-1), 1, "positive"), (dict(n_heads=0), 1, "positive"),
    (dict(seq=(1 << 20) + 1), 2, "2^20"), (dict(n_heads=1025), 2, "1024"), (dict(batch=2048, seq=1 << 18, n_heads=8), 2, "2^23"), (dict(batch=1 << 21, seq=1, n_heads=8), 2, "2^23"),
    (dict(batch=2147483647, seq=1 << 20, n_heads=1024), 2, "2^23"),
    (dict(ws=None), 3, "256-byte"), (dict(ws=P + 15 * MB + 16), 3, "256-byte"), (dict(ws_bytes=100), 3, "needed"),
    (dict(dqp=P), 1, "overlaps"), (dict(dkp=P + 9 * MB), 1, "overlaps"), (dict(dqkv=P + 2 * MB + 16), 1, "overlaps"),
    (dict(ws=P + 8 * MB), 1, "overlaps"), (dict(key_mask=P + 10 * MB), 1, "overlaps")])
def test_attention_backward_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_attention_backward(*{**BWD, **change}.values()), want, needle)


LSE = dict(qp=P, kp=P + MB, qkv=P + 2 * MB, key_mask=None, o=P + 6 * MB, lse=P + 7 * MB, batch=1, seq=74, n_heads=2, ws=None,
           ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(lse=None), 1, "null"), (dict(kp=None), 1, "null"), (dict(lse=P + 7 * MB + 4), 1, "aligned"), (dict(seq=0), 1, "positive"),
    (dict(seq=1 << 21), 2, "2^20"), (dict(o=P + 2 * MB), 1, "overlaps"), (dict(lse=P + 6 * MB), 1, "overlaps")])
def test_attention_lse_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_attention_lse(*{**LSE, **change}.values()), want, needle)


QK = dict(qkv=P, q_norm_w=P + 4 * MB, k_norm_w=P + 4 * MB + 1024, rope_cos=P + 5 * MB, rope_sin=P + 6 * MB, rope_bstride=0,
          dqp=P + 7 * MB, dkp=P + 8 * MB, dqkv=P + 9 * MB, dq_norm_w=P + 13 * MB, dk_norm_w=P + 13 * MB + 1024, batch=1, seq=74,
          n_heads=2, eps=1e-6, ws=P + 14 * MB, ws_bytes=MB, stream=None)


@pytest.mark.parametrize("change,want,needle", [
    (dict(dqkv=None), 1, "null"), (dict(rope_sin=None), 1, "null"), (dict(dq_norm_w=P + 13 * MB + 4), 1, "aligned"),
    (dict(seq=0), 1, "positive"), (dict(rope_bstride=-4), 1, "rope_bstride"), (dict(rope_bstride=6), 1, "rope_bstride"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=math.nan), 1, "eps"), (dict(n_heads=2000), 2, "1024")])
def test_qk_backward_refusals(lib, change, want, needle):
    _refused(lib, lib.mi_qk_norm_rope_backward(*{**QK, **change}.values()), want, needle)


def _axes(lib, pairs=(16, 24, 24), pos=P, rows=10, theta=10000.0, cos=P + MB, sin=P + 2 * MB):
    arr = (ctypes.c_int * len(pairs))(*pairs) if pairs else None
    return lib.mi_rope_axes_tables(pos, rows, len(pairs), arr, theta, cos, sin, None)


@pytest.mark.parametrize("change,needle", [
    (dict(pos=None), "null"), (dict(pairs=()), "null"), (dict(cos=P + 8), "aligned"), (dict(pos=P + 2), "aligned"),
    (dict(rows=0), "rows"), (dict(pairs=(16, 24, 23)), "64"), (dict(pairs=(40, 40)), "64"), (dict(pairs=(64, 0)), "64"),
    (dict(pairs=(-1, 65)), "64"), (dict(pairs=(7,) * 9), "n_axes"), (dict(theta=1.0), "theta"), (dict(theta=math.inf), "theta"),
    (dict(theta=math.nan), "theta")])
def test_rope_axes_refusals(lib, change, needle):
    _refused(lib, _axes(lib, **change), 1, needle)


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    assert lib.mi_attention_backward_workspace_size(2, 129, 3, ctypes.byref(n)) == 0
    assert n.value >= 2 * 2 * 3 * 256 * 4 and n.value % 256 == 0
    _refused(lib, lib.mi_attention_backward_workspace_size(0, 129, 3, ctypes.byref(n)), 1, "positive")
    _refused(lib, lib.mi_attention_backward_workspace_size(1, 1, 1, None), 1, "null")
    _refused(lib, lib.mi_qk_norm_rope_backward_workspace_size(1, 0, 1, ctypes.byref(n)), 1, "positive")


def test_binding_refuses_wrong_tensors():
    import diffusion_transformer_denoiser_gb300 as mi

    t = torch.empty(10, 64)
    with pytest.raises(ValueError, match="one column per axis"):
        mi.rope_axes_tables(torch.empty(10, 2), (16, 24, 24), t, t)
    with pytest.raises(ValueError, match="too few for 2 tables"):
        mi.qk_norm_rope_backward(t, t, t, t, t, t, t, t, t, t, 2, 5, 2, t, rope_bstride=640)
    for call in (lambda: mi.rope_axes_tables(torch.empty(10, 2), (32, 32), t, t),
                 lambda: mi.attention_lse(t, t, t, None, t, t, 1, 5, 2),
                 lambda: mi.attention_backward(t, t, t, None, t, t, t, t, t, t, 1, 5, 2, t),
                 lambda: mi.qk_norm_rope_backward(t, t, t, t, t, t, t, t, t, t, 1, 5, 2, t)):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    with pytest.raises(ValueError, match="lse has 640 elements, expected 641"):
        mi._sized(t, torch.float32, 641, "lse", -1)
    with pytest.raises(ValueError, match="o must live on the GPU of the other tensors, cuda:0"):
        mi._sized(t, torch.float32, 640, "o", 0)
    with pytest.raises(TypeError, match="o: expected torch.bfloat16"):
        mi._sized(t, torch.bfloat16, 640, "o", -1)
    with pytest.raises(ValueError, match="o must be contiguous"):
        mi._sized(t.T, torch.float32, 640, "o", -1)

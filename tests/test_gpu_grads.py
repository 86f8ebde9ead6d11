"""Gradient norm and clipping over many tensors."""
import math
import random

import pytest
import torch

from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
# The kernels add at most 64 squares in fp32 (each off by F) and the rest in 64 bits: the sum is off by 64 F of itself at
# most, its root by half of that, and the norm is rounded once.
NORM_TOL = (64 / 2 + 2) * F
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _tensors(sizes, kinds, std=0.02, seed=0, shift=0):
    """Tensors of the sizes, each `shift` elements into a buffer of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.empty(n + shift, device="cuda", dtype=KINDS[kinds[i % len(kinds)]])
        t.copy_(torch.randn(n + shift, generator=g, device="cuda") * std)
        out.append(t[shift:])
    return out


def _norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def _ws(mi, s):
    return torch.full((s.workspace_size(),), 255, dtype=torch.uint8, device="cuda")


def _factor(limit, norm):
    """The factor from the norm that was returned, in fp32 as documented."""
    q = torch.tensor(limit, dtype=torch.float32) / (norm.cpu() + torch.tensor(1e-6, dtype=torch.float32))
    return torch.where(q >= 1, torch.ones_like(q), q).cuda()


def _scaled(grads, c):
    return [(g.float() * c).to(g.dtype) for g in grads]


SIZES = [
    [1], [5], [31, 0, 33], [2048], [2049, 1, 7], [4096, 4095, 4097], [100003], [0], [1, 1, 1, 1], [3 * 256 * 256, 256, 128, 128],
    [8, 16, 24, 1000000, 3, 262144], list(range(70)), [1500 + 7 * i for i in range(150)],
]


@pytest.mark.parametrize("kinds", [["bf16"], ["f16"], ["f32"], ["bf16", "f32", "f16"]])
@pytest.mark.parametrize("shift", [0, 1, 4, 7])
def test_norm_and_clip(kinds, shift):
    mi = require_gpu()
    norm = torch.full((3,), 7.0, device="cuda")
    for sizes in SIZES:
        grads = _tensors(sizes, kinds, shift=shift)
        want = _norm64(grads)
        for out_shift in (None, shift, (shift + 3) % 8):
            outs = None if out_shift is None else [torch.full((n + 10,), 7.0, dtype=g.dtype, device="cuda")[out_shift:]
                                                   for n, g in zip(sizes, grads)]
            mine = [g.clone() if outs is None else g for g in grads]
            if outs is None and shift:
                mine = _tensors(sizes, kinds, shift=shift)
            s = mi.GradSet(mine, None if outs is None else [o[:n] for n, o in zip(sizes, outs)])
            s.clip_norm(want * 0.37 + 1e-3, norm[1:2], _ws(mi, s))
            assert abs(float(norm[1]) - want) <= NORM_TOL * want and norm[0] == 7 and norm[2] == 7
            c = _factor(want * 0.37 + 1e-3, norm[1:2])
            for n, got, ref in zip(sizes, mine if outs is None else outs, _scaled(grads, c)):
                assert torch.equal(got[:n], ref)
                assert outs is None or (got[n:] == 7).all()
            if outs is not None:
                assert all(torch.equal(a, b) for a, b in zip(mine, _tensors(sizes, kinds, shift=shift)))


@pytest.mark.parametrize("count", [999, 1000, 1001, 2300])
def test_many_tensors(count):
    rng = random.Random(count)
    mi = require_gpu()
    sizes = [rng.choice([0, 1, 2, 15, 63, 64, 65, 900, 5000]) for _ in range(count)]
    grads = _tensors([sum(sizes)], ["bf16"])[0].split(sizes)
    outs = [torch.empty_like(g) for g in grads]
    s = mi.GradSet(grads, outs)
    norm = torch.empty(1, device="cuda")
    s.norm(norm, _ws(mi, s))
    want = _norm64(grads)
    assert abs(float(norm) - want) <= NORM_TOL * want
    s.clip(0.5 * want, norm)
    assert all(torch.equal(a, b) for a, b in zip(outs, _scaled(grads, _factor(0.5 * want, norm))))


def test_in_place_below_the_limit_and_out_of_place():
    mi = require_gpu()
    grads = _tensors([1000, 77, 40000], ["bf16", "f32"])
    before = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    for s in (mi.GradSet(grads), mi.GradSet(grads, outs), mi.GradSet(grads, [grads[0], *outs[1:]])):
        s.clip_norm(1e6, norm, _ws(mi, s))
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert all(torch.equal(a, b) for a, b in zip(outs, before))


@pytest.mark.parametrize("value,kind", [(1e-30, "f32"), (3e-42, "f32"), (1e25, "f32"), (3e38, "bf16"), (2.0 ** -133, "bf16"),
                                        (6e-8, "f16"), (65504.0, "f16"), (0.0, "bf16")])
def test_squares_outside_of_32_bits(value, kind):
    mi = require_gpu()
    for n in (3, 5000):
        grads = [torch.full((n,), value, device="cuda", dtype=KINDS[kind]), torch.zeros(100, device="cuda", dtype=KINDS[kind])]
        s = mi.GradSet(grads)
        norm = torch.empty(1, device="cuda")
        s.norm(norm, _ws(mi, s))
        want = _norm64(grads)
        least = 2.0 ** -149
        if want > 3.5e38:
            assert norm.isinf()
        else:
            assert abs(float(norm) - want) <= NORM_TOL * want + least, (float(norm), want)


def test_small_beside_large():
    """Neither the many small ones nor the one large gradient is lost."""
    mi = require_gpu()
    grads = [torch.full((1 << 22,), 1e-3, device="cuda"), torch.tensor([2.0], device="cuda"), torch.full((64,), 1e-22, device="cuda")]
    s = mi.GradSet(grads)
    norm = torch.empty(1, device="cuda")
    s.norm(norm, _ws(mi, s))
    assert abs(float(norm) - _norm64(grads)) <= NORM_TOL * _norm64(grads)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_not_finite(kind):
    mi = require_gpu()
    norm = torch.empty(1, device="cuda")
    for bad in (math.inf, -math.inf, math.nan):
        grads = _tensors([5000, 300], [kind])
        grads[1][17] = bad
        outs = [torch.empty_like(g) for g in grads]
        s = mi.GradSet(grads, outs)
        s.clip_norm(1.0, norm, _ws(mi, s))
        if math.isnan(bad):
            assert norm.isnan() and all(o.isnan().all() for o in outs)
        else:
            assert norm.isinf() and outs[1][17].isnan() and (outs[0] == 0).all() and outs[1].isnan().sum() == 1


def test_norms_put_together():
    """Two sets clipped by the norm of both."""
    mi = require_gpu()
    a, b = _tensors([3000, 11], ["bf16"]), _tensors([70000], ["f32"], seed=1)
    sets, norms = [mi.GradSet(a), mi.GradSet(b)], torch.empty(2, device="cuda")
    before = [t.clone() for t in a + b]
    for i, s in enumerate(sets):
        s.norm(norms[i:i + 1], _ws(mi, s))
    norm = norms.norm().view(1)
    for s in sets:
        s.clip(1.5, norm)
    assert all(torch.equal(x, y) for x, y in zip(a + b, _scaled(before, _factor(1.5, norm))))


def test_captured_repeated_and_on_two_streams():
    mi = require_gpu()
    grads = _tensors([50000, 3, 4096, 129], ["bf16", "f32"])
    outs = [torch.empty_like(g) for g in grads]
    s, norm = mi.GradSet(grads, outs), torch.empty(1, device="cuda")
    ws = _ws(mi, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.clip_norm(0.5, norm, ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s.clip_norm(0.5, norm, ws)
    torch.cuda.current_stream().wait_stream(side)
    other = [torch.empty_like(g) for g in grads]
    t, norm2 = mi.GradSet(grads, other), torch.empty(1, device="cuda")
    ws2 = _ws(mi, t)
    for seed in (3, 4):
        for g, new in zip(grads, _tensors([50000, 3, 4096, 129], ["bf16", "f32"], seed=seed)):
            g.copy_(new)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        t.clip_norm(0.5, norm2, ws2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2) and abs(float(norm) - _norm64(grads)) <= NORM_TOL * _norm64(grads)
        ref = _scaled(grads, _factor(0.5, norm))
        assert all(torch.equal(a, r) and torch.equal(b, r) for a, b, r in zip(outs, other, ref))


def test_past_32_bits():
    mi = require_gpu()
    g = torch.zeros((1 << 32) + 5, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 2.0
    g[1 << 31] = 1.0
    s, norm = mi.GradSet([g]), torch.empty(1, device="cuda")
    s.clip_norm(1.0, norm, _ws(mi, s))
    assert abs(float(norm) - math.sqrt(13.0)) <= NORM_TOL * 4
    assert torch.equal(g[-3:], (torch.full((3,), 2.0, device="cuda") * _factor(1.0, norm)).bfloat16()) and g[:1 << 20].count_nonzero() == 0


def test_a_step_of_the_block():
    """Norm forward, a loss's gradient, the norms' gradients, and the clipping of all parameter gradients together."""
    mi = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    batch, seq, hidden = 2, 90, 512

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    x, mod, target = normal(batch * seq, hidden), normal(batch, 6, hidden, std=0.1), normal(batch * seq, hidden)
    weight, bias = normal(hidden, std=0.1) + 1, normal(hidden, std=0.1)
    h, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(batch * seq, device="cuda") for _ in range(2))
    mi.mod_rmsnorm(x, mod, 0, 1, h, batch, seq)
    mi.layer_norm(h, weight, bias, y, mean, rstd)
    dy = ((y.float() - target.float()) / y.numel()).bfloat16()
    dh, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db, dmod = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda"), torch.zeros(batch, 6, hidden, device="cuda")
    ws = torch.empty(max(mi.layer_norm_backward_workspace_size(batch * seq, hidden),
                         mi.mod_rmsnorm_backward_workspace_size(batch, seq, hidden)), dtype=torch.uint8, device="cuda")
    mi.layer_norm_backward(dy, h, weight, mean, rstd, dh, dw, db, ws)
    mi.mod_rmsnorm_backward(dh, x, mod, 0, 1, dx, dmod, batch, seq, ws)
    s, norm = mi.GradSet([dw, db, dmod, dx]), torch.empty(1, device="cuda")
    before = _norm64([dw, db, dmod, dx])
    s.clip_norm(1e-3, norm, _ws(mi, s))
    # the same by autograd in 64 bits
    leaves = [t.double().requires_grad_() for t in (weight, bias, mod, x)]
    w64, b64, mod64, x64 = leaves
    r = x64.view(batch, seq, hidden)
    r = r * (r.square().mean(2, keepdim=True) + 1e-6).rsqrt() * (1 + mod64[:, 1:2]) + mod64[:, 0:1]
    y64 = torch.nn.functional.layer_norm(r, (hidden,), w64, b64, 1e-6).view(-1, hidden)
    ((y64 - target.double()).square().sum() / 2 / y.numel()).backward()
    want = _norm64([t.grad for t in leaves])
    assert abs(float(norm) - before) <= NORM_TOL * before
    # h, dh and dx are rounded to bf16 on the way (2^-8 of each value)
    assert abs(float(norm) - want) <= 4 * 2.0 ** -8 * want
    for got, ref in zip((dw, db, dmod, dx), leaves):
        ref = ref.grad * min(1.0, 1e-3 / want)
        assert float((got.double() - ref).norm()) <= 6 * 2.0 ** -8 * float(ref.norm())


def test_refusals_on_the_gpu():
    mi = require_gpu()
    g = torch.zeros(100, device="cuda")
    s, norm = mi.GradSet([g]), torch.empty(1, device="cuda")
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.GradSet([g, g])
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.GradSet([g[:60], g[50:]])
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.GradSet([g[:50]], [g[1:51]])
    mi.GradSet([g[:50], g[:50]], [g[50:100], torch.empty(50, device="cuda")])  # read twice, written once each
    with pytest.raises(mi.MiError, match="overlaps"):
        s.clip_norm(1.0, g[3:4], _ws(mi, s))
    with pytest.raises(mi.MiError, match="workspace"):
        s.norm(norm, torch.empty(0, dtype=torch.uint8, device="cuda"))
    for bad in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(mi.MiError, match="max_norm"):
            s.clip(bad, norm)
    with pytest.raises(ValueError, match="contiguous"):
        mi.GradSet([torch.zeros(4, 4, device="cuda").T])
    with pytest.raises(TypeError, match="bfloat16, float16, float32"):
        mi.GradSet([torch.zeros(4, device="cuda", dtype=torch.float64)])
    with pytest.raises(ValueError, match="type and size"):
        mi.GradSet([g], [g.half()])
    empty = mi.GradSet([])
    norm.fill_(7.0)
    empty.clip_norm(1.0, norm, torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert norm == 0

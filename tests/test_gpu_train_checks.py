"""The training pass's outputs in the 2-norm, which a gradient that is wrong by 2 % does not pass, and calls
that the element-wise tests leave out: long masks, long gradients, captured masked calls, other streams."""
import pytest
import torch

from tests._gpu import require_gpu
from tests._train import HEAD, attention64, heads_of, within
from tests._train_norms import agrees_with_difference, close_in_norm, directions, head64
from tests.test_gpu_train import BF, Case, _gen, _normal

pytestmark = pytest.mark.gpu


def _check_heads(c, heads, what=("o", "dq", "dk", "dv")):
    """Some heads of every element of a case against 64 bits."""
    b, s, h = c.dims
    o, v, g, dv = (heads_of(t, b, s, h) for t in (c.o, c.v, c.d_o, c.dv))
    for e in range(b):
        keys = torch.arange(s, device="cuda") if c.mask is None else c.mask[e].nonzero().flatten()
        for i in heads:
            r = head64(c.q[e, i].double(), c.k[e, i].double(), v[e, i], keys, g[e, i] if "dq" in what else None)
            got = {"o": o[e, i], "dq": c.dq[e, i], "dk": c.dk[e, i], "dv": dv[e, i]}
            within(c.lse[e, i], r["lse"], r["lse_tol"], "lse")
            for name in what:
                close_in_norm(got[name], r[name], f"{name} of element {e}, head {i}")
                if name in ("dk", "dv"):
                    off = torch.ones(s, dtype=torch.bool, device="cuda")
                    off[keys] = False
                    assert (got[name][off] == 0).all()


@pytest.mark.parametrize("batch,heads,seq,mask,split", [
    (1, 2, 74, None, True), (2, 2, 384, "pad", True), (2, 3, 257, "front", False), (1, 4, 1219, "pad", True),
    (2, 40, 650, "pad", True), (1, 3, 5003, "pad", True), (1, 24, 4130, None, True)])
def test_outputs_in_norm(batch, heads, seq, mask, split):
    mi = require_gpu()
    c = Case(batch, heads, seq, mask)
    c.forward(mi, split)
    c.backward(mi)
    torch.cuda.synchronize()
    assert mi.device_error() == 0
    _check_heads(c, sorted({0, heads // 2, heads - 1}))


@pytest.mark.parametrize("mask", [None, "pad"])
def test_gradients_along_directions(mask):
    """Slopes of the kernel's gradients against central differences of the 64-bit forward, along the gradient and
    along directions with a good part of it."""
    mi = require_gpu()
    c = Case(2, 2, 150, mask)
    b, s, h = c.dims
    c.forward(mi)
    c.backward(mi)
    torch.cuda.synchronize()
    r = c.ref()
    x = [c.q.double(), c.k.double(), heads_of(c.v, b, s, h)]
    g = heads_of(c.d_o, b, s, h)
    got = [c.dq, c.dk, heads_of(c.dv, b, s, h)]
    for i, name in enumerate(("dq", "dk", "dv")):
        def loss(t, u):
            y = list(x)
            y[i] = x[i] + t * u
            return float((attention64(*y, c.mask)["o"] * g).sum())

        for u in directions(r[name], _gen(6)):
            diff = (loss(1e-4, u) - loss(-1e-4, u)) / 2e-4
            agrees_with_difference(got[i], u, diff, float(r[name].norm()), name)


@pytest.mark.parametrize("split", [False, True])
def test_masks_of_more_than_65536_keys(split):
    """Longer than the forward's mask in shared memory: whole tiles masked, single keys, and the end."""
    mi = require_gpu()
    seq = 66001
    c = Case(1, 1, seq, None)
    c.mask = torch.ones(1, seq, dtype=torch.uint8, device="cuda")
    c.mask[:, 1000:3000] = 0
    c.mask[:, 40001:60000:3] = 0
    c.mask[:, 65900:] = 0
    c.forward(mi, split)
    if split:
        c.backward(mi)
    torch.cuda.synchronize()
    assert mi.device_error() == 0
    _check_heads(c, [0], ("o", "dq", "dk", "dv") if split else ("o",))


@pytest.mark.parametrize("batch,heads,seq", [(2, 40, 650), (1, 2, 333)])
def test_masked_forward_captured_and_replayed(batch, heads, seq):
    """One graph of the masked forward, on the split schedule where there is one, and the gradient: replayed with
    another mask and other inputs it gives the bytes of plain calls."""
    mi = require_gpu()
    a, b = Case(batch, heads, seq, "pad", seed=1), Case(batch, heads, seq, "empty" if batch > 1 else "front", seed=2)
    fws = torch.empty(mi.attention_workspace_size(batch, seq, heads), dtype=torch.uint8, device="cuda")
    bws = torch.empty(mi.attention_backward_workspace_size(batch, seq, heads), dtype=torch.uint8, device="cuda")

    def both():
        mi.attention_lse(a.q, a.k, a.qkv, a.mask, a.o, a.lse, batch, seq, heads, ws=fws)
        a.backward(mi, bws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        both()
    for name in ("q", "k", "qkv", "d_o", "mask"):
        getattr(a, name).copy_(getattr(b, name))
    for _ in range(2):
        graph.replay()
    b.forward(mi)
    b.backward(mi)
    torch.cuda.synchronize()
    assert mi.device_error() == 0
    assert torch.equal(a.lse, b.lse) and torch.equal(a.o, b.o)
    assert all(torch.equal(x, y) for x, y in zip(a.bits(), b.bits()))


class QkCase:
    def __init__(self, batch, heads, seq, seed):
        g = _gen(seed)
        self.dims = (batch, seq, heads)
        self.qkv = _normal(g, batch * seq, 3 * heads * HEAD)
        self.gains = [_normal(g, HEAD, std=0.3, mean=1.0) for _ in range(2)]
        self.dy = [_normal(g, batch, heads, seq, HEAD) for _ in range(2)]
        angle = torch.rand(seq, 64, generator=g, device="cuda") * 50
        self.tables = [angle.cos(), angle.sin()]
        self.dqkv = torch.full_like(self.qkv, 7.0)
        self.dg = [torch.full((HEAD,), 7.0, device="cuda") for _ in range(2)]

    def args(self, mi):
        b, s, h = self.dims
        ws = torch.empty(mi.qk_norm_rope_backward_workspace_size(b, s, h), dtype=torch.uint8, device="cuda")
        return dict(qkv=self.qkv, q_norm_w=self.gains[0], k_norm_w=self.gains[1], rope_cos=self.tables[0], rope_sin=self.tables[1],
                    dqp=self.dy[0], dkp=self.dy[1], dqkv=self.dqkv, dq_norm_w=self.dg[0], dk_norm_w=self.dg[1], batch=b, seq=s,
                    n_heads=h, ws=ws)

    def outputs(self):
        return [self.dqkv.clone()] + [t.clone() for t in self.dg]


@pytest.mark.parametrize("batch,heads,seq", [(1, 2, 30), (2, 6, 1100)])
def test_qk_gradient_on_two_streams(batch, heads, seq):
    """Two calls at once, a workspace each: the bytes of calls in turn (one cluster, and the whole GPU)."""
    mi = require_gpu()
    cases = [QkCase(batch, heads, seq, seed) for seed in (21, 22)]
    args = [c.args(mi) for c in cases]
    expected = []
    for c, a in zip(cases, args):
        mi.qk_norm_rope_backward(**a)
        expected.append(c.outputs())
        c.dqkv.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for a, s in zip(args, streams):
            mi.qk_norm_rope_backward(**a, stream=s)
    torch.cuda.synchronize()
    for c, e in zip(cases, expected):
        assert all(torch.equal(x, y) for x, y in zip(c.outputs(), e))


def test_qk_gradient_refuses_overlaps():
    mi = require_gpu()
    c = QkCase(1, 2, 74, 23)
    a = c.args(mi)
    before = c.outputs()
    raw = c.qkv.view(torch.uint8).flatten()
    for change in (dict(dqkv=c.qkv), dict(dq_norm_w=c.dg[1]), dict(dk_norm_w=c.tables[0].flatten()[64:192]),
                   dict(dqp=c.dqkv.flatten()[:c.dy[0].numel()]), dict(ws=raw[:raw.numel() // 256 * 256])):
        with pytest.raises(mi.MiError, match="overlaps"):
            mi.qk_norm_rope_backward(**{**a, **change})
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, c.outputs()))  # nothing was enqueued

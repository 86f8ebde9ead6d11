"""The training pass's outputs in the 2-norm, which a gradient that is wrong by 2 % does not pass, and calls
that the element-wise tests leave out: long masks, long gradients, captured masked calls, other streams."""
import math

import pytest
import torch

from tests._gpu import require_gpu
from tests._train import HEAD, U, attention64, heads_of, within
from tests._train_norms import agrees_with_difference, close_in_norm, directions, head64, norm_error
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


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(BF).min])
@pytest.mark.parametrize("batch,heads,seq", [(2, 2, 30), (2, 3, 300), (2, 40, 650)])
def test_padding_may_hold_anything_in_the_whole_pass(bad, batch, heads, seq):
    """The k and v columns of padded rows, and every column of an element without a valid key: what they hold
    reaches no output of the four calls.  The bytes are those of zeros in their place, which are held against
    64-bit autograd of the whole function, the q, k and v columns each by itself."""
    mi = require_gpu()
    gen = _gen(heads * seq)
    rows, width = batch * seq, heads * HEAD
    mask = torch.ones(batch, seq, dtype=torch.uint8, device="cuda")
    mask[0] = 0
    mask[-1, seq // 5:seq // 2] = 0
    off = (mask == 0).view(-1, 1)
    columns = torch.arange(3 * width, device="cuda")
    padding = (off & (columns >= width)) | (off & (torch.arange(rows, device="cuda") < seq).view(-1, 1))
    clean = _normal(gen, rows, 3 * width).masked_fill_(padding, 0.0)
    gains = [_normal(gen, HEAD, std=0.1, mean=1.2) for _ in range(2)]
    d_o = _normal(gen, rows, width)
    angle = torch.rand(seq, 64, generator=gen, device="cuda") * 50
    cos, sin = angle.cos(), angle.sin()

    def whole_pass(qkv):
        qp, kp = (torch.empty(batch, heads, seq, HEAD, dtype=BF, device="cuda") for _ in range(2))
        o, lse = torch.empty(rows, width, dtype=BF, device="cuda"), torch.empty(batch, heads, seq, device="cuda")
        mi.qk_norm_rope(qkv, *gains, cos, sin, qp, kp, batch, seq, heads)
        ws = torch.empty(mi.attention_workspace_size(batch, seq, heads), dtype=torch.uint8, device="cuda")
        mi.attention_lse(qp, kp, qkv, mask, o, lse, batch, seq, heads, ws=ws)
        dqp, dkp, dqkv = torch.empty_like(qp), torch.empty_like(kp), torch.empty_like(qkv)
        ws = torch.empty(max(mi.attention_backward_workspace_size(batch, seq, heads),
                             mi.qk_norm_rope_backward_workspace_size(batch, seq, heads)), dtype=torch.uint8, device="cuda")
        mi.attention_backward(qp, kp, qkv, mask, o, lse, d_o, dqp, dkp, dqkv, batch, seq, heads, ws)
        dg = [torch.empty(HEAD, device="cuda") for _ in range(2)]
        mi.qk_norm_rope_backward(qkv, *gains, cos, sin, dqp, dkp, dqkv, *dg, batch, seq, heads, ws)
        torch.cuda.synchronize()
        assert mi.device_error() == 0
        return {"o": o, "lse": lse, "dqkv": dqkv, "dgq": dg[0], "dgk": dg[1]}

    want, got = whole_pass(clean), whole_pass(clean.masked_fill(padding, bad))
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert (got["dqkv"][padding] == 0).all()

    x = clean.double().requires_grad_()
    g64 = [g.double().requires_grad_() for g in gains]
    parts = x.view(batch, seq, 3, heads, HEAD).permute(2, 0, 3, 1, 4)
    c64, s64 = cos.double(), sin.double()

    def turn(t, gain):
        t = t * torch.rsqrt(t.square().mean(3, keepdim=True) + 1e-6) * gain
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack([a * c64 - b * s64, a * s64 + b * c64], 4).flatten(3)

    # (element 0 has no output: the sum is over element 1)
    z = turn(parts[0], g64[0])[1] @ turn(parts[1], g64[1])[1].transpose(1, 2) / math.sqrt(HEAD)
    z = z.masked_fill((mask[1] == 0)[None, None, :], -math.inf)
    out = (torch.softmax(z, 2) @ parts[2][1]).permute(1, 0, 2).reshape(seq, width)
    (out * d_o[seq:].double()).sum().backward()
    # Roundings on the way to a gradient: q and k (which move the scores, of variance 1.2^4, and enter the last
    # product), P or dS, o, the gradient of q or k, and of qkv: six of U / sqrt(5) in the mean square, times 1.44
    # at most, in quadrature 1.6 U; never more than 4 U.
    for i, name in enumerate(("q", "k", "v")):
        cols = slice(i * width, (i + 1) * width)
        err = norm_error(got["dqkv"][:, cols], x.grad[:, cols])
        assert err <= 4 * U, f"d{name}: {err:.3g}"
    for i, name in enumerate(("dgq", "dgk")):
        err = norm_error(got[name], g64[i].grad)
        assert err <= 4 * U, f"{name}: {err:.3g}"


@pytest.mark.parametrize("batch,heads,seq", [(1, 2, 30), (2, 6, 1100)])
def test_rows_without_a_gradient_add_nothing(batch, heads, seq):
    """A head whose dq or dk is zero in a row gives a zero gradient and adds nothing to the gains', whatever x
    holds, with eps 0 too; the other head of the row, and q where k has none, stay as they are."""
    mi = require_gpu()
    c = QkCase(batch, heads, seq, 31)
    for i, bad in enumerate((math.nan, math.inf, -math.inf, 0.0, 3e38)):
        for which in (0, 1):
            c.dy[which][-1, -1, 3 * i + which] = -0.0 if i % 2 else 0.0
            c.qkv.view(batch, seq, 3, heads, HEAD)[-1, 3 * i + which, which, -1] = bad
    for eps in (1e-6, 0.0):
        a = c.args(mi)
        mi.qk_norm_rope_backward(**a, eps=eps)
        got = c.outputs()
        clean = QkCase(batch, heads, seq, 31)
        clean.dy = c.dy
        mi.qk_norm_rope_backward(**clean.args(mi), eps=eps)
        want = clean.outputs()
        assert all(t.isfinite().all() for t in got)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        dx = got[0].view(batch, seq, 3, heads, HEAD)
        for i in range(5):
            for which in (0, 1):
                assert (dx[-1, 3 * i + which, which, -1] == 0).all()
                assert (dx[-1, 3 * i + which, 1 - which, -1] != 0).any()


@pytest.mark.parametrize("batch,heads,seq,mask", [(1, 2, 300, None), (1, 2, 300, "pad"), (2, 40, 650, "pad"), (2, 40, 650, None)])
def test_log_sum_exp_of_a_row_that_is_not_a_number(batch, heads, seq, mask):
    """-inf says that a row has no valid key; a query of NaN, or with an infinity (whose scores are infinities of
    either sign), has a log-sum-exp of NaN."""
    mi = require_gpu()
    c, d = Case(batch, heads, seq, mask), Case(batch, heads, seq, mask)
    at = [0, 77, 130, seq - 1]
    c.q[:, :, at[:2]] = math.nan
    c.q[:, :, at[2:], 5] = math.inf
    c.forward(mi), d.forward(mi)
    torch.cuda.synchronize()
    assert mi.device_error() == 0
    assert c.lse[:, :, at].isnan().all()
    o, rest = heads_of(c.o, batch, seq, heads), [i for i in range(seq) if i not in at]
    assert o[:, :, at].isnan().all()
    assert torch.equal(c.lse[:, :, rest], d.lse[:, :, rest])
    assert torch.equal(o[:, :, rest], heads_of(d.o, batch, seq, heads)[:, :, rest])


@pytest.mark.parametrize("name", ["qp", "kp", "qkv", "key_mask", "o", "lse"])
def test_forward_refuses_a_workspace_that_overlaps(name):
    """On the split schedule the kernels write the workspace.  A tensor that begins in its last bytes is refused
    before anything is enqueued, one right behind it is not; a workspace that no schedule uses may be anywhere."""
    mi = require_gpu()
    for batch, heads, seq in ((2, 40, 650), (1, 2, 300)):
        c = Case(batch, heads, seq, "pad")
        need = mi.attention_workspace_size(batch, seq, heads)
        assert (need > 0) == (batch == 2)
        c.forward(mi)
        want = [c.o.clone(), c.lse.clone()]
        call = dict(qp=c.q, kp=c.k, qkv=c.qkv, key_mask=c.mask, o=c.o, lse=c.lse, batch=batch, seq=seq, n_heads=heads)
        t = call[name]
        size = t.numel() * t.element_size()
        room = torch.zeros(need + size, dtype=torch.uint8, device="cuda")
        if need > 0:
            with pytest.raises(mi.MiError, match="overlaps"):
                mi.attention_lse(**{**call, name: room[need - 256:][:size].view(t.dtype).view(t.shape)}, ws=room[:need])
            torch.cuda.synchronize()
            assert (room == 0).all()
        call[name] = room[need:].view(t.dtype).view(t.shape).copy_(t)
        mi.attention_lse(**call, ws=room[:need] if need > 0 else room[:256])
        torch.cuda.synchronize()
        assert mi.device_error() == 0
        assert torch.equal(call["o"], want[0]) and torch.equal(call["lse"], want[1])


def test_the_longest_lists_of_key_tiles():
    """As many elements as the split schedule takes (8 query-tile pairs per SM), two key tiles each; and one more,
    where every unit has its CTA."""
    mi = require_gpu()
    most = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    for batch in (most, most + 1):
        assert (mi.attention_workspace_size(batch, 251, 1) > 0) == (batch == most)
        c = Case(batch, 1, 251, None)
        c.mask = (torch.rand(batch, 251, generator=_gen(3), device="cuda") < 0.7).to(torch.uint8)
        c.mask[::3, :128] = 0
        c.mask[1::3, 120:] = 0
        c.mask[::7] = 0
        c.forward(mi)
        c.check(mi, grads=False)

"""The attention section's training pass against 64-bit forms: rotary tables with several axes, the
attention that keeps its log-sum-exp, its gradient, and the gradient of the q/k norm and rotation."""
import math

import pytest
import torch

from tests._gpu import require_gpu
from tests._train import F, HEAD, U, attention64, heads_of, qk_backward64, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(BF)


def _mask(kind, batch, seq):
    if kind is None:
        return None
    m = torch.ones(batch, seq, dtype=torch.uint8, device="cuda")
    if kind == "pad":          # padded rows inside the last element
        m[-1, seq // 5: seq // 5 + seq // 3] = 0
    elif kind == "empty":      # the first element has no valid key
        m[0] = 0
        m[-1, ::3] = 0
    elif kind == "one":        # one valid key
        m[:] = 0
        m[:, seq // 2] = 1
    elif kind == "front":      # the first tiles hold no valid key
        m[:, : (2 * seq) // 3] = 0
    return m


class Case:
    def __init__(self, batch, heads, seq, mask=None, q_std=1.0, seed=0):
        g = _gen(seed + 1000 * seq + 10 * heads + batch)
        self.dims = (batch, seq, heads)
        rows, width = batch * seq, heads * HEAD
        self.q, self.k = _normal(g, batch, heads, seq, HEAD, std=q_std), _normal(g, batch, heads, seq, HEAD)
        self.qkv = _normal(g, rows, 3 * width)
        self.d_o = _normal(g, rows, width)
        self.mask = _mask(mask, batch, seq)
        self.o = torch.full((rows, width), 7.0, dtype=BF, device="cuda")
        self.lse = torch.full((batch, heads, seq), 7.0, device="cuda")
        self.dq, self.dk = torch.full_like(self.q, 7.0), torch.full_like(self.k, 7.0)
        self.dqkv = torch.full_like(self.qkv, 7.0)

    @property
    def v(self):
        return self.qkv[:, 2 * self.dims[2] * HEAD:]

    @property
    def dv(self):
        return self.dqkv[:, 2 * self.dims[2] * HEAD:]

    def forward(self, mi, split=True):
        b, s, h = self.dims
        ws = torch.empty(mi.attention_workspace_size(b, s, h), dtype=torch.uint8, device="cuda") if split else None
        mi.attention_lse(self.q, self.k, self.qkv, self.mask, self.o, self.lse, b, s, h, ws=ws)

    def backward(self, mi, ws=None, stream=None):
        b, s, h = self.dims
        if ws is None:
            ws = torch.full((mi.attention_backward_workspace_size(b, s, h),), 255, dtype=torch.uint8, device="cuda")
        mi.attention_backward(self.q, self.k, self.qkv, self.mask, self.o, self.lse, self.d_o, self.dq, self.dk,
                              self.dqkv, b, s, h, ws, stream=stream)

    def ref(self, grads=True):
        b, s, h = self.dims
        return attention64(self.q.double(), self.k.double(), heads_of(self.v, b, s, h), self.mask,
                           heads_of(self.d_o, b, s, h) if grads else None)

    def check(self, mi, grads=True):
        torch.cuda.synchronize()
        assert mi.device_error() == 0
        b, s, h = self.dims
        r = self.ref(grads)
        within(self.lse, r["lse"], r["lse_tol"], "lse")
        within(heads_of(self.o, b, s, h), r["o"], r["o_tol"], "o")
        if grads:
            within(self.dq, r["dq"], r["dq_tol"], "dq")
            within(self.dk, r["dk"], r["dk_tol"], "dk")
            within(heads_of(self.dv, b, s, h), r["dv"], r["dv_tol"], "dv")
            assert (self.dqkv[:, : 2 * h * HEAD] == 7.0).all()  # the q and k columns are another call's

    def bits(self):
        return [t.view(torch.int16).clone() for t in (self.dq, self.dk, self.dqkv)]


SHAPES = [(1, 1, 1, None), (1, 2, 2, None), (2, 1, 31, "one"), (1, 2, 74, None), (1, 3, 127, "pad"), (2, 2, 128, None),
          (1, 2, 129, "pad"), (2, 4, 210, "pad"), (3, 2, 255, "empty"), (2, 3, 257, "front"), (1, 1, 384, "one"),
          (2, 5, 640, "empty"), (1, 4, 1219, "pad")]


@pytest.mark.parametrize("batch,heads,seq,mask", SHAPES)
@pytest.mark.parametrize("split", [False, True])
def test_forward_parity(batch, heads, seq, mask, split):
    mi = require_gpu()
    c = Case(batch, heads, seq, mask)
    c.forward(mi, split)
    c.check(mi, grads=False)


@pytest.mark.parametrize("batch,heads,seq,mask", SHAPES)
def test_backward_parity(batch, heads, seq, mask):
    mi = require_gpu()
    c = Case(batch, heads, seq, mask)
    c.forward(mi)
    c.backward(mi)
    c.check(mi)


@pytest.mark.parametrize("q_std", [0.0, 6.0])
def test_backward_flat_and_peaked_scores(q_std):
    mi = require_gpu()
    c = Case(1, 2, 333, "pad", q_std=q_std)
    c.forward(mi)
    c.backward(mi)
    c.check(mi)


def test_split_forward_with_many_units():
    """More query-tile pairs than SMs: units cut between neighbours, masks whose parts have no valid key."""
    mi = require_gpu()
    for mask in ("front", "empty"):
        c = Case(2, 40, 650, mask)
        assert mi.attention_workspace_size(2, 650, 40) > 0
        c.forward(mi)
        c.check(mi, grads=False)


@pytest.mark.parametrize("batch,heads,seq,valid", [
    (2, 36, 4096, [(0, 4096), (4000, 4001)]),   # one element of 32 key tiles, one of a single tile
    (1050, 1, 130, None),                       # more elements than are listed in shared memory
    (600, 1, 130, None),
    (5, 33, 513, [(0, 0), (0, 513), (512, 513), (0, 0), (128, 256)]),  # empty ones between, a last tile of one key
    (2, 3, 1500, [(300, 301), (1499, 1500)])])  # one CTA per unit, the only tile in the middle or last
def test_split_forward_with_uneven_padding(batch, heads, seq, valid):
    """Elements with very different numbers of key tiles: every way the work is dealt out."""
    mi = require_gpu()
    c = Case(batch, heads, seq, None)
    c.mask = torch.zeros(batch, seq, dtype=torch.uint8, device="cuda")
    for b in range(batch):
        lo, hi = valid[b] if valid else ((b * 7) % seq, seq) if b % 3 else (0, 0)
        c.mask[b, lo:hi] = 1
    if c.q.numel() * seq > 1 << 34:  # the 64-bit check takes some heads of the large case
        c.forward(mi)
        torch.cuda.synchronize()
        assert mi.device_error() == 0
        for h in (0, heads - 1):
            cols = slice(h * HEAD, (h + 1) * HEAD)
            r = attention64(c.q[:, h:h + 1].double(), c.k[:, h:h + 1].double(), heads_of(c.v[:, cols], batch, seq, 1), c.mask)
            within(c.lse[:, h:h + 1], r["lse"], r["lse_tol"], "lse")
            within(heads_of(c.o[:, cols], batch, seq, 1), r["o"], r["o_tol"], "o")
        return
    c.forward(mi)
    c.backward(mi)
    c.check(mi)


@pytest.mark.parametrize("split", [False, True])
def test_forward_equals_the_inference_call(split):
    mi = require_gpu()
    b, h, s = 2, 40, 650
    c = Case(b, h, s, "pad")
    c.forward(mi, split)
    o = torch.empty_like(c.o)
    ws = torch.empty(mi.attention_workspace_size(b, s, h), dtype=torch.uint8, device="cuda") if split else None
    mi.attention(c.q, c.k, c.qkv, c.mask, o, b, s, h, ws=ws)
    assert torch.equal(o.view(torch.int16), c.o.view(torch.int16))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(BF).min])
def test_masked_keys_may_hold_anything(bad):
    mi = require_gpu()
    c = Case(2, 2, 300, "pad")
    b, s, h = c.dims
    off = c.mask == 0
    c.k.masked_fill_(off[:, None, :, None], bad)
    c.v.masked_fill_(off.view(-1, 1), bad)
    c.forward(mi)
    c.backward(mi)
    c.check(mi)
    assert (c.dk.permute(0, 2, 1, 3)[off] == 0).all()
    assert (heads_of(c.dv, b, s, h).permute(0, 2, 1, 3)[off] == 0).all()


def test_backward_against_differences():
    """The gradient along random directions against central differences of the 64-bit forward."""
    mi = require_gpu()
    c = Case(2, 2, 150, "pad")
    b, s, h = c.dims
    c.forward(mi)
    c.backward(mi)
    r = c.ref()
    x = [c.q.double(), c.k.double(), heads_of(c.v, b, s, h)]
    g = heads_of(c.d_o, b, s, h)
    got = [c.dq.double(), c.dk.double(), heads_of(c.dv, b, s, h)]
    gen = _gen(5)
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        step = 1e-5

        def loss(t):
            y = list(x)
            y[i] = x[i] + t * u
            return float((attention64(*y, c.mask)["o"] * g).sum())

        diff = (loss(step) - loss(-step)) / (2 * step)
        along = float((got[i] * u).sum())
        # the kernel's own bound along u; the difference itself is off by about step^2 and 1e-16 / step
        assert abs(along - diff) <= float((r[name + "_tol"] * u.abs()).sum()) + 1e-5 * abs(diff) + 1e-5


def test_backward_repeats_and_ignores_its_workspace():
    mi = require_gpu()
    c = Case(2, 6, 700, "empty")
    c.forward(mi)
    n = mi.attention_backward_workspace_size(2, 700, 6)
    c.backward(mi, torch.zeros(n, dtype=torch.uint8, device="cuda"))
    first = c.bits()
    for fill in (255, 127):
        c.dq.fill_(3.0), c.dk.fill_(3.0), c.dv.fill_(3.0)
        c.backward(mi, torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(first, c.bits()))


def test_outputs_end_where_they_should():
    """Rows behind the last sequence stay as they were."""
    mi = require_gpu()
    c = Case(2, 3, 301, "pad")
    b, s, h = c.dims
    rows, n = b * s, b * h * s

    def guarded(like, extra):
        buf = torch.full((like.numel() + extra,), 9.0, dtype=like.dtype, device="cuda")
        return buf, buf[: like.numel()].view(like.shape)

    bufs = []
    for name in ("o", "lse", "dq", "dk", "dqkv"):
        buf, view = guarded(getattr(c, name), 256 * 512)
        bufs.append((buf, view.numel()))
        setattr(c, name, view)
    c.dqkv.fill_(7.0)
    c.forward(mi)
    c.backward(mi)
    c.check(mi)
    for buf, used in bufs:
        assert (buf[used:] == 9.0).all()


def test_outputs_aligned_to_16_bytes_only():
    """Tensors that start 16 bytes behind a larger boundary give the bytes of those that do not."""
    mi = require_gpu()
    c, d = Case(1, 3, 333, "pad"), Case(1, 3, 333, "pad")
    for name in ("q", "k", "qkv", "d_o", "o", "lse", "dq", "dk", "dqkv"):
        t = getattr(d, name)
        step = 16 // t.element_size()
        buf = torch.empty(t.numel() + step, dtype=t.dtype, device="cuda")
        view = buf[step:].view(t.shape)
        assert view.data_ptr() % 32 == 16
        setattr(d, name, view.copy_(t))
    for x in (c, d):
        x.forward(mi)
        x.backward(mi)
    d.check(mi)
    assert all(torch.equal(x, y) for x, y in zip(c.bits(), d.bits()))


def test_captured_and_replayed():
    """One graph of forward and gradient, replayed on other inputs, gives the bytes of plain calls."""
    mi = require_gpu()
    a, b = Case(2, 3, 421, "pad", seed=1), Case(2, 3, 421, "pad", seed=2)
    ws = torch.empty(mi.attention_backward_workspace_size(2, 421, 3), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a.forward(mi, split=False)
        a.backward(mi, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        a.forward(mi, split=False)
        a.backward(mi, ws)
    for name in ("q", "k", "qkv", "d_o"):
        getattr(a, name).copy_(getattr(b, name))
    graph.replay()
    b.forward(mi, split=False)
    b.backward(mi)
    torch.cuda.synchronize()
    assert torch.equal(a.lse, b.lse)
    assert all(torch.equal(x, y) for x, y in zip(a.bits(), b.bits()))


def test_two_streams_at_once():
    mi = require_gpu()
    cases = [Case(1, 5, 900, "pad", seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    sizes = mi.attention_backward_workspace_size(1, 900, 5)
    spaces = [torch.empty(sizes, dtype=torch.uint8, device="cuda") for _ in cases]
    for c in cases:
        c.forward(mi)
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, w in zip(cases, streams, spaces):
            c.backward(mi, w, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check(mi)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last heads of the last element against 64 bits."""
    mi = require_gpu()
    batch, heads, seq = 66, 66, 4000
    assert batch * heads * seq * HEAD > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB for the inputs and their draws")
    c = Case(batch, heads, seq, None)
    c.mask = torch.zeros(batch, seq, dtype=torch.uint8, device="cuda")
    c.mask[:, 3900:] = 1
    c.forward(mi, split=False)
    c.backward(mi)
    torch.cuda.synchronize()
    assert mi.device_error() == 0
    b, cols = batch - 1, slice((heads - 1) * HEAD, heads * HEAD)
    at = slice(b * seq, batch * seq)
    one = lambda t: t[at, cols].double().view(1, 1, seq, HEAD)  # noqa: E731
    r = attention64(c.q[b:, heads - 1:].double(), c.k[b:, heads - 1:].double(), one(c.v), c.mask[b:], one(c.d_o))
    within(c.lse[b:, heads - 1:], r["lse"], r["lse_tol"], "lse")
    within(one(c.o), r["o"], r["o_tol"], "o")
    within(c.dq[b:, heads - 1:], r["dq"], r["dq_tol"], "dq")
    within(c.dk[b:, heads - 1:], r["dk"], r["dk_tol"], "dk")
    within(one(c.dv), r["dv"], r["dv_tol"], "dv")


def test_binding_refuses_wrong_tensors_on_the_gpu():
    mi = require_gpu()
    c = Case(1, 2, 130, None)
    c.forward(mi)
    before = c.bits()
    b, s, h = c.dims
    ws = torch.empty(mi.attention_backward_workspace_size(b, s, h), dtype=torch.uint8, device="cuda")
    args = dict(qp=c.q, kp=c.k, qkv=c.qkv, key_mask=None, o=c.o, lse=c.lse, d_o=c.d_o, dqp=c.dq, dkp=c.dk, dqkv=c.dqkv,
                batch=b, seq=s, n_heads=h, ws=ws)
    for change, error in ((dict(kp=c.k[:, :, 1:]), ValueError), (dict(lse=c.lse.double()), TypeError),
                          (dict(d_o=c.d_o.float()), TypeError), (dict(dqp=c.dq.cpu()), ValueError),
                          (dict(key_mask=torch.ones(b, s + 1, dtype=torch.uint8, device="cuda")), ValueError),
                          (dict(qkv=c.qkv.T.contiguous().T), ValueError), (dict(ws=ws[:256]), mi.MiError),
                          (dict(dkp=c.dq), mi.MiError), (dict(dqp=c.q), mi.MiError)):
        with pytest.raises(error):
            mi.attention_backward(**{**args, **change})
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, c.bits()))  # nothing was enqueued
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.attention_lse(c.q, c.k, c.qkv, None, c.q.view(c.o.shape), c.lse, b, s, h)


def test_many_elements_of_one_row():
    """Batches of single rows: one unit each, most of a tile empty; the softmax of one key is 1."""
    mi = require_gpu()
    c = Case(700, 3, 1, None)
    c.mask = torch.ones(700, 1, dtype=torch.uint8, device="cuda")
    c.mask[::5] = 0
    c.forward(mi)
    c.backward(mi)
    c.check(mi)


# ------------------------------------------------------------------------------------ rotary tables
@pytest.mark.parametrize("rows,pairs,far,scale", [
    (1, (64,), 0.0, 1.0), (16, (32, 32), 0.0, 1.0), (333, (16, 24, 24), 0.0, 0.37), (1000, (1, 62, 1), 1e4, 1.0),
    (4097, (20, 22, 22), -1e5, 1.0), (77, (8,) * 8, 2.0 ** 24 - 80, 1.0), (50000, (10, 27, 27), 3.0, 1.7)])
def test_rope_axes(rows, pairs, far, scale):
    mi = require_gpu()
    gen = _gen(rows)
    pos = torch.randint(0, 64, (rows, len(pairs)), generator=gen, device="cuda").float() * scale + far
    cos = torch.full((rows + 3, 64), 7.0, device="cuda")
    sin = torch.full((rows + 3, 64), 7.0, device="cuda")
    mi.rope_axes_tables(pos, pairs, cos[:rows], sin[:rows])
    angle = torch.cat([pos[:, a:a + 1].double() * 10000.0 ** (-torch.arange(n, device="cuda").double() / n)
                       for a, n in enumerate(pairs)], 1)
    within(cos[:rows], angle.cos(), torch.full_like(angle, 3 * F), "cos")
    within(sin[:rows], angle.sin(), torch.full_like(angle, 3 * F), "sin")
    assert (cos[rows:] == 7.0).all() and (sin[rows:] == 7.0).all()


def test_rope_axes_agrees_with_the_grid_builder():
    mi = require_gpu()
    t, gh, gw = 13, 17, 19
    rows = t + gh * gw
    pos = torch.empty(rows, 2)
    pos[:t] = torch.arange(t).float().view(-1, 1)
    pos[t:, 0] = torch.arange(gh).repeat_interleave(gw).float()
    pos[t:, 1] = torch.arange(gw).repeat(gh).float()
    a = [torch.empty(rows, 64, device="cuda") for _ in range(4)]
    mi.rope_tables(t, gh, gw, a[0], a[1])
    mi.rope_axes_tables(pos.cuda(), (32, 32), a[2], a[3])
    assert (a[0] - a[2]).abs().max() <= 3 * F and (a[1] - a[3]).abs().max() <= 3 * F


def test_rope_axes_not_finite():
    mi = require_gpu()
    pos = torch.tensor([[0.0], [math.inf], [math.nan], [3e38]], device="cuda")
    cos, sin = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    mi.rope_axes_tables(pos, (64,), cos, sin)
    assert (cos[0] == 1).all() and (sin[0] == 0).all()
    assert cos[1:3].isnan().all() and sin[1:3].isnan().all()
    assert mi.device_error() == 0


# ------------------------------------------------------------------------------------ q/k gradient
@pytest.mark.parametrize("batch,heads,seq,own,x_std", [
    (1, 1, 1, False, 1.0), (1, 2, 74, False, 1.0), (2, 3, 65, True, 1.0), (3, 5, 211, False, 30.0), (1, 17, 1023, True, 1e-3),
    (2, 8, 2500, True, 1.0)])
def test_qk_backward_parity(batch, heads, seq, own, x_std):
    mi = require_gpu()
    gen = _gen(heads * seq)
    rows, width = batch * seq, heads * HEAD
    qkv = _normal(gen, rows, 3 * width, std=x_std)
    if seq > 4:
        qkv[3] = 0  # a row of zeros: the norm is eps alone
    gains = [_normal(gen, HEAD, std=0.3, mean=1.0) for _ in range(2)]
    dy = [_normal(gen, batch, heads, seq, HEAD) for _ in range(2)]
    angle = torch.rand(batch if own else 1, seq, 64, generator=gen, device="cuda") * 50
    cos, sin = angle.cos(), angle.sin()
    dqkv = torch.full((rows + 5, 3 * width), 7.0, dtype=BF, device="cuda")
    dg = [torch.full((HEAD,), 7.0, device="cuda") for _ in range(2)]
    ws = torch.full((mi.qk_norm_rope_backward_workspace_size(batch, seq, heads),), 255, dtype=torch.uint8, device="cuda")

    def call():
        mi.qk_norm_rope_backward(qkv, *gains, cos, sin, *dy, dqkv[:rows], *dg, batch, seq, heads, ws, eps=1e-6,
                                 rope_bstride=seq * 64 if own else 0)

    call()
    c64, s64 = cos.double().unsqueeze(2), sin.double().unsqueeze(2)
    for i in range(2):
        x = qkv[:, i * width:(i + 1) * width].view(batch, seq, heads, HEAD).double()
        dx, dx_tol, dgain, dgain_tol = qk_backward64(x, gains[i].double(), c64, s64, dy[i].permute(0, 2, 1, 3).double(), 1e-6)
        got = dqkv[:rows, i * width:(i + 1) * width].view(batch, seq, heads, HEAD)
        within(got, dx, dx_tol, "dx")
        within(dg[i], dgain, dgain_tol, "dgain")
    assert (dqkv[:rows, 2 * width:] == 7.0).all() and (dqkv[rows:] == 7.0).all()
    before = (dqkv.clone(), dg[0].clone(), dg[1].clone())
    ws.fill_(0)
    call()
    assert torch.equal(before[0], dqkv) and torch.equal(before[1], dg[0]) and torch.equal(before[2], dg[1])


# ------------------------------------------------------------------------------------ the whole pass
@pytest.mark.parametrize("batch,heads,text,frames,gh,gw,pad", [(2, 2, 7, 3, 5, 6, 3), (1, 4, 33, 4, 9, 13, 0)])
def test_the_pass_as_it_is_used(batch, heads, text, frames, gh, gw, pad):
    """Video tables -> norm and rotation -> attention -> both gradients, against 64-bit autograd of the
    whole function from qkv and the gains to the output."""
    mi = require_gpu()
    gen = _gen(77)
    seq = text + frames * gh * gw
    rows, width = batch * seq, heads * HEAD
    pos = torch.zeros(seq, 3)
    pos[:text] = torch.arange(text).float().view(-1, 1)
    pos[text:] = torch.cartesian_prod(torch.arange(frames), torch.arange(gh), torch.arange(gw)).float() + text
    cos, sin = torch.empty(seq, 64, device="cuda"), torch.empty(seq, 64, device="cuda")
    mi.rope_axes_tables(pos.cuda(), (16, 24, 24), cos, sin)
    qkv = _normal(gen, rows, 3 * width)
    gains = [_normal(gen, HEAD, std=0.1, mean=1.2) for _ in range(2)]
    d_o = _normal(gen, rows, width)
    mask = None
    if pad:
        mask = torch.ones(batch, seq, dtype=torch.uint8, device="cuda")
        mask[-1, text - pad:text] = 0
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

    x = qkv.double().requires_grad_()
    g64 = [g.double().requires_grad_() for g in gains]
    parts = x.view(batch, seq, 3, heads, HEAD).permute(2, 0, 3, 1, 4)
    c64, s64 = cos.double(), sin.double()

    def turn(t, gain):
        t = t * torch.rsqrt(t.square().mean(3, keepdim=True) + 1e-6) * gain
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack([a * c64 - b * s64, a * s64 + b * c64], 4).flatten(3)

    z = turn(parts[0], g64[0]) @ turn(parts[1], g64[1]).transpose(2, 3) / math.sqrt(HEAD)
    if mask is not None:
        z = z.masked_fill((mask == 0)[:, None, None, :], -math.inf)
    out = (torch.softmax(z, 3) @ parts[2]).permute(0, 2, 1, 3).reshape(rows, width)
    (out * d_o.double()).sum().backward()

    # In the 2-norm, roundings that are independent of one another: q and k, P or dS, o, and each
    # stored gradient add at most U each relative to what they enter, 8 in a chain from qkv to dqkv.
    for got, ref, name in ((o, out, "o"), (dqkv, x.grad, "dqkv"), (dg[0], g64[0].grad, "dgq"), (dg[1], g64[1].grad, "dgk")):
        rel = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert rel <= 8 * U, f"{name}: {rel:.3g}"
        print(f"{name}: {rel:.3g}")

"""Norms whose tensors share memory as far as the calls allow it, on rows that begin anywhere; and norms on two streams at once."""
import math

import pytest
import torch

from tests._gpu import require_gpu
from tests._norms import TYPES, layer_norm64, norm_backward64, within
from tests.test_gpu_norms import Mod, Norm, _gen

pytestmark = pytest.mark.gpu
MANY = {33: 20011, 255: 9001, 515: 4003, 1155: 2503, 1283: 2503, 5003: 907, 10007: 611, 16383: 331}  # several turns of every group


class Columns:
    """Tensors of `rows` rows side by side in one buffer of NaN: tensor i has `width` columns from at[i] on, rows are `stride` apart."""

    def __init__(self, rows, width, dtype, at, stride, shift=0):
        self.rows, self.width, self.at, self.stride, self.shift = rows, width, at, stride, shift
        self.buf = torch.full((shift + rows * stride + 16,), math.nan, dtype=dtype, device="cuda")
        self.grid = self.buf[shift:shift + rows * stride].view(rows, stride)
        self.t = [self.grid[:, i:i + width] for i in at]

    def clean(self, what):
        """What is outside of the tensors is still NaN."""
        rest = self.buf.clone()
        grid = rest[self.shift:self.shift + self.rows * self.stride].view(self.rows, self.stride)
        for i in self.at:
            grid[:, i:i + self.width] = math.nan
        assert rest.isnan().all(), what


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", sorted(MANY))
@pytest.mark.parametrize("gap,shift", [(0, 0), (0, 1), (3, 5)])
def test_residual_in_place_on_odd_rows(width, kind, gap, shift):
    mi = require_gpu()
    n = Norm(MANY[width], width, kind, gap=gap, shift=shift, residual=True)
    n.statistics()
    ref = n.ref()
    n.dx = n.residual
    n.backward(mi)
    for name, got in (("dx", n.dx.t), ("dweight", n.dweight[:-1]), ("dbias", n.dbias[:-1])):
        within(got, ref[name], ref[name + "_tol"], name)
    n.dx.clean("dx")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", [33, 515, 1283, 5003, 10007])
@pytest.mark.parametrize("between", [0, 1])
def test_outputs_between_inputs(width, kind, between):
    """Columns that touch without overlapping: every granule at a border is read for one tensor while another is written."""
    mi = require_gpu()
    rows, step, g = MANY[width] // 2, width + between, _gen(width)
    c = Columns(rows, width, TYPES[kind], [0, step], 2 * step + 1, shift=1)
    x, y = c.t
    x.copy_(torch.randn(rows, width, generator=g, device="cuda") + 0.5)
    before = x.clone()
    mi.layer_norm(x, None, None, y)
    ref = layer_norm64(before, None, None, 1e-6)
    within(y, ref["y"], ref["y_tol"], "y")
    assert torch.equal(x, before)
    c.clean("forward")
    c = Columns(rows, width, TYPES[kind], [0, step, 2 * step, 3 * step], 4 * step, shift=3)
    dy, dx, x, r = c.t
    dy.copy_(torch.randn(rows, width, generator=g, device="cuda") * 0.05)
    x.copy_(before)
    r.copy_(torch.randn(rows, width, generator=g, device="cuda") * 0.05)
    inputs = [t.clone() for t in (dy, x, r)]
    mean, rstd = ref["mean"].float(), ref["rstd"].float()
    ws = torch.empty(mi.layer_norm_backward_workspace_size(rows, width), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    mi.layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, ws, residual=r)
    ref = norm_backward64(inputs[0], inputs[1], torch.ones(width, dtype=torch.float64, device="cuda"), mean.double()[:, None],
                          rstd.double()[:, None], inputs[2])
    for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
        within(got, ref[name], ref[name + "_tol"], name)
    assert all(torch.equal(a, b) for a, b in zip((dy, x, r), inputs))
    c.clean("backward")


def test_two_streams_at_once():
    """Replays of a captured pass and passes on another stream, with nothing between them that orders the two."""
    mi = require_gpu()
    a, m = Norm(3000, 1024, residual=True), Mod(2, 900, 512)
    b, k = Norm(2500, 1283, "f16", residual=True, seed=1), Mod(3, 700, 1280, seed=1)
    spaces = [t.workspace(mi) for t in (a, m, b, k)]
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def first():
        a.forward(mi)
        a.backward(mi, spaces[0])
        m.backward(mi, ws=spaces[1])

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        first()
        main.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            for _ in range(3):
                first()
    for t in (a, b):
        for out in (t.out, t.dx):
            out.t.zero_()
    for t in (m, k):
        t.dx.zero_()
    torch.cuda.synchronize()
    for _ in range(8):
        with torch.cuda.stream(main):
            graph.replay()
        for _ in range(3):
            b.forward(mi, stream=side)
            b.backward(mi, spaces[2], stream=side)
            k.backward(mi, ws=spaces[3], stream=side)
    torch.cuda.synchronize()
    for t in (a, b):
        ref = layer_norm64(t.x.t, t.weight, t.bias, 1e-6)
        within(t.out.t, ref["y"], ref["y_tol"], "y")
        t.check_backward()
    m.check()
    k.check()

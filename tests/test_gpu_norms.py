"""Layer norm, its gradient and the modulated RMSNorm's gradient against 64-bit forms."""
import math

import pytest
import torch

from tests._gpu import require_gpu
from tests._norms import TYPES, layer_norm64, norm_backward64, rms64, within

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Rows:
    """A tensor of rows inside a larger buffer of sevens: `gap` elements between rows, `shift` elements in front."""

    def __init__(self, rows, width, dtype, gap=0, shift=0, value=None):
        self.buf = torch.full((shift + max(rows, 1) * (width + gap) + 9,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[shift:shift + rows * (width + gap)].view(rows, width + gap)[:, :width]
        if value is not None:
            self.t.copy_(value)

    def clean(self, what):
        """Nothing around the rows was written."""
        rest = self.buf.clone()
        rows, stride = self.t.shape[0], self.t.stride(0)
        at = self.t.storage_offset()
        rest[at:at + rows * stride].view(rows, stride)[:, :self.t.shape[1]] = 7.0
        assert (rest == 7.0).all(), f"{what}: written outside its rows"


class Norm:
    def __init__(self, rows, width, kind="bf16", weights=None, gap=0, shift=0, offset=0.0, residual=False, seed=0):
        g = _gen(seed + 131 * rows + width)
        self.rows, self.width, self.dtype = rows, width, TYPES[kind]
        p = TYPES[weights or kind]

        def normal(*shape, std=1.0, mean=0.0):
            return torch.randn(*shape, generator=g, device="cuda") * std + mean

        x = normal(rows, width) + normal(1, width) + offset
        self.x = Rows(rows, width, self.dtype, gap, shift, x)
        self.dy = Rows(rows, width, self.dtype, 2 * gap, shift, normal(rows, width, std=0.05))
        self.residual = Rows(rows, width, self.dtype, gap, shift, normal(rows, width, std=0.05)) if residual else None
        self.weight, self.bias = normal(width, std=0.3, mean=1.0).to(p), normal(width, std=0.3).to(p)
        self.out = Rows(rows, width, self.dtype, 3 * gap, shift)
        self.dx = Rows(rows, width, self.dtype, gap, shift)
        self.mean, self.rstd = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
        self.dweight, self.dbias = (torch.full((width + 1,), 7.0, device="cuda") for _ in range(2))

    def forward(self, mi, eps=1e-6, **kw):
        mi.layer_norm(self.x.t, self.weight, self.bias, self.out.t, self.mean, self.rstd, eps=eps, **kw)

    def check_forward(self, mi, eps=1e-6):
        self.forward(mi, eps)
        ref = layer_norm64(self.x.t, self.weight, self.bias, eps)
        for name, got in (("y", self.out.t), ("mean", self.mean), ("rstd", self.rstd)):
            within(got, ref[name], ref[name + "_tol"], name)
        self.out.clean("out")

    def statistics(self, eps=1e-6):
        ref = layer_norm64(self.x.t, None, None, eps)
        self.mean.copy_(ref["mean"])
        self.rstd.copy_(ref["rstd"])

    def workspace(self, mi):
        return torch.full((mi.layer_norm_backward_workspace_size(self.rows, self.width),), 255, dtype=torch.uint8, device="cuda")

    def backward(self, mi, ws=None, **kw):
        mi.layer_norm_backward(self.dy.t, self.x.t, self.weight, self.mean, self.rstd, self.dx.t, self.dweight[:self.width],
                               self.dbias[:self.width], self.workspace(mi) if ws is None else ws,
                               residual=None if self.residual is None else self.residual.t, **kw)

    def ref(self):
        return norm_backward64(self.dy.t, self.x.t, self.weight.double(), self.mean.double()[:, None], self.rstd.double()[:, None],
                               None if self.residual is None else self.residual.t)

    def check_backward(self):
        ref = self.ref()
        for name, got in (("dx", self.dx.t), ("dweight", self.dweight[:-1]), ("dbias", self.dbias[:-1])):
            within(got, ref[name], ref[name + "_tol"], name)
        assert self.dweight[-1] == 7.0 and self.dbias[-1] == 7.0
        self.dx.clean("dx")


WIDTHS = [1, 2, 7, 8, 24, 31, 33, 64, 127, 128, 256, 257, 264, 511, 512, 520, 768, 1000, 1155, 1283, 1536, 1537, 2047, 2048, 2560, 4096,
          4097, 4104, 5003, 8191, 8192, 8200, 10007, 12288, 16383, 16384]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_layer_norm(width, kind, weights):
    mi = require_gpu()
    for rows in (1, 5, 74):
        Norm(rows, width, kind, weights).check_forward(mi)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind,weights", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_layer_norm_backward(width, kind, weights):
    mi = require_gpu()
    for rows, residual in ((1, False), (5, True), (74, False), (311, True)):
        n = Norm(rows, width, kind, weights, residual=residual)
        n.statistics()
        n.backward(mi)
        n.check_backward()


@pytest.mark.parametrize("width", [255, 513, 767, 769, 1023, 1025, 1535, 1791, 4095])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_odd_rows_where_the_layout_changes(width, kind):
    mi = require_gpu()
    for residual in (False, True):
        n = Norm(629, width, kind, residual=residual)
        n.check_forward(mi)
        n.statistics()
        n.backward(mi)
        n.check_backward()


@pytest.mark.parametrize("rows,width,kind", [(4130, 2560, "bf16"), (16418, 256, "bf16"), (100003, 40, "f16"), (9237, 1155, "f32"),
                                             (4503, 1283, "f16"), (20011, 33, "bf16"), (3001, 4096, "f32")])
def test_many_rows(rows, width, kind):
    mi = require_gpu()
    n = Norm(rows, width, kind, "f32", residual=rows % 2 == 1)
    n.check_forward(mi)
    n.statistics()
    n.backward(mi)
    n.check_backward()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gap,shift", [(8, 8), (8, 3), (3, 0), (1, 1), (16, 0), (5, 7)])
def test_strided_and_shifted_rows(kind, gap, shift):
    """Rows apart from each other, and buffers that begin anywhere."""
    mi = require_gpu()
    for rows, width in ((9, 40), (70, 256), (33, 1283), (12, 4096)):
        n = Norm(rows, width, kind, gap=gap, shift=shift, residual=True)
        n.check_forward(mi)
        n.statistics()
        n.backward(mi)
        n.check_backward()


def test_one_operand_out_of_line():
    """All but one tensor on 16-byte boundaries: the others' alignment does not count for it."""
    mi = require_gpu()
    for odd in ("x", "dy", "residual", "dx", "out", "weight", "bias"):
        n = Norm(37, 512, residual=True)
        if odd in ("weight", "bias"):
            v = torch.empty(513, dtype=n.dtype, device="cuda")[1:]
            v.copy_(getattr(n, odd))
            setattr(n, odd, v)
        else:
            setattr(n, odd, Rows(37, 512, n.dtype, 0, 1, getattr(n, odd).t))
        n.check_forward(mi)
        n.statistics()
        n.backward(mi)
        n.check_backward()


def test_without_parameters_and_statistics():
    mi = require_gpu()
    for rows, width in ((5, 33), (70, 1024)):
        n = Norm(rows, width)
        mi.layer_norm(n.x.t, None, None, n.out.t)
        ref = layer_norm64(n.x.t, None, None, 1e-6)
        within(n.out.t, ref["y"], ref["y_tol"], "y")
        n.weight = torch.ones_like(n.weight)
        n.statistics()
        mi.layer_norm_backward(n.dy.t, n.x.t, None, n.mean, n.rstd, n.dx.t, None, None, n.workspace(mi))
        ref = n.ref()
        within(n.dx.t, ref["dx"], ref["dx_tol"], "dx")
        for one in ("dweight", "dbias"):
            out = {"dweight": None, "dbias": None, one: getattr(n, one)[:-1]}
            mi.layer_norm_backward(n.dy.t, n.x.t, None, n.mean, n.rstd, n.dx.t, out["dweight"], out["dbias"], n.workspace(mi))
            within(out[one], ref[one], ref[one + "_tol"], one)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [50.0, -3000.0])
def test_rows_far_from_zero(kind, offset):
    """The mean is many deviations away: a variance from squares of x would be lost."""
    mi = require_gpu()
    for width in (40, 1000, 4096):
        Norm(21, width, kind, offset=offset).check_forward(mi)


def test_constant_rows_and_large_eps():
    mi = require_gpu()
    n = Norm(6, 257)
    n.x.t[:] = 3.0
    n.forward(mi)
    assert (n.mean == 3.0).all() and torch.allclose(n.rstd, torch.full_like(n.rstd, 1000.0), rtol=1e-6)
    assert torch.equal(n.out.t, n.bias.expand(6, 257))
    Norm(6, 300).check_forward(mi, eps=10.0)


def test_not_finite_rows_stay_alone():
    mi = require_gpu()
    for width in (33, 256, 2560, 5000):
        n = Norm(19, width)
        n.x.t[3, width // 2] = math.nan
        n.x.t[7, 0] = math.inf
        n.forward(mi)
        good = [i for i in range(19) if i not in (3, 7)]
        assert n.out.t[3].isnan().all() and n.mean[3].isnan() and n.rstd[3].isnan() and n.out.t[7].isnan().all()
        ref = layer_norm64(n.x.t[good], n.weight, n.bias, 1e-6)
        within(n.out.t[good], ref["y"], ref["y_tol"], "y")


@pytest.mark.parametrize("width,kind", [(33, "bf16"), (256, "bf16"), (1283, "f16"), (2560, "bf16"), (5000, "f32"), (16384, "bf16")])
def test_rows_without_a_gradient(width, kind):
    """dy = 0 (of either sign): dx is the residual's part and the row adds nothing, whatever x and the statistics hold."""
    mi = require_gpu()
    for rows, residual in ((9, True), (9, False), (200, True)):
        n = Norm(rows, width, kind, residual=residual)
        n.statistics()
        n.dy.t[2] = 0.0
        n.x.t[2] = math.nan
        n.dy.t[4] = -0.0
        n.x.t[4, width - 1] = -math.inf
        n.mean[4], n.rstd[4] = math.inf, math.nan
        n.dy.t[6] = 0.0
        n.mean[6] = math.nan
        n.backward(mi)
        n.mean[[4, 6]], n.rstd[4] = 0.0, 1.0
        n.check_backward()
        for i in (2, 4, 6):
            assert torch.equal(n.dx.t[i], n.residual.t[i] if residual else torch.zeros_like(n.dx.t[i]))
        n.dy.t[2, 0] = 1.0  # one entry, and the row counts: its NaN has to be seen
        n.backward(mi)
        assert n.dx.t[2].isnan().all() and n.dweight[:-1].isnan().all()


def test_no_rows():
    mi = require_gpu()
    n = Norm(0, 40)
    n.forward(mi)
    n.backward(mi)
    assert (n.dweight[:-1] == 0).all() and (n.dbias[:-1] == 0).all()


def test_residual_in_place_and_broadcast_rows():
    mi = require_gpu()
    n = Norm(50, 1024, residual=True)
    n.statistics()
    ref = n.ref()
    n.dx = n.residual
    n.backward(mi)
    within(n.dx.t, ref["dx"], ref["dx_tol"], "dx")
    n = Norm(50, 1024)
    row = n.dy.t[:1].clone()
    n.dy.t.copy_(row)
    n.statistics()
    ref = n.ref()
    mi.layer_norm_backward(row.expand(50, 1024), n.x.t, n.weight, n.mean, n.rstd, n.dx.t, n.dweight[:-1], n.dbias[:-1],
                           n.workspace(mi))
    within(n.dx.t, ref["dx"], ref["dx_tol"], "dx")
    within(n.dweight[:-1], ref["dweight"], ref["dweight_tol"], "dweight")


def test_columns_of_one_buffer():
    """Outputs beside inputs in the same rows."""
    mi = require_gpu()
    buf = torch.randn(40, 768, device="cuda").to(BF)
    x, y = buf[:, :256], buf[:, 512:]
    before = buf[:, :512].clone()
    mi.layer_norm(x, None, None, y)
    ref = layer_norm64(x, None, None, 1e-6)
    within(y, ref["y"], ref["y_tol"], "y")
    assert torch.equal(before, buf[:, :512])


def test_gradient_against_differences():
    """The slope of sum(dy y) along a direction, from the fp32 forward and backward, against the 64-bit forward."""
    mi = require_gpu()
    for rows, width in ((7, 96), (40, 1283)):
        n = Norm(rows, width, "f32")
        n.forward(mi)
        n.backward(mi)
        g = _gen(5)
        for name in ("x", "weight", "bias"):
            at = {"x": n.x.t.double(), "weight": n.weight.double(), "bias": n.bias.double()}
            got = {"x": n.dx.t, "weight": n.dweight[:-1], "bias": n.dbias[:-1]}[name].double()
            u = torch.randn(at[name].shape, generator=g, device="cuda", dtype=torch.float64)

            def loss(t):
                p = {**at, name: at[name] + t * u}
                return float((layer_norm64(p["x"], p["weight"], p["bias"], 1e-6)["y"] * n.dy.t.double()).sum())

            diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
            size = float(got.norm() * u.norm())
            assert abs(diff - float((got * u).sum())) <= 1e-5 * size, name  # 1e-6 of each, the difference's 1e-8 squared


# ------------------------------------------------------------------------------- modulated RMSNorm
class Mod:
    def __init__(self, batch, seq, hidden, residual=True, seed=0):
        g = _gen(seed + 17 * seq + hidden + batch)
        rows = batch * seq

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)

        self.dims = (batch, seq, hidden)
        self.x = normal(rows, hidden) * (1 + torch.arange(rows, device="cuda")[:, None] % 3).to(BF)
        self.dy, self.mod = normal(rows, hidden, std=0.05), normal(batch, 6, hidden, std=0.3)
        self.residual = normal(rows, hidden, std=0.05) if residual else None
        self.dx = torch.full_like(self.x, 7.0)
        self.dmod = torch.full((batch, 6, hidden), 7.0, device="cuda")

    def workspace(self, mi):
        return torch.full((mi.mod_rmsnorm_backward_workspace_size(*self.dims),), 255, dtype=torch.uint8, device="cuda")

    def backward(self, mi, shift_row=3, scale_row=1, ws=None, eps=1e-6, **kw):
        b, s, _ = self.dims
        mi.mod_rmsnorm_backward(self.dy, self.x, self.mod, shift_row, scale_row, self.dx, self.dmod, b, s,
                                self.workspace(mi) if ws is None else ws, eps=eps, residual=self.residual, **kw)

    def check(self, shift_row=3, scale_row=1, eps=1e-6):
        b, s, _ = self.dims
        for i in range(b):
            at = slice(i * s, (i + 1) * s)
            r, rel = rms64(torch.where((self.dy[at] == 0).all(1, keepdim=True), 0.0, self.x[at].double()), eps)
            ref = norm_backward64(self.dy[at], self.x[at], 1.0 + self.mod[i, scale_row].double(), None, r,
                                  None if self.residual is None else self.residual[at], rel)
            within(self.dx[at], ref["dx"], ref["dx_tol"], "dx")
            if shift_row == scale_row:
                within(self.dmod[i, scale_row], ref["dweight"] + ref["dbias"], ref["dweight_tol"] + ref["dbias_tol"]
                       + 2.0 ** -24 * (ref["dweight"] + ref["dbias"]).abs(), "dmod")
            else:
                within(self.dmod[i, scale_row], ref["dweight"], ref["dweight_tol"], "dscale")
                within(self.dmod[i, shift_row], ref["dbias"], ref["dbias_tol"], "dshift")
        rest = [k for k in range(6) if k not in (shift_row, scale_row)]
        assert (self.dmod[:, rest] == 7.0).all()


@pytest.mark.parametrize("batch,seq", [(1, 1), (1, 74), (2, 336), (3, 5), (7, 1), (2, 1500)])
@pytest.mark.parametrize("hidden", [256, 512, 1280, 1792, 2560, 4096])
def test_mod_backward(batch, seq, hidden):
    mi = require_gpu()
    for residual in (True, False):
        m = Mod(batch, seq, hidden, residual)
        m.backward(mi)
        m.check()


@pytest.mark.parametrize("hidden", [768, 1024, 2304, 2816, 3328, 3840])
def test_mod_backward_where_the_layout_changes(hidden):
    mi = require_gpu()
    for residual in (True, False):
        m = Mod(2, 701, hidden, residual)
        m.backward(mi)
        m.check()


def test_mod_backward_many_elements():
    mi = require_gpu()
    m = Mod(700, 3, 256)
    m.backward(mi)
    m.check()


def test_mod_backward_one_row_for_both():
    mi = require_gpu()
    m = Mod(2, 50, 512)
    m.backward(mi, 4, 4, eps=0.1)
    m.check(4, 4, eps=0.1)


def test_mod_backward_padded_rows():
    """Rows whose dy is zero may hold anything in x, and dx may be the residual's own tensor."""
    mi = require_gpu()
    for hidden in (256, 2560):
        m = Mod(2, 90, hidden)
        m.dy[10:30], m.dy[170] = 0.0, -0.0
        m.x[10:20], m.x[25], m.x[170, 5] = math.nan, math.inf, -math.inf
        res = m.residual.clone()
        m.dx = m.residual
        m.backward(mi)
        m.residual = res
        m.check()
        assert torch.equal(m.dx[10:30], res[10:30])


def test_mod_backward_follows_the_forward():
    """The slope of sum(dy y) of mod_rmsnorm's own formula, in 64 bits."""
    mi = require_gpu()
    m = Mod(2, 30, 256, residual=False)
    m.backward(mi, 2, 5)
    g = _gen(9)
    u = torch.randn(m.x.shape, generator=g, device="cuda", dtype=torch.float64)
    v = torch.randn(m.mod.shape, generator=g, device="cuda", dtype=torch.float64)

    def loss(t):
        x, mod = (m.x.double() + t * u).view(2, 30, 256), m.mod.double() + t * v
        y = x * (x.square().mean(2, keepdim=True) + 1e-6).rsqrt() * (1 + mod[:, 5:6]) + mod[:, 2:3]
        return float((y * m.dy.double().view(2, 30, 256)).sum())

    diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
    at = m.dmod.double()[:, [2, 5]]
    slope = float((m.dx.double() * u).sum() + (at * v[:, [2, 5]]).sum())
    # dx is rounded to bf16: each entry by 2^-8 at most, with u's signs at random
    assert abs(diff - slope) <= 2.0 ** -8 * float((m.dx.double() * u).norm()) * 4 + 1e-5 * abs(diff)


# ------------------------------------------------------------------------------------- both
def test_repeats_have_the_same_bytes():
    mi = require_gpu()
    for rows, width, kind in ((300, 1283, "f16"), (4130, 1024, "bf16"), (74, 256, "bf16")):
        n = Norm(rows, width, kind, residual=True)
        n.forward(mi)
        n.backward(mi)
        first = [t.clone() for t in (n.out.t, n.mean, n.rstd, n.dx.t, n.dweight, n.dbias)]
        Norm(50, 700).forward(mi)
        n.forward(mi)
        n.backward(mi, torch.zeros_like(n.workspace(mi)))
        assert all(torch.equal(a, b) for a, b in zip(first, (n.out.t, n.mean, n.rstd, n.dx.t, n.dweight, n.dbias)))


def test_captured_and_on_another_stream():
    """The pass captured into a graph and replayed on new inputs, with other work on a second stream."""
    mi = require_gpu()
    n, m = Norm(333, 1024, residual=True), Mod(2, 150, 512)
    ws, wm = n.workspace(mi), m.workspace(mi)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n.forward(mi)
        n.backward(mi, ws)
        m.backward(mi, ws=wm)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            n.forward(mi)
            n.backward(mi, ws)
            m.backward(mi, ws=wm)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2):
        new, new_m = Norm(333, 1024, residual=True, seed=seed), Mod(2, 150, 512, seed=seed)
        for a, b in ((n.x, new.x), (n.dy, new.dy), (n.residual, new.residual)):
            a.t.copy_(b.t)
        for a, b in ((m.x, new_m.x), (m.dy, new_m.dy), (m.residual, new_m.residual), (m.mod, new_m.mod)):
            a.copy_(b)
        graph.replay()
        other = Norm(200, 512, residual=True, seed=seed)
        side.wait_stream(torch.cuda.current_stream())
        other.forward(mi, stream=side)
        other.backward(mi, torch.full_like(other.workspace(mi), 9), stream=side)
        torch.cuda.synchronize()
        n.check_backward()
        m.check()
        other.check_backward()


def test_rows_past_32_bits():
    """More than 2^31 elements: offsets of the last rows."""
    mi = require_gpu()
    rows, width = 140000, 16384
    x = torch.zeros(rows, width, dtype=BF, device="cuda")
    last = slice(rows - 40, rows)
    g = _gen(3)
    x[last] = torch.randn(40, width, generator=g, device="cuda").to(BF)
    dy = torch.zeros_like(x)
    dy[last] = torch.randn(40, width, generator=g, device="cuda").to(BF)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    mi.layer_norm(x, None, None, out, mean, rstd)
    ws = torch.empty(mi.layer_norm_backward_workspace_size(rows, width), dtype=torch.uint8, device="cuda")
    mi.layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, ws)
    ref = layer_norm64(x[last], None, None, 1e-6)
    within(out[last], ref["y"], ref["y_tol"], "y")
    ref = norm_backward64(dy[last], x[last], torch.ones(width, dtype=torch.float64, device="cuda"), mean[last].double()[:, None],
                          rstd[last].double()[:, None])
    within(dx[last], ref["dx"], ref["dx_tol"], "dx")
    within(dw, ref["dweight"], ref["dweight_tol"], "dweight")
    assert (out[:rows - 40].count_nonzero() == 0) and (dx[:rows - 40].count_nonzero() == 0)


def test_refusals_on_the_gpu():
    mi = require_gpu()
    n = Norm(10, 64)
    ws = n.workspace(mi)
    with pytest.raises(mi.MiError, match="workspace 255 bytes"):
        n.backward(mi, ws[:255])
    with pytest.raises(ValueError, match="expected 10 rows of 64"):
        mi.layer_norm(n.x.t, n.weight, n.bias, n.out.t[:9])
    with pytest.raises(TypeError, match="out: expected torch.bfloat16"):
        mi.layer_norm(n.x.t, n.weight, n.bias, n.out.t.float())
    with pytest.raises(TypeError, match="weight and bias: expected torch.bfloat16 or torch.float32"):
        mi.layer_norm(n.x.t, n.weight.half(), None, n.out.t)
    with pytest.raises(TypeError, match="bias: expected torch.bfloat16"):
        mi.layer_norm(n.x.t, n.weight, n.bias.float(), n.out.t)
    with pytest.raises(ValueError, match="contiguous"):
        mi.layer_norm(n.x.t, n.weight, n.bias, torch.empty(64, 10, dtype=BF, device="cuda").T)
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.layer_norm(n.x.t, n.weight, n.bias, n.x.t)
    with pytest.raises(mi.MiError, match="overlaps"):
        mi.layer_norm_backward(n.dy.t, n.x.t, n.weight, n.mean, n.rstd, n.dy.t, None, None, ws)
    m = Mod(1, 10, 256)
    with pytest.raises(ValueError, match="dmod has 1280 elements, expected 1536"):
        mi.mod_rmsnorm_backward(m.dy, m.x, m.mod, 0, 1, m.dx, m.dmod[:, :5].contiguous(), 1, 10, ws)

"""Rows whose dy is zero in layer norm's gradient, with finite values of any size in x and the statistics."""
import pytest
import torch

from tests._gpu import require_gpu
from tests.test_gpu_norms import Norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width,kind", [(33, "bf16"), (33, "f32"), (256, "f16"), (257, "f32"), (1283, "f16"), (2560, "bf16"),
                                        (5000, "f32"), (5003, "bf16"), (16384, "bf16")])
def test_finite_extremes_in_rows_without_a_gradient(width, kind):
    """(x - mean) rstd overflows, and the sums of the row are zeros: dx is the residual's part, and the row adds nothing."""
    mi = require_gpu()
    large = 6e4 if kind == "f16" else 1e30
    for rows, residual in ((9, True), (9, False), (400, True)):
        n = Norm(rows, width, kind, residual=residual)
        n.statistics()
        dead = {2: (large, 0.0, 1e38), 3: (-large, 1e20, 3e38), 6: (0.0, -3e38, 1e10), rows - 1: (large, -large, 1e36)}
        for i, (x, mean, rstd) in dead.items():
            n.dy.t[i] = -0.0 if i == 3 else 0.0
            n.x.t[i, :] = x
            n.x.t[i, ::3] = 0.5
            n.mean[i], n.rstd[i] = mean, rstd
        n.backward(mi)
        for i in dead:
            assert torch.equal(n.dx.t[i], n.residual.t[i] if residual else torch.zeros_like(n.dx.t[i]))
            n.mean[i], n.rstd[i] = 0.0, 1.0
        n.check_backward()


@pytest.mark.parametrize("width,kind", [(34, "bf16"), (256, "f32"), (1284, "f16"), (2560, "bf16"), (5000, "f32"), (16384, "bf16")])
def test_rows_whose_sums_are_zero_count(width, kind):
    """g and g n add up to nothing, but dy is not zero: the row has a gradient."""
    mi = require_gpu()
    n = Norm(21, width, kind)
    n.weight.fill_(1.0)
    n.x.t[4], n.dy.t[4] = 3.0, 0.0
    n.dy.t[4, 0::2], n.dy.t[4, 1::2] = 0.25, -0.25
    n.statistics()
    n.backward(mi)
    n.check_backward()
    assert torch.equal(n.dx.t[4].double(), (n.dy.t[4].double() * n.rstd[4].double()).float().to(n.dtype).double())

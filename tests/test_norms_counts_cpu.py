"""Counts of rows that do not fit the library's 32-bit integers are refused, not cut to their low bits."""
import pytest
import torch

MANY = [(1 << 31), (1 << 32), (1 << 32) + 5]


class Many:
    """Stands for a tensor on the GPU of so many rows of two columns."""
    dtype, shape = torch.bfloat16, (0, 2)

    def __init__(self, rows):
        self.rows = rows

    def numel(self):
        return 2 * self.rows


@pytest.fixture
def mi(monkeypatch):
    import diffusion_transformer_denoiser_gb300 as mi
    from diffusion_transformer_denoiser_gb300 import _build

    _build.build()
    monkeypatch.setattr(mi, "_on_current", lambda t, name: 0)
    return mi


@pytest.mark.parametrize("rows", MANY)
def test_more_rows_than_an_int(mi, rows):
    t = Many(rows)
    for call in (lambda: mi.layer_norm(t, None, None, t),
                 lambda: mi.layer_norm_backward(t, t, None, t, t, t, None, None, None),
                 lambda: mi.layer_norm_backward_workspace_size(rows, 2),
                 lambda: mi.layer_norm_backward_workspace_size(2, rows),
                 lambda: mi.mod_rmsnorm_backward_workspace_size(rows, 1, 256),
                 lambda: mi.mod_rmsnorm_backward_workspace_size(1, rows, 256),
                 lambda: mi.mod_rmsnorm_backward_workspace_size(1, 1, rows)):
        with pytest.raises(ValueError, match=f"={rows}: at most 2147483647"):
            call()


def test_counts_that_fit(mi):
    assert mi._count(0x7fffffff, "rows") == 0x7fffffff and mi._count(-1, "rows") == -1
    with pytest.raises(mi.MiError, match="negative"):
        mi.layer_norm_backward_workspace_size(-1, 2)

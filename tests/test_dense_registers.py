"""The dense layers' kernels in the built library (CPU): next to none keeps values in scratch memory, whose reloads would
wait for every load in flight; and their references' derivatives are slopes."""
import pytest
import torch

from dense_helpers import ACTS, act64
from test_kernel_registers import found  # noqa: F401  (the fixture)

MOST = 4


@pytest.mark.parametrize("kernel", ["tile_kernel", "pair_kernel", "few_anywhere_kernel", "few_stream_kernel", "join_kernel",
                                    "gate_grad_kernel", "dz_kernel", "norm_kernel", "norm_long_kernel", "norm_grad_kernel", "norm_grad_long_kernel",
                                    "norm_columns_kernel", "join_columns_kernel"])
def test_no_kernel_spills(found, kernel):  # noqa: F811
    these = [k for k in found if kernel in k[".name"]]
    assert these
    spilled = {k[".name"]: k[".vgpr_spill_count"] for k in these if k[".vgpr_spill_count"] > MOST}
    assert not spilled


@pytest.mark.parametrize("act", ACTS)
def test_derivatives_are_slopes(act):
    """Central differences in float64: h^2 / 6 of a third derivative below 2, and 2^-52 of the values over h."""
    z, h = torch.linspace(-8, 8, 4001, dtype=torch.float64) + 1e-4, 1e-5
    slope = (act64(z + h, act)[0] - act64(z - h, act)[0]) / (2 * h)
    assert float((slope - act64(z, act)[1]).abs().max()) <= 2 * h * h / 6 + 8 * 2.0 ** -51 / h

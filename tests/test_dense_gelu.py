"""The fit of the normal distribution's tail that GELU takes (CPU): its constants, read from the kernel's source, against
64 bits."""
import os
import re

import pytest
import torch

from combine_expert_histogram_amd import build


def test_the_fit_is_as_near_as_its_comment_says():
    with open(os.path.join(build.CSRC, "dense.h")) as f:
        body = f.read().split("float gelu_cdf(", 1)[1].split("bell =", 1)[0]
    slope, one = (float(v) for v in re.search(r"fmaf\(([\d.]+)f, fabsf\(z\), ([\d.]+)f\)", body).groups())
    first = float(re.search(r"float q = (-?[\d.e-]+)f;", body).group(1))
    rest = [float(v) for v in re.findall(r"q = fmaf\(q, t, (-?[\d.e-]+)f\)", body)]
    assert (slope, one, len(rest)) == (0.375, 1.0, 8)
    u = torch.cat((torch.linspace(0, 40, 400001, dtype=torch.float64), torch.logspace(-12, 6, 40001, dtype=torch.float64)))
    # e^(u^2 / 2) erfc(u / sqrt 2) / 2
    want = torch.special.erfcx(u / 2 ** 0.5) / 2
    t, q = 1 / (1 + 0.375 * u), torch.full_like(u, first).float().double()
    for c in rest:
        q = q * t + float(torch.tensor(c, dtype=torch.float32))
    worst = float((q * t / want - 1).abs().max())
    assert worst == pytest.approx(2.53e-7, rel=0.01)
    assert float((q * t / want - 1).abs()[0]) == pytest.approx(worst, rel=1e-3), "the largest error is at 0"

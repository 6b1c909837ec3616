"""The trained-layer operators where an evaluation loses digits.  F32 is half a step of fp32, TC a
whole one (an add that truncates)."""

import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from matrix_aware_optimizers_02_b200 import api as A
    yield A
    assert A.layer_status() == (0, 0)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ layer norm far from zero
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("cols", [24, 264, 1000, 1544, 5000, 8200, 14336, 20008])
def test_norm_far_from_zero(api, cols, dt):
    """Constant rows, rows of one spike and rows of small noise, all with a large mean.

    A row sum has a chain of at most 72 adds, so the mean of one pass is off by delta <= 72 F32
    |mean|; that must leave no trace but its own rounding, (72 F32)^2 |mean|, in what is scaled
    by rstd.  The deviations d themselves round once, their squares' sum in another chain."""
    g = _gen(cols)
    t = DT[dt]
    top = 30000.0 if dt == "fp16" else 1e5
    base = torch.empty((48, 1), device="cuda").uniform_(100.0, top, generator=g)
    x = base.expand(48, cols).contiguous()
    step = torch.finfo(t).eps
    x[16:32, 3] *= 1 + 3 * step
    x[32:] *= 1 + 4 * step * torch.randn((16, cols), generator=g, device="cuda")
    x = x.to(t)
    w, b = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    eps = 1e-5
    y, mean, rstd, _ = api.layer_norm(x, w, b, eps=eps)
    want, mean_w, rstd_w = R.layer_norm(x, w, b, eps)
    d = (x.double() - mean_w[:, None]).abs()
    chain = 72 * R.F32
    far = chain ** 2 * mean_w.abs()
    R.close(mean, mean_w, 1.01 * R.F32 * mean_w.abs() + far + 2 * R.F32 * d.mean(1), "mean")
    var = (d * d).mean(1)
    delta = chain * mean_w.abs()
    # of the variance: its sum's chain, with delta^2 in it until that is taken off
    rel = 0.5 * (2 * chain * (var + 2 * delta ** 2) / (var + eps)) + 8 * R.F32
    assert float(rel.max()) < 0.5  # else the bound says nothing
    R.close(rstd, rstd_w, rel * rstd_w, "rstd")
    scaled = d * rstd_w[:, None] * w.double().abs()
    tol = 1.01 * R.HALF_STEP[t] * want.abs() + scaled * (rel[:, None] + 8 * R.F32)
    tol = tol + (far * rstd_w)[:, None] * w.double().abs() + 4 * R.F32 * (scaled + b.double().abs())
    R.close(y, want, tol, "y")

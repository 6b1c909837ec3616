"""The trained-layer operators where an evaluation loses digits.  F32 is half a step of fp32, TC a
whole one (an add that truncates)."""

import math

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


# ------------------------------------------------------------------ fp32 read-back through an activation
@pytest.mark.parametrize("act", R.ACTS)
def test_restore_to_fp32_keeps_the_tails(api, act):
    """Relative to each value, from -108 to 108 (where exp(-|z|) and the results are subnormal)
    and far outside.  In half steps: CUDA's expf is off by at most 2 units in the last place (4
    half steps), erfcf-like functions by 4 (8); a relative error of an exponential's argument v
    counts |v| times; every product, quotient and sum of one sign adds 1.

    gelu: 4 + 8, the tail function's argument 2 (its own relative slope is at most 1), products 3,
    and where z > 0 one from 1 - tail: 18.  silu: 4, the sum 2, quotient and products 3: 9.
    gelu_tanh: the same with an argument off by 4, so 4 |v| more.  A subnormal exponential is off
    by 2^-150, its result by |z| times that, and rounds to 2^-150 itself."""
    z = torch.cat([torch.linspace(-14, 14, 16384), torch.linspace(-108, 108, 8192),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-6, -1e-6, 1e15, -1e15, 1e25, -1e25, 1e38, -1e38] * 2 + [0.0] * 8)])
    z = z.view(-1, 32).cuda()
    k = api.checkpoint8(z)
    z = k.restore()
    assert torch.equal(z.double(), R.unpack(k.q, k.e, 32))
    zd = z.double()
    tiny = torch.zeros_like(zd)
    if act == "gelu":
        half = torch.full_like(zd, 18.0)
    elif act == "silu":
        half = torch.full_like(zd, 10.0)
    elif act == "gelu_tanh":
        v = 2 * math.sqrt(2 / math.pi) * (zd.abs() + 0.044715 * zd.abs() ** 3)
        half = 10 + 4 * v.clamp(max=120.0)
    else:
        half = torch.full_like(zd, 1.0)
    if act in ("gelu", "silu", "gelu_tanh"):
        tiny = 2.0 ** -149 * (1 + zd.abs().clamp(max=128.0))
    # the 64-bit values of the tails, without the cancellation of 1 + tanh
    want = R.act(zd, act) if act != "gelu_tanh" else \
        zd * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (zd + 0.044715 * zd ** 3))
    want = torch.where(want > torch.finfo(torch.float32).max, torch.full_like(want, math.inf), want)
    R.close(k.restore(act=act), want, 1.01 * half * R.F32 * want.abs() + tiny, act)
    nan = api.Checkpoint8(torch.zeros((1, 32), dtype=torch.int8, device="cuda"),
                          torch.full((1, 1), 255, dtype=torch.uint8, device="cuda"), 32, torch.float32)
    assert torch.isnan(nan.restore(act=act)).all()


# ------------------------------------------------------------------ slopes of the largest values
@pytest.mark.parametrize("act", [a for a in R.ACTS if a != "none"])
def test_slopes_of_the_largest_values(api, act):
    """z up to the end of bf16's range, whose square fp32 cannot hold: the slope is 0, 1 or 2 z."""
    t = torch.bfloat16
    z = torch.tensor([1e4, 1e9, 1e13, 1.8e19, 2e19, 1e25, 1e30, 1.6e38], device="cuda").to(t)
    z = torch.cat([z, -z, z, -z]).view(1, 32)
    dy = torch.ones((1, 32), dtype=t, device="cuda")
    w = torch.eye(32, dtype=t, device="cuda")
    want = torch.where(z.double() > 0, 2 * z.double() if act == "relu2" else torch.ones_like(z.double()), 0.0)
    for zz in (z, api.checkpoint8(z.view(32, 1).expand(32, 32).contiguous())):
        rows = 1 if zz is z else 32
        d = dy.expand(rows, 32).contiguous()
        x = torch.zeros((rows, 32), dtype=t, device="cuda")
        s = want if rows == 1 else want.view(32, 1).expand(32, 32)
        if rows == 32 and act == "relu2":
            v = zz.restore().double()
            s = torch.where(v > 0, 2 * v, 0.0)
        dx, dw, db = api.linear_backward(d, x, w, z=zz, act=act)
        R.close(dx, s, 1.01 * R.HALF_STEP[t] * s.abs() + 1e-6, "dx")
        assert (dw == 0).all()
        # fp32 sums of at most 32 terms; two of relu2's largest pass fp32's end
        total = s.sum(0)
        total = torch.where(total > torch.finfo(torch.float32).max, torch.full_like(total, math.inf), total)
        R.close(db, total, 34 * R.F32 * s.abs().sum(0) + 1e-6, "db")


# ------------------------------------------------------------------ long sums
def _positive(g, rows, cols, lo, hi, t):
    return torch.empty((rows, cols), device="cuda").uniform_(lo, hi, generator=g).to(t)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_16_bit_results_of_long_one_signed_sums(api, dt):
    """2^17 tokens into a 16-bit dW.  With sums joined in fp32 every 8192 terms a sum is off by 512
    truncated adds of at most a step each (and 40 for the products inside and the joining), beside
    half a step of the result."""
    g = _gen(3)
    t = DT[dt]
    rows, n, m = 1 << 17, 4096, 4096
    dy, x = _positive(g, rows, m, 0.05, 0.15, t), _positive(g, rows, n, 0.05, 0.15, t)
    w = torch.zeros((m, n), dtype=t, device="cuda")
    _, dw, _ = api.linear_backward(dy, x, w, need_dx=False, need_db=False, dw_dtype=t)
    del w
    want = torch.zeros((m, 256), dtype=torch.float64, device="cuda")
    for r in range(0, rows, 16384):
        want += dy[r:r + 16384].double().t() @ x[r:r + 16384, :256].double()
    R.close(dw[:, :256], want, (1.01 * R.HALF_STEP[t] + 552 * R.TC) * want, "dw")


def test_fp32_gradient_of_one_sign(api):
    """A truncated add is off to one side, so a sum of one sign shows it in full.  16384 tokens:
    parts of at most 12 k-blocks have 48 such adds of at most one step of what is summed so far
    (half the part in the mean), and 16 products inside each; 22 parts are joined by rounded adds.
    One sum of the whole K is off by 1.0e-4, sixteen times the bound."""
    g = _gen(1)
    t = torch.float16
    rows, n, m = 16384, 2048, 4096
    dy, x = _positive(g, rows, m, 0.5, 1.5, t), _positive(g, rows, n, 0.5, 1.5, t)
    w = torch.zeros((m, n), dtype=t, device="cuda")
    _, dw, _ = api.linear_backward(dy, x, w, need_dx=False, need_db=False)
    want = dy.double().t() @ x.double()
    R.close(dw, want, ((48 / 2 + 16) * R.TC + 23 * R.F32) * want, "dw")


def test_kept_z_rounds_as_its_sums_do(api):
    """Values of a kept z that round the other way than the exact z's: an error e of a sum does
    that with probability |e| / step.  In the model of truncating adds the sums of parts of 11
    k-blocks (K = 4096, unit results) are off by 5.9e-7 in the mean, one sum of the whole K by
    4.0e-6 (553 such values, where the first expects 97); at most twice the first is allowed."""
    g = _gen(2)
    t = torch.bfloat16
    rows, n, m = 2048, 4096, 2048
    x = torch.randn((rows, n), generator=g, device="cuda").to(t)
    w = (torch.randn((m, n), generator=g, device="cuda") * n ** -0.5).to(t)
    _, kept = api.linear(x, w, checkpoint=True)
    q, e = R.pack(x.double() @ w.double().t())
    same = (kept.e == e).repeat_interleave(32, 1)
    flips = int(((kept.q != q) & same).sum())
    per = float((5.9e-7 / torch.exp2(e.double() - 127)).sum()) * 32
    assert flips <= 2 * per + 5 * math.sqrt(2 * per), f"{flips} values round the other way, {per:.0f} expected"
    assert int((~same).sum()) <= 32 * 32  # a block whose largest value lies that close to a power of two

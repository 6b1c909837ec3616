"""The trained-layer operators on the GPU against their definitions in 64 bits (layer_ref).

Tolerances count roundings.  u is half a step of the output's type; an fp32 sum over a row or a
column is off by at most (its longest chain of adds) * 2^-24 of the sum of magnitudes; a
tensor-core sum over K truncates once per 16 of K and inside each group of 16 products, at
most (K / 16 + 16) steps of 2^-23 of the sum of magnitudes.
"""

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


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _strided(t, extra=16):
    """The same values with a row stride larger than the row."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device=t.device)
    buf[:, 8:8 + t.shape[1]] = t
    return buf[:, 8:8 + t.shape[1]]


# ------------------------------------------------------------------ checkpoints
SIZES = [(1, 8), (3, 24), (5, 32), (2, 40), (129, 768), (7, 1000), (33, 4104), (1, 14336), (3000, 16)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_checkpoint_bits(api, rows, cols, dt):
    g = _gen(rows * 7 + cols)
    x = _randn(g, rows, cols) * torch.exp2(torch.randint(-30, 20, (rows, 1), generator=g, device="cuda").float())
    x = x.to(DT[dt])
    for v in (x, _strided(x)):
        k = api.checkpoint8(v)
        q, e = R.pack(x)
        assert torch.equal(k.q, q) and torch.equal(k.e, e)
        assert k.nbytes == rows * 33 * ((cols + 31) // 32)
        back = k.restore()
        assert back.dtype == DT[dt]
        want = R.unpack(q, e, cols)
        # exact, fp16 included; a block whose fp16 inputs hold an infinity is NaN in both
        R.close(back, want, 0.0, "restored")


def test_checkpoint_borders(api):
    """Zeros, ties, limits, the largest and smallest magnitudes, NaN and infinities."""
    big = torch.finfo(torch.float32).max
    rows = [[0.0] * 32,
            [127.4, 64.0] + [0.5, 1.5, 2.5, -0.5, -1.5, -2.5] * 5,         # ties to even at step 1
            [127.6, -127.6, 127.5, 126.5] + [1.0] * 28,                    # limited to +-127
            [big, -big] + [0.0] * 30,
            [1e-45, -1e-45] + [0.0] * 30, [2.0 ** -120, 2.0 ** -126] + [0.0] * 30,
            [math.nan] + [1.0] * 31, [math.inf] + [1.0] * 31, [1.0] * 31 + [-math.inf],
            [-0.0] * 32]
    x = torch.tensor(rows, device="cuda")
    k = api.checkpoint8(x)
    q, e = R.pack(x)
    assert torch.equal(k.q, q) and torch.equal(k.e, e)
    back = k.restore()
    assert torch.isnan(back[6:9]).all() and torch.isfinite(back[:6]).all()
    assert torch.equal(back[:6].double(), R.unpack(q, e, 32)[:6])
    # fp16's largest values stay finite
    h = torch.full((1, 32), torch.finfo(torch.float16).max, dtype=torch.float16, device="cuda")
    assert torch.equal(api.checkpoint8(h).restore(), torch.full_like(h, 65024.0))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("act", R.ACTS)
def test_restore_through_an_activation(api, act, dt):
    x = _randn(_gen(3), 67, 1000, std=2.5, dtype=DT[dt])
    k = api.checkpoint8(x)
    z = R.unpack(k.q, k.e, 1000)
    want = R.act(z, act)
    # fp32 evaluation: __expf is off by 2 + 1.2 |arg| steps, the few products by a step each
    tol = R.HALF_STEP[DT[dt]] * want.abs() * 1.01 + (16 + 6 * z.abs()) * R.TC * z.abs() * (1 + z.abs()) + 2.0 ** -25 * (dt == "fp16")
    R.close(k.restore(act=act), want, tol, act)


def test_restore_dtype_and_empty(api):
    k = api.checkpoint8(_randn(_gen(1), 9, 64, dtype=torch.bfloat16))
    assert k.restore(dtype=torch.float32).dtype == torch.float32
    assert torch.equal(k.restore(dtype=torch.float32).bfloat16(), k.restore())
    e = api.checkpoint8(torch.empty((0, 64), device="cuda"))
    assert e.shape == (0, 64) and e.restore().shape == (0, 64)


# ------------------------------------------------------------------ layer norm
NORM = [(1, 8), (2, 24), (5, 256), (129, 264), (300, 768), (1, 1000), (7, 1544), (3000, 1536), (33, 2056), (65, 4096),
        (3, 4104), (5, 8200), (9, 14336), (2, 16392), (3, 32768)]


def _norm_tol(x, w, b, y, rstd, u):
    """A row's sums have chains of at most 32 + 5 + 32 adds; mean, deviation and variance each
    bring that many half steps of the row's largest magnitude, the scaling a few more."""
    big = (x.double().abs().amax(1) * rstd)[:, None] * w.double().abs()
    bias = 0 if b is None else b.double().abs()
    return u * y.abs() * 1.01 + 256 * R.F32 * (big + y.abs() + bias)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", NORM)
def test_layer_norm(api, rows, cols, dt):
    g = _gen(rows + cols)
    x = (_randn(g, rows, cols) + 3.0).to(DT[dt])
    w, b = 1 + _randn(g, cols, std=0.2), _randn(g, cols, std=0.2)
    if dt != "fp32" and rows % 2:
        w, b = w.to(DT[dt]), b.to(DT[dt])
    if rows == 129:
        b = None
    want, mean_w, rstd_w = R.layer_norm(x, w, b, 1e-5)
    y, mean, rstd, kept = api.layer_norm(_strided(x) if cols % 16 else x, w, b, eps=1e-5, checkpoint=rows % 3 != 1)
    big = x.double().abs().amax(1)
    R.close(mean, mean_w, 128 * R.F32 * big, "mean")
    R.close(rstd, rstd_w, 256 * R.F32 * rstd_w * (1 + 2 * big * rstd_w), "rstd")
    R.close(y, want, _norm_tol(x, w, b, want, rstd_w, R.HALF_STEP[DT[dt]]), "y")
    if rows % 3 != 1:  # the fused checkpoint is that of y, bit for bit
        q, e = R.pack(y)
        assert torch.equal(kept.q, q) and torch.equal(kept.e, e)
    else:
        assert kept is None


def test_layer_norm_odd_rows(api):
    """Constant rows, a NaN row and a far mean among ordinary rows; rows behind stay untouched."""
    x = _randn(_gen(5), 6, 768)
    x[1] = 2.5
    x[2, 5] = math.nan
    x[3] += 1000.0
    w, b = torch.ones(768, device="cuda"), torch.zeros(768, device="cuda")
    y, mean, rstd, kept = api.layer_norm(x, w, b, checkpoint=True)
    want, _, rstd_w = R.layer_norm(x, w, b, 1e-5)
    assert torch.isnan(y[2]).all() and torch.isnan(kept.restore()[2]).all()
    assert (y[1] == 0).all()
    fine = [0, 1, 3, 4, 5]
    R.close(y[fine], want[fine], _norm_tol(x[fine], w, b, want[fine], rstd_w[fine], R.F32), "y")
    e = api.layer_norm(x[:0], w, b, checkpoint=True)
    assert e[0].shape == (0, 768) and e[3].shape == (0, 768)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", NORM)
def test_layer_norm_backward(api, rows, cols, dt):
    g = _gen(rows * 3 + cols)
    t = DT[dt]
    x = (_randn(g, rows, cols) + 0.5).to(t)
    dy = _randn(g, rows, cols, std=0.1, dtype=t)
    w = 1 + _randn(g, cols, std=0.2)
    dres = _randn(g, rows, cols, std=0.1, dtype=t) if rows % 2 else None
    kept = api.checkpoint8(x) if cols % 3 else None
    xv = R.unpack(kept.q, kept.e, cols) if kept is not None else x.double()
    _, mean, rstd = R.layer_norm(xv, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want = R.layer_norm_backward(dy, xv, w, mean, rstd, dres)
    dx, dw, db = api.layer_norm_backward(_strided(dy) if cols % 16 else dy, kept if kept is not None else x, w, mean, rstd, dres=dres)
    h = ((xv - mean.double()[:, None]) * rstd.double()[:, None]).abs()
    u_ = dy.double().abs() * w.double().abs()
    terms = rstd.double()[:, None] * (u_ + u_.mean(1, keepdim=True) + h * (u_ * h).mean(1, keepdim=True))
    if dres is not None:
        terms = terms + dres.double().abs()
    # h has 3 roundings, the row sums chains of at most 32 + 5 + 32 adds
    R.close(dx, want[0], R.HALF_STEP[t] * want[0].abs() * 1.01 + 128 * R.F32 * terms, "dx")
    # a column's chain: the rows of one block, then the blocks
    chain = (rows / 100 + 400 + 8) * R.F32
    R.close(dw, want[1], chain * (dy.double().abs() * h).sum(0), "dw")
    R.close(db, want[2], chain * dy.double().abs().sum(0), "db")


def test_layer_norm_backward_against_differences(api):
    """The gradient of sum(dy * y) by central differences of the forward's definition."""
    g = _gen(11)
    x, w, b = _randn(g, 3, 40), 1 + _randn(g, 40, std=0.2), _randn(g, 40)
    dy = _randn(g, 3, 40)
    _, mean, rstd, _ = api.layer_norm(x, w, b)
    dx, dw, db = api.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        return (R.layer_norm(x, w, b, 1e-5)[0] * dy.double()).sum().item()

    h = 1e-5
    for grad, args in ((dx, 0), (dw, 1), (db, 2)):
        for i in range(0, grad.numel(), 7):
            lo, hi = [x.double(), w.double(), b.double()], [x.double(), w.double(), b.double()]
            lo[args] = lo[args].clone()
            hi[args] = hi[args].clone()
            lo[args].view(-1)[i] -= h
            hi[args].view(-1)[i] += h
            # fp32 results of unit-sized terms, and h^2 times a third derivative below ~100
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - grad.view(-1)[i].item()) < 2e-5


def test_layer_norm_backward_empty(api):
    w = torch.ones(64, device="cuda")
    z = torch.empty(0, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    dx, dw, db = api.layer_norm_backward(e, e, w, z, z)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = api.layer_norm_backward(e, api.checkpoint8(e), w, z, z)
    assert (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------------------ linear
# one tile, ragged tiles, CTA pairs, K slices, single tokens
LINEAR = [(1, 8, 8), (3, 64, 40), (33, 768, 2304), (129, 72, 264), (257, 1000, 520), (300, 2048, 768), (1, 4096, 1024),
          (2048, 2048, 2048), (700, 4096, 1536), (2500, 512, 4104), (4001, 1536, 1544), (64, 14336, 256)]


def _z_tol(x, w, z):
    k = x.shape[1]
    return (k / 16 + 20) * R.TC * (x.double().abs() @ w.double().abs().t()) + 4 * R.TC * z.abs()


def _lipschitz(z, act):
    return 2 * z.abs() + 0.01 if act == "relu2" else torch.full_like(z, 1.13)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,m", LINEAR)
def test_linear(api, rows, n, m, dt):
    g = _gen(rows + n + m)
    t = DT[dt]
    x, w = _randn(g, rows, n, dtype=t), _randn(g, m, n, std=n ** -0.5, dtype=t)
    b = _randn(g, m) if rows % 2 else _randn(g, m, dtype=t)
    res = _randn(g, rows, m, dtype=t)
    z = x.double() @ w.double().t() + b.double()
    tol = _z_tol(x, w, z)
    for i, act in enumerate(R.ACTS):
        strided = i == 1
        keep = (False, True, "tensor")[i % 3]
        y, kept = api.linear(_strided(x) if strided else x, w, b, act=act, residual=_strided(res) if strided else
                             (res if i % 2 else None), checkpoint=keep)
        want = R.act(z, act) + (res.double() if i % 2 else 0)
        R.close(y, want, R.HALF_STEP[t] * want.abs() * 1.01 + tol * _lipschitz(z, act) +
                (16 + 6 * z.abs()) * R.TC * z.abs() * (1 + z.abs()) + 2.0 ** -25, f"y {act}")
        if keep is True:
            # a value is off by half a step of its block, a whole one where q is limited, and the sums' own error
            step = torch.exp2(kept.e.double() - 127).repeat_interleave(32, 1)[:, :m]
            lim = kept.q[:, :m].abs() == 127
            R.close(kept.restore(dtype=torch.float32), z, step * torch.where(lim, 1.0, 0.5) + tol, "z in 8 bits")
            amax = torch.zeros((rows, kept.e.shape[1] * 32), dtype=torch.float64, device="cuda")
            amax[:, :m] = z.abs()
            amax = amax.view(rows, -1, 32).amax(2)
            assert ((torch.log2(amax) + 121 - kept.e.double()).abs() < 1.001).all()  # e = floor(log2 amax) + 121
            if m % 32:
                assert (kept.q[:, m:] == 0).all()
        elif keep == "tensor":
            R.close(kept, z, R.HALF_STEP[t] * z.abs() * 1.01 + tol + 2.0 ** -25, "z")
    y, kept = api.linear(x, w)
    want = x.double() @ w.double().t()
    R.close(y, want, R.HALF_STEP[t] * want.abs() * 1.01 + tol + 2.0 ** -25, "y plain")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,m", LINEAR)
def test_linear_backward(api, rows, n, m, dt):
    g = _gen(rows + 2 * n + m)
    t = DT[dt]
    u = R.HALF_STEP[t]
    x, w = _randn(g, rows, n, dtype=t), _randn(g, m, n, std=n ** -0.5, dtype=t)
    dy, z = _randn(g, rows, m, dtype=t), _randn(g, rows, m, std=1.5, dtype=t)
    xk, zk = api.checkpoint8(x), api.checkpoint8(z)
    start = _randn(g, m, n)
    for i, act in enumerate(R.ACTS):
        kept = i % 2 == 1
        xv = R.unpack(xk.q, xk.e, n) if kept else x.double()
        zv = R.unpack(zk.q, zk.e, m) if kept else z.double()
        dz = dy.double() * R.slope(zv, act)
        f32 = i != 2
        acc = i in (0, 3)
        dw_in = start.clone() if acc else None
        dx, dw, db = api.linear_backward(_strided(dy) if i == 4 else dy, xk if kept else (_strided(x) if i == 4 else x), w,
                                         z=None if act == "none" else (zk if kept else z), act=act, dw=dw_in,
                                         accumulate=acc, dw_dtype=torch.float32 if f32 else t)
        # dz: rounded to t where there is an activation; the slope's own evaluation in fp32
        es = (16 + 6 * zv.abs()) * R.TC * (1 + zv.abs()) ** 2 * dy.double().abs()
        ez = es + (u * dz.abs() * 1.01 + 2.0 ** -25 if act != "none" else 0)
        adz = dz.abs() + ez
        want = dz @ w.double()
        aw = w.double().abs()
        R.close(dx, want, u * want.abs() * 1.01 + ez @ aw + (m / 16 + 20) * R.TC * (adz @ aw) + 2.0 ** -25, f"dx {act}")
        want = dz.t() @ xv + (start.double() if acc else 0)
        ax = xv.abs()
        # fp32: at most 64 truncating adds per 1024 of K, then rounded adds
        steps = min(rows / 16, 64) + 20 + rows / 1024
        tol = ez.t() @ ax + (steps if f32 else rows / 16 + 20) * R.TC * (adz.t() @ ax)
        tol = tol + (4 * R.F32 * want.abs() if f32 else u * want.abs() * 1.01 + 2.0 ** -25)
        if acc:
            tol = tol + R.F32 * start.double().abs()
            assert dw.data_ptr() == dw_in.data_ptr()
        R.close(dw, want, tol, f"dw {act}")
        R.close(db, dz.sum(0), (rows / 64 + 900 + 16) * R.F32 * dz.abs().sum(0) + es.sum(0), f"db {act}")


def test_linear_backward_parts(api):
    """Each output alone is what it is among the others.  The products of a call share a launch,
    and how K is cut depends on all of them, so sums may be joined in another order: each of the
    two results is off by at most (K / 16 + 20) truncated adds of the sum of magnitudes (db: its
    chain of adds), and dx is rounded to bf16 after that, which may move it by a step."""
    g = _gen(2)
    x, w = _randn(g, 200, 256, dtype=torch.bfloat16), _randn(g, 512, 256, std=0.06, dtype=torch.bfloat16)
    dy, z = _randn(g, 200, 512, dtype=torch.bfloat16), _randn(g, 200, 512, dtype=torch.bfloat16)
    dx, dw, db = api.linear_backward(dy, x, w, z=z, act="silu")
    dz = (dy.double() * R.slope(z.double(), "silu")).abs() * (1 + R.HALF_STEP[torch.bfloat16])
    tol = (2 * (512 / 16 + 20) * R.TC * (dz @ w.double().abs()) + 2 * 1.01 * R.HALF_STEP[torch.bfloat16] * dx.double().abs(),
           2 * (200 / 16 + 20) * R.TC * (dz.t() @ x.double().abs()), 2 * 216 * R.F32 * dz.sum(0))
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        got = api.linear_backward(dy, x, w, z=z, act="silu", need_dx=need[0], need_dw=need[1], need_db=need[2])
        for a, b, n, t in zip(got, (dx, dw, db), need, tol):
            if n:
                R.close(a, b, t, "alone")
            else:
                assert a is None


def test_linear_empty(api):
    w = torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
    e, dy = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    y, kept = api.linear(e, w, checkpoint=True, act="gelu")
    assert y.shape == (0, 16) and kept.shape == (0, 16)
    for x in (e, api.checkpoint8(e)):
        dx, dw, db = api.linear_backward(dy, x, w, z=kept, act="gelu")
        assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    G = torch.full((16, 64), 3.0, device="cuda")
    api.linear_backward(dy, e, w, dw=G, accumulate=True)
    assert (G == 3.0).all()


def test_linear_nonfinite_rows(api):
    """A NaN or an infinity in one token's row stays in that token's outputs."""
    g = _gen(8)
    x, w = _randn(g, 70, 200, dtype=torch.bfloat16), _randn(g, 328, 200, std=0.1, dtype=torch.bfloat16)
    clean, ck = api.linear(x, w, act="silu", checkpoint=True)
    x2 = x.clone()
    x2[3, 7], x2[69, 199] = math.nan, math.inf
    y, kept = api.linear(x2, w, act="silu", checkpoint=True)
    ok = torch.ones(70, dtype=torch.bool, device="cuda")
    ok[[3, 69]] = False
    assert torch.equal(y[ok], clean[ok]) and torch.equal(kept.q[ok], ck.q[ok]) and torch.equal(kept.e[ok], ck.e[ok])
    assert torch.isnan(y[3]).all() and torch.isnan(kept.restore()[[3, 69]]).all()


def test_rows_behind_the_last_are_untouched(api):
    """The C entry points on buffers with room behind: nothing there changes."""
    import ctypes

    from matrix_aware_optimizers_02_b200 import _lib as L
    lib = L.load()
    g = _gen(4)
    rows, n, m = 37, 72, 136
    x, w = _randn(g, rows, n, dtype=torch.float16), _randn(g, m, n, dtype=torch.float16)
    y = torch.full((rows + 200, m + 8), 5.0, dtype=torch.float16, device="cuda")
    q = torch.full((rows + 200, 160), 9, dtype=torch.int8, device="cuda")
    e = torch.full((rows + 200, 6), 9, dtype=torch.uint8, device="cuda")
    a = L.LinearArgs(rows, n, m, L.MAO_F16, x.data_ptr(), n, w.data_ptr(), None, 0, 0, None, 0, y.data_ptr(), m + 8, None,
                     0, L.Ckpt8(q.data_ptr(), e.data_ptr(), 160, 6))
    nb = ctypes.c_size_t(0)
    L.check(lib.mao_linear_workspace_size(ctypes.byref(a), ctypes.byref(nb)))
    ws = torch.empty(nb.value + 256, dtype=torch.uint8, device="cuda")
    L.check(lib.mao_linear(ctypes.byref(a), ws.data_ptr(), nb.value, torch.cuda.current_stream().cuda_stream))
    assert (y[rows:] == 5).all() and (y[:, m:] == 5).all() and (q[rows:] == 9).all() and (e[rows:] == 9).all()
    assert (e[:, 5] == 9).all()
    want, kept = api.linear(x, w, checkpoint=True)
    assert torch.equal(y[:rows, :m], want) and torch.equal(q[:rows], kept.q) and torch.equal(e[:rows, :5], kept.e)


def test_repeat_stream_and_graph(api):
    """The same bits on a second run, on a side stream, and in a replayed graph; two graphs
    captured apart keep apart."""
    g = _gen(6)
    t = torch.bfloat16
    x, w = _randn(g, 500, 768, dtype=t), _randn(g, 768, 768, std=0.04, dtype=t)
    lw, lb = torch.ones(768, device="cuda"), torch.zeros(768, device="cuda")
    dy = _randn(g, 500, 768, dtype=t)

    def step(x):
        h, mean, rstd, hk = api.layer_norm(x, lw, lb, checkpoint=True)
        y, zk = api.linear(h, w, act="gelu", checkpoint=True)
        dh, dw, db = api.linear_backward(dy, hk, w, z=zk, act="gelu")
        dx, dlw, dlb = api.layer_norm_backward(dh, x, lw, mean, rstd, dres=dy)
        return y, dw, db, dx, dlw, dlb

    want = step(x)
    assert all(torch.equal(a, b) for a, b in zip(step(x), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x2 = _randn(g, 500, 768, dtype=t)
    want2 = step(x2)
    xs = [x.clone(), x2.clone()]
    graphs, outs = [], []
    for v in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(v))
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))
    assert all(torch.equal(a, b) for a, b in zip(outs[1], want2))
    xs[0].copy_(x2)
    graphs[0].replay()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want2))


# ------------------------------------------------------------------ the layers and the step together
def test_block_gradient_and_step(api):
    """A norm and two linear layers with 8-bit checkpoints: gradients against the same block in
    64 bits on the kept values, then a Muon step on the G that the backward pass wrote."""
    import numpy as np

    from oracle import mao_oracle as O
    g = _gen(21)
    t = torch.bfloat16
    T, d, f = 333, 256, 640
    x = _randn(g, T, d, dtype=t)
    W1, W2 = _randn(g, f, d, std=d ** -0.5), _randn(g, d, f, std=f ** -0.5)
    G1, G2 = torch.empty_like(W1), torch.zeros_like(W2)
    M1, M2 = torch.zeros_like(W1), torch.zeros_like(W2)
    b1, b2 = _randn(g, f, std=0.1), _randn(g, d, std=0.1)
    lw, lb = 1 + _randn(g, d, std=0.1), _randn(g, d, std=0.1)
    dy = _randn(g, T, d, std=0.1, dtype=t)
    w1, w2 = W1.to(t), W2.to(t)
    muon = api.MuonBatch([(W1, G1, M1), (W2, G2, M2)], mu=0.95, lr=0.02)

    h, mean, rstd, hk = api.layer_norm(x, lw, lb, checkpoint=True)
    a, zk = api.linear(h, w1, b1, act="gelu", checkpoint=True)
    y, _ = api.linear(a, w2, b2, residual=x)
    da, _, db2 = api.linear_backward(dy, zk.restore(act="gelu"), w2, dw=G2, accumulate=True)
    dh, _, db1 = api.linear_backward(da, hk, w1, z=zk, act="gelu", dw=G1)
    dx, dlw, dlb = api.layer_norm_backward(dh, x, lw, mean, rstd, dres=dy)

    # 64 bits, from what each call was given: the stored intermediates h, a, z, da, dh
    D = torch.float64
    zv, hv = R.unpack(zk.q, zk.e, f), R.unpack(hk.q, hk.e, d)
    u = R.HALF_STEP[t]
    want = a.to(D) @ w2.to(D).t() + b2.to(D) + x.to(D)
    R.close(y, want, u * want.abs() * 1.01 + 64 * R.TC * (a.to(D).abs() @ w2.to(D).abs().t() + 1), "y")
    av = zk.restore(act="gelu").to(D)
    R.close(G2, dy.to(D).t() @ av, 96 * R.TC * (dy.to(D).abs().t() @ av.abs()), "G2")
    R.close(db2, dy.to(D).sum(0), 1024 * R.F32 * dy.to(D).abs().sum(0), "db2")
    dz = da.to(D) * R.slope(zv, "gelu")
    ez = u * dz.abs() * 1.01 + 64 * R.TC * da.to(D).abs() * (1 + zv.abs()) ** 2
    R.close(G1, dz.t() @ hv, (ez + 96 * R.TC * dz.abs()).t() @ hv.abs(), "G1")
    want = dz @ w1.to(D)
    R.close(dh, want, u * want.abs() * 1.01 + (ez + 96 * R.TC * dz.abs()) @ w1.to(D).abs(), "dh")
    want = R.layer_norm_backward(dh, x, lw, mean, rstd, dy)
    R.close(dx, want[0], u * want[0].abs() * 1.01 + 512 * R.F32 * (dy.to(D).abs() + dh.to(D).abs() * 8 + 1), "dx")

    # against the same block without 8-bit checkpoints: the kept values are off by half a step of 2^-7 of
    # their block's largest magnitude, a relative error of a few 2^-8 in the gradients' norm
    hd = R.layer_norm(x, lw, lb, 1e-5)[0]
    zd = hd @ w1.to(D).t() + b1.to(D)
    dad = dy.to(D) @ w2.to(D)
    G1d, G2d = (dad * R.slope(zd, "gelu")).t() @ hd, dy.to(D).t() @ R.act(zd, "gelu")
    for G, Gd in ((G1, G1d), (G2, G2d)):
        assert (G.to(D) - Gd).norm() / Gd.norm() < 0.03

    hostW = [W.double().cpu().numpy() for W in (W1, W2)]
    hostG = [G.double().cpu().numpy() for G in (G1, G2)]
    muon()
    assert muon.device_status() == 0
    for W, W0, G in zip((W1, W2), hostW, hostG):
        ref = O.muon_step(W0, G, np.zeros_like(G), mu=0.95, lr=0.02)[0] - W0
        got = W.double().cpu().numpy() - W0
        assert np.linalg.norm(got - ref) / np.linalg.norm(ref) < 2e-2


def test_linear_gradient_against_differences(api):
    """dW, dx and db of sum(dy * y) by central differences of the definition."""
    g = _gen(31)
    t = torch.float16
    x, w = _randn(g, 5, 24, dtype=t), _randn(g, 16, 24, std=0.3, dtype=t)
    b = _randn(g, 16)
    dy = _randn(g, 5, 16, dtype=t)
    for act in ("gelu", "gelu_tanh", "silu"):
        y, z = api.linear(x, w, b, act=act, checkpoint="tensor")
        dx, dw, db = api.linear_backward(dy, x, w, z=z, act=act)

        def loss(x, w, b):
            return (R.act(x @ w.t() + b, act) * dy.double()).sum().item()

        base = [x.double(), w.double(), b.double()]
        for k, grad in enumerate((dx, dw, db)):
            for i in range(0, grad.numel(), 11):
                lo, hi = list(base), list(base)
                lo[k], hi[k] = lo[k].clone(), hi[k].clone()
                lo[k].view(-1)[i] -= 1e-5
                hi[k].view(-1)[i] += 1e-5
                d = (loss(*hi) - loss(*lo)) / 2e-5
                # fp16 z (2^-11 |z|, |z| < 8, slope' < 1.2) and fp16 dz in sums of up to 24 products below ~2 each
                assert abs(d - grad.view(-1)[i].item()) < 0.05

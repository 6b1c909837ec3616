"""The trained-layer operators where calls go wrong: two streams at once, a first call inside a
graph capture, buffers with room around them, more than 2^31 elements, unusual checkpoints, the
binding's refusals, and the device status."""

import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

from matrix_aware_optimizers_02_b200 import _lib as L
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def _stream():
    return torch.cuda.current_stream().cuda_stream


def test_two_streams_at_once(api):
    """The same bits from two streams that run at the same time, both with K slices and workspaces."""
    t = torch.bfloat16
    work = []
    for seed, (rows, n, m) in ((1, (640, 4096, 256)), (2, (300, 2048, 768))):
        g = _gen(seed)
        x, w = _randn(g, rows, n, dtype=t), _randn(g, m, n, std=n ** -0.5, dtype=t)
        dy, lw = _randn(g, rows, m, dtype=t), torch.ones(n, device="cuda")

        def step(x=x, w=w, dy=dy, lw=lw):
            h, mean, rstd, hk = api.layer_norm(x, lw, checkpoint=True)
            y, zk = api.linear(h, w, act="silu", checkpoint=True)
            dh, dw, db = api.linear_backward(dy, hk, w, z=zk, act="silu")
            return (y, dw, db) + tuple(api.layer_norm_backward(dh, x, lw, mean, rstd))

        work.append((step, step()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(work[i][0]())
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, work[i][1]))


_FIRST_IN_CAPTURE = """
import torch
from matrix_aware_optimizers_02_b200 import api
torch.manual_seed(0)
t = torch.bfloat16
x, w = torch.randn(200, 512, device="cuda").to(t), (torch.randn(384, 512, device="cuda") * 0.05).to(t)
dy, lw = torch.randn(200, 384, device="cuda").to(t), torch.ones(512, device="cuda")
def step():
    h, mean, rstd, hk = api.layer_norm(x, lw, checkpoint=True)
    y, zk = api.linear(h, w, act="gelu", checkpoint=True)
    dh, dw, db = api.linear_backward(dy, hk, w, z=zk, act="gelu")
    return (y, dw, db, hk.restore(act="relu")) + tuple(api.layer_norm_backward(dh, api.checkpoint8(x), lw, mean, rstd))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
want = step()
assert all(torch.equal(a, b) for a, b in zip(out, want))
assert api.layer_status() == (0, 0)
print("captured ok")
"""


def test_first_call_inside_a_capture(api):
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr


def _framed(rows, cols, dtype, value):
    """rows x cols inside a larger buffer of one value: (buffer, pointer, leading dimension)."""
    ld = cols + 24
    buf = torch.full((rows + 300, ld), value, dtype=dtype, device="cuda")
    return buf, buf[100:, 8:].data_ptr() if dtype != torch.uint8 else buf[100:].data_ptr(), ld


def _check_frame(buf, rows, cols, value, left=8):
    inner = torch.zeros_like(buf, dtype=torch.bool)
    inner[100:100 + rows, left:left + cols] = True
    assert (buf[~inner] == value).all()
    return buf[100:100 + rows, left:left + cols]


@pytest.mark.parametrize("rows,cols", [(1, 8), (37, 264), (130, 4104), (5, 9000)])
def test_only_the_matrix_is_written(api, rows, cols):
    """Norm, its gradient and the checkpoint passes on buffers with room on every side."""
    lib = L.load()
    g = _gen(rows)
    t, dt = torch.bfloat16, L.MAO_BF16
    x, dy = _randn(g, rows, cols, dtype=t), _randn(g, rows, cols, dtype=t)
    w = 1 + _randn(g, cols, std=0.1)
    y, yp, ld = _framed(rows, cols, t, 3.0)
    blocks = (cols + 31) // 32
    q = torch.full((rows + 300, blocks * 32 + 64), 77, dtype=torch.int8, device="cuda")
    e = torch.full((rows + 300, blocks + 3), 77, dtype=torch.uint8, device="cuda")
    k = L.Ckpt8(q[100:, 32:].data_ptr(), e[100:, 1:].data_ptr(), q.shape[1], e.shape[1])
    st = torch.full((2, rows + 20), 9.0, device="cuda")
    a = L.LayerNormArgs(rows, cols, dt, L.MAO_F32, x.data_ptr(), cols, w.data_ptr(), None, 1e-5, yp, ld,
                        st[0, 5:].data_ptr(), st[1, 5:].data_ptr(), k)
    L.check(lib.mao_layer_norm(ctypes.byref(a), _stream()))
    want, mean, rstd, kept = api.layer_norm(x, w, checkpoint=True)
    assert torch.equal(_check_frame(y, rows, cols, 3.0), want)
    assert torch.equal(_check_frame(q, rows, blocks * 32, 77, 32), kept.q)
    assert torch.equal(_check_frame(e, rows, blocks, 77, 1), kept.e)
    assert torch.equal(st[0, 5:5 + rows], mean) and torch.equal(st[1, 5:5 + rows], rstd)
    assert (st[:, :5] == 9).all() and (st[:, 5 + rows:] == 9).all()

    out, op, ld_o = _framed(rows, cols, t, 3.0)
    L.check(lib.mao_checkpoint8_restore(ctypes.byref(k), rows, cols, 1, op, dt, ld_o, _stream()))
    assert torch.equal(_check_frame(out, rows, cols, 3.0), kept.restore(act="relu"))
    q.fill_(77), e.fill_(77)
    L.check(lib.mao_checkpoint8(yp, dt, rows, cols, ld, ctypes.byref(k), _stream()))
    assert torch.equal(_check_frame(q, rows, blocks * 32, 77, 32), kept.q)
    assert torch.equal(_check_frame(e, rows, blocks, 77, 1), kept.e)

    dx, dxp, ld_dx = _framed(rows, cols, t, 3.0)
    sums = torch.full((2, cols + 16), 9.0, device="cuda")
    b = L.LayerNormBackwardArgs(rows, cols, dt, L.MAO_F32, dy.data_ptr(), cols, None, 0, k, w.data_ptr(), mean.data_ptr(),
                                rstd.data_ptr(), yp, ld, dxp, ld_dx, sums[0, 8:].data_ptr(), sums[1, 8:].data_ptr())
    nb = ctypes.c_size_t(0)
    L.check(lib.mao_layer_norm_backward_workspace_size(ctypes.byref(b), ctypes.byref(nb)))
    ws = torch.full((nb.value + 512,), 5, dtype=torch.uint8, device="cuda")
    L.check(lib.mao_layer_norm_backward(ctypes.byref(b), ws.data_ptr(), nb.value, _stream()))
    want = api.layer_norm_backward(dy, kept, w, mean, rstd, dres=y[100:100 + rows, 8:8 + cols].contiguous())
    assert torch.equal(_check_frame(dx, rows, cols, 3.0), want[0])
    assert torch.equal(sums[0, 8:8 + cols], want[1]) and torch.equal(sums[1, 8:8 + cols], want[2])
    assert (sums[:, :8] == 9).all() and (sums[:, 8 + cols:] == 9).all() and (ws[nb.value:] == 5).all()


def test_linear_backward_writes_only_its_outputs(api):
    lib = L.load()
    g = _gen(3)
    t, dt = torch.float16, L.MAO_F16
    rows, n, m = 77, 200, 136
    x, dy, z = _randn(g, rows, n, dtype=t), _randn(g, rows, m, dtype=t), _randn(g, rows, m, dtype=t)
    w = _randn(g, m, n, std=0.1, dtype=t)
    dx, dxp, ld_dx = _framed(rows, n, t, 3.0)
    dw = torch.full((m + 4, n), 9.0, device="cuda")
    db = torch.full((m + 8,), 9.0, device="cuda")
    no = L.Ckpt8(None, None, 0, 0)
    a = L.LinearBackwardArgs(rows, n, m, dt, dy.data_ptr(), m, x.data_ptr(), n, no, w.data_ptr(), L.ACTIVATIONS["gelu"],
                             z.data_ptr(), m, no, dxp, ld_dx, dw[2:].data_ptr(), L.MAO_F32, 0, db[4:].data_ptr())
    nb = ctypes.c_size_t(0)
    L.check(lib.mao_linear_backward_workspace_size(ctypes.byref(a), ctypes.byref(nb)))
    ws = torch.full((nb.value + 512,), 5, dtype=torch.uint8, device="cuda")
    L.check(lib.mao_linear_backward(ctypes.byref(a), ws.data_ptr(), nb.value, _stream()))
    want = api.linear_backward(dy, x, w, z=z, act="gelu")
    assert torch.equal(_check_frame(dx, rows, n, 3.0), want[0])
    assert torch.equal(dw[2:2 + m], want[1]) and (dw[:2] == 9).all() and (dw[2 + m:] == 9).all()
    assert torch.equal(db[4:4 + m], want[2]) and (db[:4] == 9).all() and (db[4 + m:] == 9).all()
    assert (ws[nb.value:] == 5).all()


def test_more_than_2_31_elements(api):
    """Rows whose elements lie past 32-bit offsets: the last ones are what they are alone."""
    rows, cols, last = 270000, 8192, 40  # 2.2e9 elements
    t = torch.bfloat16
    g = _gen(1)
    tail = _randn(g, last, cols, dtype=t)
    x = torch.zeros((rows, cols), dtype=t, device="cuda")
    x[-last:] = tail
    w = torch.ones(cols, device="cuda")
    y, mean, rstd, kept = api.layer_norm(x, w, checkpoint=True)
    y1, mean1, rstd1, kept1 = api.layer_norm(tail, w, checkpoint=True)
    assert torch.equal(y[-last:], y1) and torch.equal(mean[-last:], mean1) and torch.equal(rstd[-last:], rstd1)
    assert torch.equal(kept.q[-last:], kept1.q) and torch.equal(kept.e[-last:], kept1.e) and (y[:-last] == 0).all()
    del y
    back = kept.restore()
    assert torch.equal(back[-last:], kept1.restore())
    del back
    k = api.checkpoint8(x)
    assert torch.equal(k.q[-last:], api.checkpoint8(tail).q)
    del k
    # the gradient of x itself: 0 for all but the last rows' share
    dx, dw, db = api.layer_norm_backward(x, kept, w, mean, rstd)
    dx1, _, _ = api.layer_norm_backward(tail, kept1, w, mean1, rstd1)
    assert torch.equal(dx[-last:], dx1)
    R.close(db, tail.double().sum(0), 700 * R.F32 * tail.double().abs().sum(0), "db")
    del dx
    W = _randn(g, 16, cols, std=0.01, dtype=t)
    y, _ = api.linear(x, W)
    R.close(y[-last:], api.linear(tail, W)[0], 2.02 * R.HALF_STEP[t] * (tail.double() @ W.double().t()).abs() +
            (cols / 8 + 40) * R.TC * (tail.double().abs() @ W.double().abs().t()), "y")
    assert (y[:-last] == 0).all()
    dy = torch.zeros((rows, 16), dtype=t, device="cuda")
    dy[-last:] = _randn(g, last, 16, dtype=t)
    dx, dw, db = api.linear_backward(dy, x, W)
    d = dy[-last:].double()
    R.close(dw, d.t() @ tail.double(), 100 * R.TC * (d.abs().t() @ tail.double().abs()), "dw")
    want = d @ W.double()
    R.close(dx[-last:], want, 1.01 * R.HALF_STEP[t] * want.abs() + 32 * R.TC * (d.abs() @ W.double().abs()), "dx")
    assert (dx[:-last] == 0).all()


def test_checkpoints_made_elsewhere(api):
    """Bytes that the library itself does not write: e = 0 is zeros, 255 is NaN, and the largest
    steps, where the value may pass the type's range."""
    q = torch.tensor([[127, -128, 1, -1] * 8] * 4, dtype=torch.int8, device="cuda")
    e = torch.tensor([[0], [255], [247], [100]], dtype=torch.uint8, device="cuda")
    k = api.Checkpoint8(q, e, 32, torch.float32)
    v = k.restore()
    want = R.unpack(q, e, 32)
    assert (v[0] == 0).all() and torch.isnan(v[1]).all()
    assert torch.equal(v[2:].double(), want[2:])
    assert torch.equal(k.restore(dtype=torch.bfloat16)[2:].double(), want[2:])
    # the norm's gradient and the linear layer's read them the same way
    w, one = torch.ones(32, device="cuda"), torch.ones(4, device="cuda")
    dy = torch.ones((4, 32), dtype=torch.bfloat16, device="cuda")
    kb = api.Checkpoint8(q, e, 32, torch.bfloat16)
    a = api.layer_norm_backward(dy, kb, w, one, one)[0]
    b = api.layer_norm_backward(dy, kb.restore(), w, one, one)[0]
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


def test_binding_refusals(api):
    t = torch.bfloat16
    x, w = torch.zeros((4, 64), dtype=t, device="cuda"), torch.zeros((32, 64), dtype=t, device="cuda")
    dy, lw = torch.zeros((4, 32), dtype=t, device="cuda"), torch.ones(64, device="cuda")
    st = torch.zeros(4, device="cuda")
    k = api.checkpoint8(x)
    bad = [
        lambda: api.linear(x.float(), w.float()), lambda: api.linear(x, w.half()), lambda: api.linear(x[:, :40], w),
        lambda: api.linear(x, w.t()), lambda: api.linear(x.view(2, 2, 64), w), lambda: api.linear(x, w, act="tanh"),
        lambda: api.linear(x, w, torch.zeros(33, device="cuda")), lambda: api.linear(x, w, residual=x),
        lambda: api.linear(x, w, checkpoint="yes"), lambda: api.linear(x[:, 1:41], w[:, 1:41]),
        lambda: api.linear_backward(dy, x, w, act="gelu"), lambda: api.linear_backward(dy, x[:3], w),
        lambda: api.linear_backward(dy, k, w[:, :40].contiguous()), lambda: api.linear_backward(dy, x, w, accumulate=True),
        lambda: api.linear_backward(dy, x, w, dw=torch.zeros_like(w), accumulate=True),
        lambda: api.linear_backward(dy, x, w, dw=torch.zeros((64, 32), device="cuda")),
        lambda: api.linear_backward(dy, x, w, dw_dtype=torch.float16),
        lambda: api.linear_backward(dy, x, w, dw=torch.zeros((32, 64), device="cuda"), need_dw=False),
        lambda: api.layer_norm(x, lw.half()), lambda: api.layer_norm(x, lw, lw.to(t)), lambda: api.layer_norm(x, lw[:32]),
        lambda: api.layer_norm(x.double(), lw), lambda: api.layer_norm_backward(x, x, lw, st[:3], st),
        lambda: api.layer_norm_backward(x, x.float(), lw, st, st), lambda: api.layer_norm_backward(x, x, lw, st.half(), st),
        lambda: api.checkpoint8(x.double()), lambda: api.checkpoint8(x[:, :12]), lambda: api.checkpoint8(x.t()),
        lambda: k.restore(act="swish"), lambda: k.restore(dtype=torch.float64),
        lambda: api.Checkpoint8(k.q[:, :32], k.e, 64, t), lambda: api.Checkpoint8(k.q, k.e.int(), 64, t),
        lambda: api.linear(x, w.cpu()), lambda: api.linear_backward(dy, "x", w),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    # misaligned storage is the library's to refuse
    flat = torch.zeros(4 * 64 + 1, dtype=t, device="cuda")
    with pytest.raises(L.MaoError) as err:
        api.checkpoint8(flat[1:].view(4, 64))
    assert err.value.status == L.MAO_ERR_ALIGN
    with pytest.raises(L.MaoError) as err:
        api.layer_norm(torch.zeros((2, L.LAYER_NORM_MAX_COLS + 8), device="cuda"),
                       torch.ones(L.LAYER_NORM_MAX_COLS + 8, device="cuda"))
    assert err.value.status == L.MAO_ERR_UNSUPPORTED
    p = torch.nn.Parameter(w.clone())
    with pytest.raises(ValueError, match="requires grad"):
        api.linear(x, p)
    with torch.no_grad():
        api.linear(x, p)
    assert torch.equal(x, torch.zeros_like(x))


def test_status_reads_and_clears(api):
    lib = L.load()
    where = ctypes.c_int32(5)
    assert lib.mao_layer_status(_stream(), ctypes.byref(where)) == 0 and where.value == 0
    assert lib.mao_layer_status(None, None) == 0


@pytest.mark.parametrize("act", R.ACTS)
def test_activations_far_out(api, act):
    """Values far in the tails and at the ends of the range, through both passes."""
    t = torch.bfloat16
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 6.0, -6.0, 12.0, -12.0, 40.0, -40.0, 88.0, -88.0, 200.0, -200.0],
                     device="cuda").repeat(2).view(1, 32).to(t)
    dy = torch.ones((1, 32), dtype=t, device="cuda")
    eye = torch.eye(32, dtype=t, device="cuda")
    y, kept = api.linear(z, eye, act=act, checkpoint="tensor")
    assert torch.equal(kept, z)
    zd = z.double()
    want = R.act(zd, act)
    # below 2^-126 a reciprocal or an exponential is flushed to 0: off by at most |z| 2^-125
    flush = zd.abs() * 2.0 ** -125
    tail = torch.exp(-zd.clamp(max=0).abs() / 2)  # the activations fall off at least this fast
    R.close(y, want, 1.01 * R.HALF_STEP[t] * want.abs() + 2e-6 * (1 + zd.abs()) * tail + flush, "y")
    dx, _, db = api.linear_backward(dy, z, eye, z=z, act=act)
    s = R.slope(zd, act)
    R.close(db, s[0], 4e-6 * (1 + zd[0].abs()) * tail[0] + 2 * R.F32 * s[0].abs() + flush[0], "slope")
    R.close(dx, s, 1.01 * R.HALF_STEP[t] * s.abs() + 4e-6 * (1 + zd.abs()), "dx")
    assert math.isfinite(float(dx.float().abs().max()))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("cols", [24, 264, 1032])
def test_norm_backward_of_a_huge_constant_row(api, cols, kept):
    """mean * rstd overflows, x - mean does not: lanes behind the last column must add nothing.

    h = 0, so dx = rstd (u - mean u) with u = dy w.  Sums of cols terms of size 1 in fp32 are off
    by cols 2^-24 at most, and dx is rounded to bf16 (2^-8 of its size)."""
    g = torch.Generator("cuda").manual_seed(cols)
    rows, rstd = 5, 316.0
    x = torch.full((rows, cols), 2.0**122, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    w = torch.randn(cols, device="cuda", generator=g)
    mean = torch.full((rows,), 2.0**122, device="cuda")
    dx, dw, db = api.layer_norm_backward(dy, api.checkpoint8(x) if kept else x, w, mean,
                                         torch.full((rows,), rstd, device="cuda"))
    u = dy.double() * w.double()
    want = rstd * (u - u.mean(1, keepdim=True))
    size = rstd * (u.abs() + u.abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= 2.0**-8 * want.abs() + (cols + 4) * 2.0**-23 * size).all()
    assert (dw == 0).all()
    assert ((db.double() - dy.double().sum(0)).abs() <= 8 * 2.0**-24 * dy.double().abs().sum(0)).all()

"""Refusals of the trained-layer entry points, checked before any GPU is touched (these run on
a machine without one: the calls use addresses that are never dereferenced)."""

import ctypes

import pytest
import torch

from matrix_aware_optimizers_02_b200 import _lib as L
from matrix_aware_optimizers_02_b200 import api

A16, MIS = 0x10000, 0x10004
NONE = L.Ckpt8(None, None, 0, 0)


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _set(args, **kw):
    for k, v in kw.items():
        setattr(args, k, v)
    return args


def test_checkpoint_refusals(lib):
    def call(x=A16, dtype=L.MAO_BF16, rows=4, cols=40, ld=40, q=A16, e=A16, ld_q=64, ld_e=2):
        return lib.mao_checkpoint8(x, dtype, rows, cols, ld, ctypes.byref(L.Ckpt8(q, e, ld_q, ld_e)), None)

    assert call(dtype=5) == L.MAO_ERR_DTYPE
    assert call(rows=-1) == L.MAO_ERR_SHAPE
    assert call(cols=0, ld=0) == L.MAO_ERR_SHAPE
    assert call(cols=36) == L.MAO_ERR_SHAPE
    assert call(ld=32) == L.MAO_ERR_SHAPE
    assert call(ld=44) == L.MAO_ERR_SHAPE
    assert call(ld_q=40) == L.MAO_ERR_SHAPE
    assert call(ld_q=32) == L.MAO_ERR_SHAPE
    assert call(ld_e=1) == L.MAO_ERR_SHAPE
    assert call(x=None) == L.MAO_ERR_INVALID_ARG
    assert call(q=None) == L.MAO_ERR_INVALID_ARG
    assert call(e=None) == L.MAO_ERR_INVALID_ARG
    assert call(x=MIS) == L.MAO_ERR_ALIGN
    assert call(q=MIS) == L.MAO_ERR_ALIGN
    assert lib.mao_checkpoint8(A16, L.MAO_F32, 4, 40, 40, None, None) == L.MAO_ERR_INVALID_ARG
    k = L.Ckpt8(A16, A16, 64, 2)
    assert lib.mao_checkpoint8_restore(ctypes.byref(k), 4, 40, 9, A16, L.MAO_BF16, 40, None) == L.MAO_ERR_INVALID_ARG
    assert lib.mao_checkpoint8_restore(ctypes.byref(k), 4, 40, 0, A16, 3, 40, None) == L.MAO_ERR_DTYPE
    assert lib.mao_checkpoint8_restore(ctypes.byref(k), 4, 40, 0, MIS, L.MAO_BF16, 40, None) == L.MAO_ERR_ALIGN
    assert lib.mao_checkpoint8_restore(ctypes.byref(k), 4, 40, 0, None, L.MAO_BF16, 40, None) == L.MAO_ERR_INVALID_ARG


def test_layer_norm_refusals(lib):
    def args(**kw):
        return _set(L.LayerNormArgs(4, 40, L.MAO_BF16, L.MAO_F32, A16, 40, A16, A16, 1e-5, A16, 40, A16, A16, NONE), **kw)

    def call(**kw):
        return lib.mao_layer_norm(ctypes.byref(args(**kw)), None)

    assert lib.mao_layer_norm(None, None) == L.MAO_ERR_INVALID_ARG
    assert call(dtype=4) == L.MAO_ERR_DTYPE
    assert call(w_dtype=L.MAO_F16) == L.MAO_ERR_DTYPE
    assert call(rows=-2) == L.MAO_ERR_SHAPE
    assert call(cols=44, ld_x=48, ld_y=48) == L.MAO_ERR_SHAPE
    assert call(cols=L.LAYER_NORM_MAX_COLS + 8, ld_x=40000, ld_y=40000) == L.MAO_ERR_UNSUPPORTED
    for name in ("x", "w", "y", "mean", "rstd"):
        assert call(**{name: None}) == L.MAO_ERR_INVALID_ARG, name
    for name in ("x", "w", "b", "y"):
        assert call(**{name: MIS}) == L.MAO_ERR_ALIGN, name
    assert call(eps=-1.0) == L.MAO_ERR_INVALID_ARG
    assert call(eps=float("nan")) == L.MAO_ERR_INVALID_ARG
    assert call(yc=L.Ckpt8(A16, A16, 32, 2)) == L.MAO_ERR_SHAPE
    assert call(yc=L.Ckpt8(A16, None, 64, 2)) == L.MAO_ERR_INVALID_ARG


def test_layer_norm_backward_refusals(lib):
    def call(ws=A16, ws_bytes=1 << 40, **kw):
        a = _set(L.LayerNormBackwardArgs(4, 40, L.MAO_BF16, L.MAO_F32, A16, 40, A16, 40, NONE, A16, A16, A16, None, 0,
                                         A16, 40, A16, A16), **kw)
        return lib.mao_layer_norm_backward(ctypes.byref(a), ws, ws_bytes, None)

    assert call(dtype=4) == L.MAO_ERR_DTYPE
    assert call(cols=42) == L.MAO_ERR_SHAPE
    for name in ("dy", "x", "w", "dx", "mean", "rstd"):
        assert call(**{name: None}) == L.MAO_ERR_INVALID_ARG, name
    assert call(x=None, xc=L.Ckpt8(A16, A16, 40, 2)) == L.MAO_ERR_SHAPE
    assert call(dres=A16, ld_dres=32) == L.MAO_ERR_SHAPE
    assert call(dres=MIS, ld_dres=40) == L.MAO_ERR_ALIGN
    assert call(ws=None) == L.MAO_ERR_WORKSPACE
    assert call(ws_bytes=100) == L.MAO_ERR_WORKSPACE
    assert call(ws=A16 + 16) == L.MAO_ERR_ALIGN
    n = ctypes.c_size_t(0)
    assert lib.mao_layer_norm_backward_workspace_size(None, ctypes.byref(n)) == L.MAO_ERR_INVALID_ARG


def _linear(**kw):
    return _set(L.LinearArgs(4, 40, 72, L.MAO_BF16, A16, 40, A16, A16, L.MAO_F32, 0, A16, 72, A16, 72, None, 0, NONE), **kw)


def test_linear_refusals(lib):
    def call(ws=A16, ws_bytes=1 << 40, **kw):
        return lib.mao_linear(ctypes.byref(_linear(**kw)), ws, ws_bytes, None)

    assert lib.mao_linear(None, None, 0, None) == L.MAO_ERR_INVALID_ARG
    assert call(dtype=L.MAO_F32) == L.MAO_ERR_DTYPE
    assert call(b_dtype=L.MAO_F16) == L.MAO_ERR_DTYPE
    assert call(n=44) == L.MAO_ERR_SHAPE
    assert call(m=0) == L.MAO_ERR_SHAPE
    assert call(rows=-1) == L.MAO_ERR_SHAPE
    assert call(act=6) == L.MAO_ERR_INVALID_ARG
    assert call(act=-1) == L.MAO_ERR_INVALID_ARG
    assert call(ld_x=36) == L.MAO_ERR_SHAPE
    assert call(ld_res=64) == L.MAO_ERR_SHAPE
    for name in ("x", "W", "y"):
        assert call(**{name: None}) == L.MAO_ERR_INVALID_ARG, name
    for name in ("x", "W", "b", "res", "y"):
        assert call(**{name: MIS}) == L.MAO_ERR_ALIGN, name
    assert call(z=MIS, ld_z=72) == L.MAO_ERR_ALIGN
    assert call(zc=L.Ckpt8(A16, A16, 72, 3)) == L.MAO_ERR_SHAPE
    assert call(rows=1 << 30, ld_x=1 << 20) == L.MAO_ERR_SHAPE  # past a tensor map's strides
    # a product cut into K slices needs its workspace
    n = ctypes.c_size_t(0)
    big = dict(rows=64, n=14336, m=256, ld_x=14336, ld_y=256, ld_res=256)
    L.check(lib.mao_linear_workspace_size(ctypes.byref(_linear(**big)), ctypes.byref(n)))
    assert n.value > 0
    assert call(ws=None, **big) == L.MAO_ERR_WORKSPACE
    assert call(ws_bytes=n.value - 1, **big) == L.MAO_ERR_WORKSPACE
    assert call(ws=A16 + 16, **big) == L.MAO_ERR_ALIGN


def test_linear_backward_refusals(lib):
    def call(ws=A16, ws_bytes=1 << 40, **kw):
        a = _set(L.LinearBackwardArgs(4, 40, 72, L.MAO_BF16, A16, 72, A16, 40, NONE, A16, 1, A16, 72, NONE, A16, 40, A16,
                                      L.MAO_F32, 0, A16), **kw)
        return lib.mao_linear_backward(ctypes.byref(a), ws, ws_bytes, None)

    assert call(dtype=L.MAO_F32) == L.MAO_ERR_DTYPE
    assert call(dw_dtype=L.MAO_F16) == L.MAO_ERR_DTYPE
    assert call(dw_dtype=L.MAO_BF16, accumulate=1) == L.MAO_ERR_DTYPE
    assert call(act=7) == L.MAO_ERR_INVALID_ARG
    for name in ("dy", "x", "W", "z"):
        assert call(**{name: None}) == L.MAO_ERR_INVALID_ARG, name
    for name in ("dy", "x", "W", "z", "dx", "dW", "db"):
        assert call(**{name: MIS}) == L.MAO_ERR_ALIGN, name
    assert call(x=None, xc=L.Ckpt8(A16, A16, 32, 2)) == L.MAO_ERR_SHAPE
    assert call(z=None, zc=L.Ckpt8(A16, A16, 96, 2)) == L.MAO_ERR_SHAPE
    assert call(ld_dx=32) == L.MAO_ERR_SHAPE
    assert call(ws=None) == L.MAO_ERR_WORKSPACE
    assert call(ws=A16 + 16) == L.MAO_ERR_ALIGN


def test_optimizer_gradients_stay_fp32_or_bf16(lib):
    """MAO_F16 is a type of the trained layers; the steps refuse it."""
    mats = (L.MuonMat * 1)(L.MuonMat(16, 32, A16, A16, L.MAO_F16, A16))
    p = L.MuonParams(0.95, 0.02, 0.0, 1e-7, 5, None, 0)
    assert lib.mao_muon_step(mats, 1, ctypes.byref(p), A16, 1 << 40, None, None) == L.MAO_ERR_DTYPE


def test_python_refuses_host_tensors_and_bad_names():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    w = torch.zeros((8, 16), dtype=torch.bfloat16)
    for call in (lambda: api.checkpoint8(x), lambda: api.layer_norm(x, torch.ones(16)), lambda: api.linear(x, w),
                 lambda: api.linear_backward(x, x, w), lambda: api.layer_norm_backward(x, x, x[0], x[0], x[0]),
                 lambda: api.Checkpoint8(torch.zeros((4, 32), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.uint8),
                                         16, torch.bfloat16)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        api.Checkpoint8(None, None, 16, torch.int32)
    with pytest.raises(ValueError):
        api.Checkpoint8(None, None, 12, torch.bfloat16)


@pytest.mark.parametrize("rows", [2**30 + 1, 2**31, 2**32 + 5])
def test_row_counts_past_the_limit_are_refused(monkeypatch, rows):
    """2^32 + 5 rows must not reach the C structs, whose 32-bit fields would make 5 of them."""
    from matrix_aware_optimizers_02_b200 import layers
    monkeypatch.setattr(layers, "_check", lambda *a, **k: None)
    x = torch.empty((rows, 8), dtype=torch.bfloat16, device="meta")
    for call in (lambda: layers.checkpoint8(x), lambda: layers.layer_norm(x, x), lambda: layers.linear(x, x),
                 lambda: layers.layer_norm_backward(x, x, x, x, x), lambda: layers.linear_backward(x, x, x)):
        with pytest.raises(ValueError, match="at most"):
            call()


def test_entry_points_refuse_sizes_past_the_limit(lib):
    big = 2**30 + 8
    k = L.Ckpt8(A16, A16, 32, 1)
    assert lib.mao_checkpoint8(A16, L.MAO_BF16, big, 8, 8, ctypes.byref(k), None) == L.MAO_ERR_SHAPE
    a = L.LinearArgs(4, 8, 8, L.MAO_BF16, A16, 8, A16, None, 0, 0, None, 0, A16, 8, None, 8, NONE)
    n = ctypes.c_size_t(0)
    assert lib.mao_linear_workspace_size(ctypes.byref(a), ctypes.byref(n)) == L.MAO_OK
    for kw in (dict(rows=big), dict(n=big), dict(m=big)):
        b = L.LinearArgs(*[getattr(a, f[0]) for f in a._fields_])
        assert lib.mao_linear_workspace_size(ctypes.byref(_set(b, **kw)), ctypes.byref(n)) == L.MAO_ERR_SHAPE

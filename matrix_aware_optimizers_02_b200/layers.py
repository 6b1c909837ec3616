"""The trained layers around a stepped weight matrix: layer norm, the linear layer, their
backward passes, and 8-bit checkpoints of activations that the backward passes read.

    from matrix_aware_optimizers_02_b200 import api
    h, mean, rstd, hk = api.layer_norm(x, w, b, checkpoint=True)      # hk: h in 8 bits
    a, zk = api.linear(h, W.bfloat16(), bias, act="gelu", checkpoint=True)
    ...
    dh, _, dbias = api.linear_backward(da, hk, W.bfloat16(), z=zk, act="gelu", dw=G)
    dx, dw, db = api.layer_norm_backward(dh, x, w, mean, rstd, dres=dy)
    muon()            # a MuonBatch built on (W, G, M)

Explicit forward / backward pairs: no autograd graph is recorded.  A tensor that requires
grad is refused while grad mode is on, one with a forward-mode tangent always.
Activations are 2-D CUDA tensors (a row per token) with contiguous rows of a multiple of 8
elements, 16-byte aligned; a row stride larger than the row is allowed.  Work runs on the
current stream of the tensors' device.  Outputs and scratch come from torch's allocator on
that stream; nothing is kept between calls.  Argument marshalling only; every arithmetic
step runs in the library's kernels.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch
from torch.autograd import forward_ad

from . import _lib as L

_DTYPES = {torch.float32: L.MAO_F32, torch.bfloat16: L.MAO_BF16, torch.float16: L.MAO_F16}
_HALF = (torch.bfloat16, torch.float16)
_MOST = 2**30
_NO_CKPT = L.Ckpt8(None, None, 0, 0)


def _has_tangent(t: torch.Tensor) -> bool:
    return torch._C._is_fwd_grad_enabled() and forward_ad.unpack_dual(t).tangent is not None


def _check(name: str, t: torch.Tensor, device=None, dtype=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: these calls record no graph (use torch.no_grad() or detach())")
    # no_grad leaves forward mode on; outside a dual level, which is nearly always, one comparison
    if getattr(forward_ad, "_current_level", 0) >= 0 and _has_tangent(t):
        raise ValueError(f"{name} carries a forward-mode tangent: these calls have none (use unpack_dual(...).primal)")


def _check_acts(name: str, t: torch.Tensor, shape=None, device=None, dtype=None) -> int:
    """Checks a matrix of activations and returns its leading dimension."""
    _check(name, t, device, dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D (tokens, features), got {tuple(t.shape)}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if cols % 8 or cols == 0:
        raise ValueError(f"{name} has {cols} columns: a positive multiple of 8 is needed")
    if max(rows, cols) > _MOST:  # above 32 bits the C structs' fields would cut it without an error
        raise ValueError(f"{name} has shape {tuple(t.shape)}: at most {_MOST} rows and columns")
    if rows > 1:
        ld = t.stride(0)
        if t.stride(1) != 1 or ld < cols or ld % 8:
            raise ValueError(f"{name} needs contiguous rows and a row stride that is a multiple of 8, got strides "
                             f"{t.stride()}")
        return ld
    if rows == 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs contiguous rows, got strides {t.stride()}")
    return cols


def _check_param(name: str, t: torch.Tensor, n: int, device, dtypes) -> None:
    _check(name, t, device)
    if tuple(t.shape) != (n,):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n,)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _act(name: str) -> int:
    if name not in L.ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(L.ACTIVATIONS)}")
    return L.ACTIVATIONS[name]


def _elsewhere(device) -> bool:
    """Whether the tensors' device is not the current one; such a call is made again with it current."""
    return device.index != torch.cuda.current_device()


def _stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same without building a Stream object: 0.1 against 2.2 us, of a call that takes about 10
# (a torch built without CUDA does not have it, and imports all the same)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class Checkpoint8:
    """A matrix of activations held in 8 bits: blocks of 32 columns with a power-of-two step.

    q: int8 (rows, 32 * ceil(cols / 32)); e: uint8 (rows, ceil(cols / 32)); a value is
    q * 2^(e - 127) (include/mao.h, mao_ckpt8, has the format in full).  `dtype` is the type
    of the values it was made from, which restore() gives back by default.  Every value is exact
    in bfloat16 and float32; float16 holds those of a float16 checkpoint.
    A checkpoint takes 33/64 of the bytes of a 16-bit matrix.
    """

    __slots__ = ("q", "e", "cols", "dtype")

    def __init__(self, q: torch.Tensor, e: torch.Tensor, cols: int, dtype: torch.dtype):
        cols = int(cols)
        if dtype not in _DTYPES:
            raise TypeError(f"checkpoint dtype {dtype} not supported")
        if cols < 8 or cols % 8:
            raise ValueError(f"{cols} columns: a positive multiple of 8 is needed")
        _check("q", q, dtype=torch.int8)
        _check("e", e, q.device, torch.uint8)
        blocks = (cols + 31) // 32
        if q.dim() != 2 or e.dim() != 2 or q.shape[1] != 32 * blocks or tuple(e.shape) != (q.shape[0], blocks):
            raise ValueError(f"a checkpoint of {cols} columns has q (rows, {32 * blocks}) and e (rows, {blocks}), got "
                             f"{tuple(q.shape)} and {tuple(e.shape)}")
        if max(q.shape[0], cols) > _MOST:
            raise ValueError(f"a checkpoint of {q.shape[0]} x {cols}: at most {_MOST} rows and columns")
        if not q.is_contiguous() or not e.is_contiguous():
            raise ValueError("q and e must be contiguous")
        self.q, self.e, self.cols, self.dtype = q, e, cols, dtype

    @classmethod
    def _like(cls, x: torch.Tensor, rows: int, cols: int) -> "Checkpoint8":
        """Room for rows x cols of x's type, on its device; nothing to check."""
        blocks = (cols + 31) // 32
        k = object.__new__(cls)
        k.q = x.new_empty((rows, 32 * blocks), dtype=torch.int8)
        k.e = x.new_empty((rows, blocks), dtype=torch.uint8)
        k.cols, k.dtype = cols, x.dtype
        return k

    @property
    def shape(self) -> Tuple[int, int]:
        return (self.q.shape[0], self.cols)

    @property
    def device(self):
        return self.q.device

    @property
    def nbytes(self) -> int:
        return self.q.numel() + self.e.numel()

    def _c(self) -> "L.Ckpt8":
        return L.Ckpt8(self.q.data_ptr(), self.e.data_ptr(), self.q.shape[1], self.e.shape[1])

    def restore(self, act: str = "none", dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """act(values), rounded to `dtype` (default: the checkpoint's own)."""
        a = _act(act)
        dtype = self.dtype if dtype is None else dtype
        if dtype not in _DTYPES:
            raise TypeError(f"dtype {dtype} not supported")
        dev = self.q.device
        if _elsewhere(dev):
            with torch.cuda.device(dev):
                return self.restore(act, dtype)
        rows = self.q.shape[0]
        y = self.q.new_empty((rows, self.cols), dtype=dtype)
        c = self._c()
        L.check(L.load().mao_checkpoint8_restore(ctypes.byref(c), rows, self.cols, a, y.data_ptr(), _DTYPES[dtype],
                                                 self.cols, _stream(dev.index)), "mao_checkpoint8_restore")
        return y


def checkpoint8(x: torch.Tensor) -> Checkpoint8:
    """The 8-bit checkpoint of x (float32, bfloat16 or float16)."""
    ld = _check_acts("x", x)
    if x.dtype not in _DTYPES:
        raise TypeError(f"x dtype {x.dtype} not supported (float32, bfloat16 or float16)")
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return checkpoint8(x)
    k = Checkpoint8._like(x, x.shape[0], x.shape[1])
    c = k._c()
    L.check(L.load().mao_checkpoint8(x.data_ptr(), _DTYPES[x.dtype], x.shape[0], x.shape[1], ld, ctypes.byref(c),
                                     _stream(dev.index)), "mao_checkpoint8")
    return k


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
               checkpoint: bool = False):
    """Layer norm of each row: (y, mean, rstd, kept).

    x: float32, bfloat16 or float16, up to 32768 columns; weight and bias: both float32 or
    both of x's type.  mean and rstd are float32, one per row, for the backward pass.  With
    `checkpoint`, kept is y's Checkpoint8, written in the same pass; else None.
    """
    ld = _check_acts("x", x)
    if x.dtype not in _DTYPES:
        raise TypeError(f"x dtype {x.dtype} not supported (float32, bfloat16 or float16)")
    rows, cols = x.shape
    dev = x.device
    _check_param("weight", weight, cols, dev, (torch.float32, x.dtype))
    if bias is not None:
        _check_param("bias", bias, cols, dev, (weight.dtype,))
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return layer_norm(x, weight, bias, eps=eps, checkpoint=checkpoint)
    y = x.new_empty((rows, cols))
    mean, rstd = x.new_empty(rows, dtype=torch.float32), x.new_empty(rows, dtype=torch.float32)
    kept = Checkpoint8._like(x, rows, cols) if checkpoint else None
    a = L.LayerNormArgs(rows, cols, _DTYPES[x.dtype], _DTYPES[weight.dtype], x.data_ptr(), ld, weight.data_ptr(),
                        _ptr(bias), eps, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(),
                        kept._c() if checkpoint else _NO_CKPT)
    L.check(L.load().mao_layer_norm(ctypes.byref(a), _stream(dev.index)), "mao_layer_norm")
    return y, mean, rstd, kept


def _check_kept(name: str, k, shape, device, dtype):
    """A tensor or a Checkpoint8 of the given shape: (pointer, leading dimension, Ckpt8)."""
    if isinstance(k, Checkpoint8):
        if k.shape != tuple(shape):
            raise ValueError(f"{name} has shape {k.shape}, expected {tuple(shape)}")
        if k.device != device:
            raise ValueError(f"{name} is on {k.device}, expected {device}")
        return None, shape[1], k._c()
    ld = _check_acts(name, k, shape, device, dtype)
    return k.data_ptr(), ld, _NO_CKPT


def layer_norm_backward(dy: torch.Tensor, x: Union[torch.Tensor, Checkpoint8], weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, *, dres: Optional[torch.Tensor] = None):
    """Layer norm's gradient: (dx, dw, db), dw and db in float32.

    x is the forward input, or a Checkpoint8 of it; mean and rstd are the forward's.  dres,
    the gradient that reaches x past the norm, is added to dx.
    """
    ld_dy = _check_acts("dy", dy)
    if dy.dtype not in _DTYPES:
        raise TypeError(f"dy dtype {dy.dtype} not supported (float32, bfloat16 or float16)")
    rows, cols = dy.shape
    dev = dy.device
    xp, ld_x, xc = _check_kept("x", x, (rows, cols), dev, dy.dtype)
    _check_param("weight", weight, cols, dev, (torch.float32, dy.dtype))
    _check_param("mean", mean, rows, dev, (torch.float32,))
    _check_param("rstd", rstd, rows, dev, (torch.float32,))
    ld_dres = _check_acts("dres", dres, (rows, cols), dev, dy.dtype) if dres is not None else 0
    lib = L.load()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return layer_norm_backward(dy, x, weight, mean, rstd, dres=dres)
    dx = dy.new_empty((rows, cols))
    dw, db = dy.new_empty(cols, dtype=torch.float32), dy.new_empty(cols, dtype=torch.float32)
    a = L.LayerNormBackwardArgs(rows, cols, _DTYPES[dy.dtype], _DTYPES[weight.dtype], dy.data_ptr(), ld_dy, xp,
                                ld_x, xc, weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(dres),
                                ld_dres, dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr())
    n = ctypes.c_size_t(0)
    L.check(lib.mao_layer_norm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)),
            "mao_layer_norm_backward_workspace_size")
    ws = dy.new_empty(n.value, dtype=torch.uint8)
    L.check(lib.mao_layer_norm_backward(ctypes.byref(a), ws.data_ptr(), n.value, _stream(dev.index)),
            "mao_layer_norm_backward")
    return dx, dw, db


def _check_weight(W: torch.Tensor, device, dtype) -> Tuple[int, int]:
    _check("W", W, device, dtype)
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be 2-D (out features, in features) and contiguous")
    if W.shape[0] % 8 or W.shape[1] % 8 or W.numel() == 0:
        raise ValueError(f"W has shape {tuple(W.shape)}: both sides must be positive multiples of 8")
    if max(W.shape) > _MOST:
        raise ValueError(f"W has shape {tuple(W.shape)}: at most {_MOST} rows and columns")
    return W.shape


def linear(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, *, act: str = "none",
           residual: Optional[torch.Tensor] = None, checkpoint: Union[bool, str] = False):
    """y = act(x W^T + bias) + residual: (y, kept).

    x (tokens, n), W (m, n) and residual (tokens, m): all bfloat16 or all float16; bias (m):
    float32 or of that type.  kept is what the backward pass needs of z = x W^T + bias:
    None, with checkpoint=True its Checkpoint8 (written in the product's epilogue), or with
    checkpoint="tensor" z itself, rounded to x's type.
    """
    ld_x = _check_acts("x", x)
    if x.dtype not in _HALF:
        raise TypeError(f"x dtype {x.dtype} not supported (bfloat16 or float16)")
    a_id = _act(act)
    if checkpoint not in (False, True, "tensor"):
        raise ValueError('checkpoint must be False, True or "tensor"')
    dev, dt = x.device, x.dtype
    m, n = _check_weight(W, dev, dt)
    rows = x.shape[0]
    if x.shape[1] != n:
        raise ValueError(f"x has {x.shape[1]} columns, W takes {n}")
    if bias is not None:
        _check_param("bias", bias, m, dev, (torch.float32, dt))
    ld_res = _check_acts("residual", residual, (rows, m), dev, dt) if residual is not None else 0
    lib = L.load()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear(x, W, bias, act=act, residual=residual, checkpoint=checkpoint)
    y = x.new_empty((rows, m))
    kept, z, zc = None, None, _NO_CKPT
    if checkpoint == "tensor":
        kept = z = x.new_empty((rows, m))
    elif checkpoint:
        kept = Checkpoint8._like(x, rows, m)
        zc = kept._c()
    a = L.LinearArgs(rows, n, m, _DTYPES[dt], x.data_ptr(), ld_x, W.data_ptr(), _ptr(bias),
                     _DTYPES[bias.dtype] if bias is not None else 0, a_id, _ptr(residual), ld_res, y.data_ptr(),
                     m, _ptr(z), m, zc)
    nb = ctypes.c_size_t(0)
    ref = ctypes.byref(a)
    L.check(lib.mao_linear_workspace_size(ref, ctypes.byref(nb)), "mao_linear_workspace_size")
    ws = x.new_empty(nb.value, dtype=torch.uint8) if nb.value else None
    L.check(lib.mao_linear(ref, _ptr(ws), nb.value, _stream(dev.index)), "mao_linear")
    return y, kept


def linear_backward(dy: torch.Tensor, x: Union[torch.Tensor, Checkpoint8], W: torch.Tensor, *,
                    z: Union[None, torch.Tensor, Checkpoint8] = None, act: str = "none",
                    dw: Optional[torch.Tensor] = None, accumulate: bool = False,
                    dw_dtype: torch.dtype = torch.float32, need_dx: bool = True, need_dw: bool = True,
                    need_db: bool = True):
    """The linear layer's gradient: (dx, dw, db); the residual's own gradient is dy.

    x is the forward input or its Checkpoint8 (of float16 values where dy is float16); z, which act other than "none" needs, is what
    linear() kept.  dw (m, n) is float32 or of dy's type: the given tensor (a batch's G), or a
    new one of dw_dtype.  accumulate adds to the given float32 dw.  db is float32.  What
    need_* leaves out comes back as None and costs nothing.
    """
    ld_dy = _check_acts("dy", dy)
    if dy.dtype not in _HALF:
        raise TypeError(f"dy dtype {dy.dtype} not supported (bfloat16 or float16)")
    a_id = _act(act)
    dev, dt = dy.device, dy.dtype
    m, n = _check_weight(W, dev, dt)
    rows = dy.shape[0]
    if dy.shape[1] != m:
        raise ValueError(f"dy has {dy.shape[1]} columns, W gives {m}")
    xp, ld_x, xc = _check_kept("x", x, (rows, n), dev, dt)
    if need_dw and dt == torch.float16 and isinstance(x, Checkpoint8) and x.dtype != dt:
        raise TypeError(f"x is a checkpoint of {x.dtype} values, which the product dz^T x would read as {dt}: above "
                        f"65504 they would be infinite (Checkpoint8(x.q, x.e, x.cols, {dt}) says that they are not)")
    zp, ld_z, zc = None, 0, _NO_CKPT
    if a_id:
        if z is None:
            raise ValueError(f'act="{act}" needs z')
        zp, ld_z, zc = _check_kept("z", z, (rows, m), dev, dt)
    if dw is not None:
        if not need_dw:
            raise ValueError("dw is given, but need_dw is False")
        _check("dw", dw, dev)
        if tuple(dw.shape) != (m, n) or not dw.is_contiguous():
            raise ValueError(f"dw must be contiguous of shape {(m, n)}, got {tuple(dw.shape)}")
        dw_dtype = dw.dtype
    elif accumulate:
        raise ValueError("accumulate needs dw")
    if dw_dtype not in (torch.float32, dt):
        raise TypeError(f"dw must be torch.float32 or {dt}, got {dw_dtype}")
    if accumulate and dw_dtype != torch.float32:
        raise TypeError("accumulate needs a float32 dw")
    lib = L.load()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear_backward(dy, x, W, z=z, act=act, dw=dw, accumulate=accumulate, dw_dtype=dw_dtype,
                                   need_dx=need_dx, need_dw=need_dw, need_db=need_db)
    dx = dy.new_empty((rows, n)) if need_dx else None
    if dw is None and need_dw:
        dw = dy.new_empty((m, n), dtype=dw_dtype)
    db = dy.new_empty(m, dtype=torch.float32) if need_db else None
    a = L.LinearBackwardArgs(rows, n, m, _DTYPES[dt], dy.data_ptr(), ld_dy, xp, ld_x, xc, W.data_ptr(), a_id, zp,
                             ld_z, zc, _ptr(dx), n, _ptr(dw), _DTYPES[dw_dtype], int(bool(accumulate)), _ptr(db))
    nb = ctypes.c_size_t(0)
    ref = ctypes.byref(a)
    L.check(lib.mao_linear_backward_workspace_size(ref, ctypes.byref(nb)), "mao_linear_backward_workspace_size")
    ws = dy.new_empty(nb.value, dtype=torch.uint8) if nb.value else None
    L.check(lib.mao_linear_backward(ref, _ptr(ws), nb.value, _stream(dev.index)), "mao_linear_backward")
    return dx, dw, db


def layer_status(device=None) -> Tuple[int, int]:
    """(status, site) of the first condition that these operators recorded on the device
    since the last call (0: none).  Synchronises the device's current stream."""
    dev = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if dev.index is None else dev.index
    where = ctypes.c_int32(0)
    with torch.cuda.device(index):
        st = L.load().mao_layer_status(_stream(index), ctypes.byref(where))
    return st, where.value

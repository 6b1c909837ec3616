"""Rules of the trained layers that a machine without a GPU can check: in the kernels' source,
in the host's plans, and in the binding."""

import ctypes
import glob
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from matrix_aware_optimizers_02_b200 import _lib as L
from matrix_aware_optimizers_02_b200 import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAYERS = os.path.join(ROOT, "matrix_aware_optimizers_02_b200", "csrc", "layers")


def _functions():
    """(name, head, body) of each function of the trained layers' sources: head is all between
    the end of what comes before and the body's opening brace."""
    for path in sorted(glob.glob(os.path.join(LAYERS, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__(?:global|device)__[^;{}]*?\b(\w+)\s*\(((?:[^(){};]|\([^(){};]*\))*)\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield m.group(1), m.group(0), text[m.end():i]


def test_dependent_kernels_promise_nothing_of_their_inputs():
    """A kernel that waits for the one before it may run while that one still writes what this
    one reads.  __restrict__ on such a pointer would promise the compiler that nobody does, and
    allow loads that the wait does not order."""
    functions = list(_functions())
    waits = {n for n, _, body in functions if "wait_for_previous()" in body}
    kernels = [(n, head, body) for n, head, body in functions
               if "__global__" in head and (n in waits or any(re.search(rf"\b{w}\s*<", body) for w in waits))]
    names = {n for n, _, _ in kernels}
    assert {"col_reduce_kernel", "lin_join_kernel", "lin_kernel", "lin_pair_kernel"} <= names
    for n, head, body in kernels:
        assert "__restrict__" not in head, f"{n} takes a __restrict__ pointer"
    for n, head, body in functions:
        if n in waits:
            assert "__ldg" not in body and "ld.global.nc" not in body, f"{n} reads by the non-coherent path"


@pytest.mark.parametrize("big", [2**30 + 8, 2**32 + 8])
def test_weights_and_checkpoints_past_the_limit_are_refused(monkeypatch, big):
    """The C structs' fields have 32 bits: 2^32 + 8 rows of a weight, or columns of a checkpoint,
    would reach the library as 8 without an error."""
    monkeypatch.setattr(layers, "_check", lambda *a, **k: None)
    t = torch.bfloat16

    def meta(rows, cols, dtype=t):
        return torch.empty((rows, cols), dtype=dtype, device="meta")

    calls = [lambda: layers.linear(meta(1, 8), meta(big, 8)), lambda: layers.linear(meta(1, big), meta(8, big)),
             lambda: layers.linear_backward(meta(1, big), meta(1, 8), meta(big, 8))]
    blocks = (big + 31) // 32
    calls += [lambda: layers.Checkpoint8(meta(1, 32 * blocks, torch.int8), meta(1, blocks, torch.uint8), big, t),
              lambda: layers.Checkpoint8(meta(big, 32, torch.int8), meta(big, 1, torch.uint8), 8, t)]
    for call in calls:
        with pytest.raises(ValueError, match="at most"):
            call()


@pytest.mark.parametrize("kept", [torch.bfloat16, torch.float32])
def test_float16_products_refuse_checkpoints_of_wider_types(monkeypatch, kept):
    """dW = dz^T x reads x back in dy's type, and float16 ends at 65504."""
    monkeypatch.setattr(layers, "_check", lambda *a, **k: None)
    k = object.__new__(layers.Checkpoint8)
    k.q = torch.empty((4, 32), dtype=torch.int8, device="meta")
    k.e = torch.empty((4, 1), dtype=torch.uint8, device="meta")
    k.cols, k.dtype = 16, kept
    dy = torch.empty((4, 8), dtype=torch.float16, device="meta")
    w = torch.empty((8, 16), dtype=torch.float16, device="meta")
    with pytest.raises(TypeError, match="checkpoint of"):
        layers.linear_backward(dy, k, w)


def test_forward_mode_tangents_are_refused():
    """These calls record no graph, so a tangent would be dropped without an error; under no_grad
    too, which does not stop forward mode."""
    import torch.autograd.forward_ad as fw

    class OnDevice(torch.Tensor):  # passes for a CUDA tensor, so that the check goes on
        is_cuda = True

    x = torch.zeros((4, 8))
    plain = torch.Tensor._make_subclass(OnDevice, x)
    layers._check("x", plain)
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        on = torch.Tensor._make_subclass(OnDevice, x)
        dual = fw.make_dual(on, torch.ones_like(x))
        if not isinstance(dual, OnDevice):
            dual = dual.as_subclass(OnDevice)
        assert fw.unpack_dual(dual).tangent is not None and fw.unpack_dual(d).tangent is not None
        layers._check("x", plain)
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises(ValueError, match="tangent"):
                layers._check("x", dual)
        layers._check("x", fw.unpack_dual(dual).primal)
        with fw._set_fwd_grad_enabled(False):
            layers._check("x", dual)
    layers._check("x", plain)


_WITHOUT_CUDA = """
import torch
for name in ("_cuda_getCurrentRawStream",):  # a torch built without CUDA has no such name
    delattr(torch._C, name)
from matrix_aware_optimizers_02_b200 import api, layers
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda device: Stream if device == 3 else None
assert layers._stream(3) == 77
try:
    api.checkpoint8(torch.zeros((4, 16)))
except ValueError as e:
    assert "CUDA tensor" in str(e)
print("imported")
"""


def test_binding_imports_without_cuda_in_torch():
    """The package's host side (layer sets, plans, refusals) works with a torch built for the CPU."""
    r = subprocess.run([sys.executable, "-c", _WITHOUT_CUDA], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stdout + r.stderr


def _deal(lib, sizes, backward, workers, room):
    flat = (ctypes.c_int64 * 6)(*[v for s in sizes for v in s])
    plan = (ctypes.c_int32 * 14)()
    st = lib.mao_test_linear_deal(flat, len(sizes), int(backward), workers, plan, room.ctypes.data, room.nbytes)
    return st, list(plan)


@pytest.mark.parametrize("seed", range(6))
def test_every_work_item_is_dealt_once(seed):
    """Random sizes of one product and of a gradient's two, on a B200's workers, on fewer, and on
    an odd number: each tile, and each K slice of a sliced tile, is in exactly one list, and the
    slices of a tile cover its K."""
    lib = L.load()
    rng = np.random.default_rng(seed)
    room = np.zeros(1 << 22, dtype=np.uint8)

    def size(low, high):
        return int(round(np.exp(rng.uniform(np.log(low), np.log(high)))))

    for _ in range(300):
        rows, n, m = size(1, 70000), 8 * size(1, 2048), 8 * size(1, 2048)
        dx, dw = (rows, n, m), (m, n, rows)
        for sizes, backward in (([(rows, m, n)], 0), ([dx], 1), ([dw], 1), ([dx, dw] if m >= rows else [dw, dx], 1)):
            for grid in (None, 1, 37):
                st, plan = _deal(lib, sizes, backward, grid or 74, room)
                if grid is None and plan[1] != 74:
                    st, plan = _deal(lib, sizes, backward, plan[1], room)
                assert st == L.MAO_OK, (sizes, backward, grid)
                edge, items = plan[0], 0
                for i, (M, N, K) in enumerate(sizes):
                    tm, tn, nk, full, slices, blocks = plan[2 + 6 * i:8 + 6 * i]
                    assert (tm, tn, nk) == (-(-M // edge), -(-N // edge), -(-K // 64))
                    assert 0 <= full <= tm * tn and slices >= 1
                    if slices > 1:  # the last slice is not empty
                        assert (slices - 1) * blocks < nk <= slices * blocks
                    items += full + (tm * tn - full) * slices
                assert (room[:items] == 1).all(), (sizes, backward, grid, np.unique(room[:items], return_counts=True))


def test_deal_refusals():
    lib = L.load()
    room = np.zeros(4, dtype=np.uint8)
    assert _deal(lib, [(256, 256, 64)], 0, 74, room)[0] == L.MAO_OK
    assert _deal(lib, [(4096, 4096, 64)], 0, 74, room)[0] == L.MAO_ERR_WORKSPACE
    assert _deal(lib, [(0, 256, 64)], 0, 74, room)[0] == L.MAO_ERR_SHAPE
    assert _deal(lib, [(256, 256, 64)], 0, 0, room)[0] == L.MAO_ERR_INVALID_ARG
    assert _deal(lib, [(256, 256, 64)] * 2, 0, 74, room)[0] == L.MAO_ERR_INVALID_ARG

"""Forms of the trained-layer calls that the documentation allows: checkpoints of one type read
in another, the status that the device recorded."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from matrix_aware_optimizers_02_b200 import api as A
    yield A
    assert A.layer_status() == (0, 0)


def test_checkpoints_of_another_type(api):
    """A checkpoint's values are exact in bf16 and fp32, so bf16 products and the norm's gradient read
    any checkpoint as they read its values; fp16 products read those of fp16 alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    bf, hf = torch.bfloat16, torch.float16
    x = torch.randn((70, 72), generator=g, device="cuda") * 3e4
    x[5] = 1e6
    dy = torch.randn((70, 136), generator=g, device="cuda")
    w = torch.randn((136, 72), generator=g, device="cuda")
    for src in (torch.float32, bf):
        k = api.checkpoint8(x.to(src))
        v = k.restore(dtype=bf)
        assert torch.equal(v.float(), k.restore(dtype=torch.float32))
        want = api.linear_backward(dy.to(bf), v, w.to(bf))
        assert all(torch.equal(a, b) for a, b in zip(api.linear_backward(dy.to(bf), k, w.to(bf)), want))
        with pytest.raises(TypeError, match="checkpoint of"):
            api.linear_backward(dy.to(hf), k, w.to(hf))
        dx, dw, db = api.linear_backward(dy.to(hf), k, w.to(hf), need_dw=False)  # x is not read
        assert dw is None and torch.isfinite(dx).all()
        # the norm's gradient works in fp32
        ones, mean, rstd = torch.ones(72, device="cuda"), v.float().mean(1), 1 / v.float().std(1).clamp(min=1.0)
        d = torch.randn((70, 72), generator=g, device="cuda").to(hf)
        got = api.layer_norm_backward(d, k, ones, mean, rstd)
        ref = api.layer_norm_backward(d.float(), v.float(), ones, mean, rstd)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        assert torch.equal(got[0], ref[0].to(hf)) and torch.equal(got[1], ref[1])
    # z is read in fp32 whatever its type
    zk = api.checkpoint8(dy.to(bf) * 1e5)
    dx, _, _ = api.linear_backward(dy.to(hf), x.to(hf).clamp(-1, 1), w.to(hf), z=zk, act="gelu")
    assert torch.isfinite(dx).all()


def test_status_is_returned_once(api):
    """What a bounded wait would record: the status and its site once, then nothing."""
    from matrix_aware_optimizers_02_b200 import _lib as L
    L.check(L.load().mao_test_set_layer_status(L.MAO_ERR_TIMEOUT, 53))
    assert api.layer_status() == (L.MAO_ERR_TIMEOUT, 53)
    assert api.layer_status() == (0, 0)
    assert api.layer_status(torch.cuda.current_device()) == (0, 0)

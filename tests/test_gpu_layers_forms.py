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
        # one made from values that fit may say so
        small = api.checkpoint8((x / 1e6).to(src))
        said = api.Checkpoint8(small.q, small.e, small.cols, hf)
        want = api.linear_backward(dy.to(hf), said.restore(), w.to(hf))
        assert all(torch.equal(a, b) for a, b in zip(api.linear_backward(dy.to(hf), said, w.to(hf)), want))
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


def test_threads_on_streams_of_their_own(api):
    """Four host threads, each with its own sizes and stream: the bits of a call alone, rows far
    from zero among them."""
    import threading
    bf = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def make(rows, n, m):
        x = (torch.randn((rows, n), generator=g, device="cuda") + 30).to(bf)
        w = (torch.randn((m, n), generator=g, device="cuda") * n ** -0.5).to(bf)
        dy, lw = torch.randn((rows, m), generator=g, device="cuda").to(bf), torch.ones(n, device="cuda")

        def step():
            h, mean, rstd, hk = api.layer_norm(x, lw, checkpoint=True)
            y, zk = api.linear(h, w, act="gelu_tanh", checkpoint=True)
            r = api.linear_backward(dy, hk, w, z=zk, act="gelu_tanh")
            return (y, hk.restore("silu", torch.float32)) + r + tuple(api.layer_norm_backward(r[0], x, lw, mean, rstd))

        return step

    steps = [make(*s) for s in ((333, 768, 2304), (1000, 1024, 264), (77, 14336, 512), (4096, 256, 1024))]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                out = steps[i]()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(out, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("kept", ["", "x", "z", "xz"])
def test_every_subset_of_gradients(api, act, kept):
    """What need_* leaves out comes back as None, the rest as it is among the others, whichever of
    x and z is a checkpoint.  Two bf16 roundings of one value differ by a step at most, 2^-7 of it."""
    bf = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, w = torch.randn((300, 520), generator=g, device="cuda").to(bf), torch.randn((264, 520), generator=g, device="cuda").to(bf)
    dy, z = (torch.randn((300, 264), generator=g, device="cuda").to(bf) for _ in range(2))
    x = api.checkpoint8(x) if "x" in kept else x
    z = api.checkpoint8(z) if "z" in kept else z
    full = api.linear_backward(dy, x, w, z=z, act=act)
    for b in range(8):
        out = api.linear_backward(dy, x, w, z=z, act=act, need_dx=bool(b & 1), need_dw=bool(b & 2), need_db=bool(b & 4))
        for got, want, bit in zip(out, full, (1, 2, 4)):
            assert (got is None) == (not b & bit)
            if got is not None:
                assert (got.double() - want.double()).norm() <= 2.0 ** -7 * want.double().norm()

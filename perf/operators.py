"""The operators of a trained linear layer, as cases to be timed and compared.

The optimizers of this package take the gradient G of a weight matrix W.  The operators
here are what makes that gradient: layer norm, the linear layer itself (product, bias,
activation and residual), its backward pass, and the 8-bit checkpoints of activations that
the backward pass reads.  `run` computes each of them either in a plain form, in elementary
torch operations, or (`own` true) by the package's public entry points.

8-bit checkpoint: a row's columns in blocks of 32, the last one possibly short.  A block
holds a byte e and 32 whole numbers q in [-127, 127]; a value is q * 2^(e - 127).  With a the
block's largest magnitude and E = floor(log2 a): e = max(E + 121, 1), and q is the value
divided by 2^(e - 127), rounded to nearest even and limited to +-127.  q is stored with rows
padded to whole blocks.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")
_EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a small model's attention, a batch of a few dozen tokens
        {"name": "norm-short", "op": "norm", "rows": 48, "cols": 768, "type": "bf16", "checkpoint": False},
        # the norm of a wide model over a full batch, with its output kept in 8 bits for the backward pass
        {"name": "norm-kept", "op": "norm", "rows": 16384, "cols": 4096, "type": "bf16", "checkpoint": True},
        # its gradient in a mid-sized model: odd token count, the residual stream's gradient joined
        {"name": "norm-grad", "op": "norm_grad", "rows": 8191, "cols": 1536, "type": "bf16", "kept": False, "residual": True},
        # the same for a wide model whose input was kept in 8 bits
        {"name": "norm-grad-kept", "op": "norm_grad", "rows": 16384, "cols": 4096, "type": "fp16", "kept": True, "residual": False},
        # activations of an expert's input written to 8 bits and read back through the activation
        {"name": "keep-act", "op": "keep", "rows": 5003, "cols": 2048, "type": "bf16", "act": "gelu"},
        # a wide residual stream written and read back
        {"name": "keep-wide", "op": "keep", "rows": 16384, "cols": 4096, "type": "fp32", "act": "none"},
        # fused q, k, v projection of a small model, a few dozen tokens: latency
        {"name": "linear-short", "op": "linear", "rows": 33, "in": 768, "out": 2304, "type": "bf16", "act": "none",
         "bias": True, "residual": False, "checkpoint": False},
        # down projection of a mid-sized model into the residual stream
        {"name": "linear-residual", "op": "linear", "rows": 4001, "in": 6144, "out": 1536, "type": "fp16", "act": "none",
         "bias": True, "residual": True, "checkpoint": False},
        # up projection of a wide model, its values before the activation kept in 8 bits
        {"name": "linear-kept", "op": "linear", "rows": 8192, "in": 4096, "out": 14336, "type": "bf16", "act": "silu",
         "bias": True, "residual": False, "checkpoint": True},
        # an expert with few tokens, gradient added to the fp32 buffer of earlier microbatches
        {"name": "linear-grad-expert", "op": "linear_grad", "rows": 301, "in": 2048, "out": 768, "type": "bf16",
         "act": "none", "kept": False, "grad": "fp32", "add": True},
        # attention's output projection in a mid-sized model
        {"name": "linear-grad", "op": "linear_grad", "rows": 4096, "in": 1536, "out": 1536, "type": "fp16", "act": "none",
         "kept": True, "grad": "fp32", "add": False},
        # up projection of a wide model, from 8-bit checkpoints of its input and of what its activation took
        {"name": "linear-grad-kept", "op": "linear_grad", "rows": 8192, "in": 4096, "out": 14336, "type": "bf16",
         "act": "gelu", "kept": True, "grad": "bf16", "add": False},
    ]


def _log(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "keep", "linear", "linear", "linear_grad", "linear_grad"))
    half = rng.choice(("bf16", "fp16"))
    if op in ("norm", "norm_grad", "keep"):
        cols = _log(rng, 8, 14336, 8)
        rows = _log(rng, 1, max(2, min(40000, 16384 * 4096 // cols)))
        c = {"op": op, "rows": rows, "cols": cols, "type": rng.choice(("bf16", "fp16", "fp32"))}
        if op == "norm":
            return {**c, "checkpoint": rng.random() < 0.5}
        if op == "norm_grad":
            return {**c, "kept": rng.random() < 0.5, "residual": rng.random() < 0.5}
        return {**c, "act": rng.choice(_ACTS)}
    n, m = _log(rng, 8, 14336, 8), _log(rng, 8, 14336, 8)
    most = 8192 * 4096 * 14336 // (n * m)
    c = {"op": op, "rows": _log(rng, 1, max(2, min(16384, most))), "in": n, "out": m, "type": half, "act": rng.choice(_ACTS)}
    if op == "linear":
        return {**c, "bias": rng.random() < 0.7, "residual": rng.random() < 0.5, "checkpoint": rng.random() < 0.5}
    # a gradient in 32 bits belongs to an exact dy, as where there is no activation
    if rng.random() < 0.5:
        return {**c, "act": "none", "kept": rng.random() < 0.5, "grad": "fp32", "add": rng.random() < 0.5}
    return {**c, "kept": rng.random() < 0.5, "grad": half if half == "bf16" else "fp16", "add": False}


# ------------------------------------------------------------------ inputs
def _blocks(cols):
    return (cols + 31) // 32


def _pack(x):
    """(q padded to whole blocks, e) of a matrix, in elementary operations."""
    rows, cols = x.shape
    nb = _blocks(cols)
    v = x.float()
    if nb * 32 != cols:
        v = torch.cat((v, v.new_zeros(rows, nb * 32 - cols)), 1)
    v = v.view(rows, nb, 32)
    a = v.abs().amax(2)
    _, p = torch.frexp(a)  # a = f 2^p with f in [1/2, 1): floor(log2 a) = p - 1
    e = torch.where(a > 0, p - 1 + 121, torch.ones_like(p)).clamp(min=1)
    q = torch.round(torch.ldexp(v, (127 - e).unsqueeze(2))).clamp(-127, 127)
    return q.to(torch.int8).view(rows, nb * 32), e.to(torch.uint8)


def _unpack(q, e, cols):
    """The fp32 values that a checkpoint stands for."""
    v = q.view(q.shape[0], -1, 32).float()
    return torch.ldexp(v, (e.int() - 127).unsqueeze(2)).reshape(q.shape[0], -1)[:, :cols]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    t = _TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    def stream(rows, cols):
        """Values as in a residual stream: unit scale, a few features many times larger."""
        x = normal(rows, cols)
        big = torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=dev)
        x[:, big] *= 12.0
        return x

    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        x = stream(rows, cols) + 0.2
        s["w"] = 1.0 + normal(cols, std=0.1)
        if case["op"] == "norm":
            s["x"] = x.to(t)
            s["b"] = normal(cols, std=0.1)
            return s
        x = x.to(t)
        if case["kept"]:
            s["q"], s["e"] = _pack(x)
            x = _unpack(s["q"], s["e"], cols)
        else:
            s["x"] = x
        x = x.double()
        s["mean"] = x.mean(1).float()
        s["rstd"] = (x.var(1, correction=0) + _EPS).rsqrt().float()
        s["dy"] = normal(rows, cols, std=0.02).to(t)
        s["dres"] = normal(rows, cols, std=0.02).to(t) if case["residual"] else None
        return s
    if case["op"] == "keep":
        s["x"] = stream(case["rows"], case["cols"]).to(t)
        return s
    rows, n, m = case["rows"], case["in"], case["out"]
    s["w"] = normal(m, n, std=n ** -0.5).to(t)
    x = normal(rows, n).to(t)
    if case["op"] == "linear":
        s["x"] = x
        s["b"] = normal(m, std=0.1) if case["bias"] else None
        s["res"] = stream(rows, m).to(t) if case["residual"] else None
        return s
    s["dy"] = normal(rows, m, std=0.02).to(t)
    z = normal(rows, m).to(t) if case["act"] != "none" else None
    if case["kept"]:
        s["xq"], s["xe"] = _pack(x)
        if z is not None:
            s["zq"], s["ze"] = _pack(z)
    else:
        s["x"] = x
        if z is not None:
            s["z"] = z
    if case["add"]:
        s["earlier"] = normal(m, n, std=0.02)
    return s


# ------------------------------------------------------------------ plain forms
def _act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) * z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))  # silu


def _slope(z, name):
    """The activation's derivative."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * z.clamp(min=0)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _run_norm(s):
    c, x = s["case"], s["x"]
    if own:
        y, mean, rstd, kept = _api().layer_norm(x, s["w"], s["b"], eps=_EPS, checkpoint=c["checkpoint"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if c["checkpoint"]:
            out["kept"] = kept.restore()
        return out
    v = x.float()
    mean = v.mean(1, keepdim=True)
    d = v - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + _EPS)
    y = (d * rstd * s["w"] + s["b"]).to(x.dtype)
    out = {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if c["checkpoint"]:
        out["kept"] = _unpack(*_pack(y), c["cols"]).to(x.dtype)
    return out


def _run_norm_grad(s):
    c, dy = s["case"], s["dy"]
    if own:
        a = _api()
        x = a.Checkpoint8(s["q"], s["e"], c["cols"], dy.dtype) if c["kept"] else s["x"]
        dx, dw, db = a.layer_norm_backward(dy, x, s["w"], s["mean"], s["rstd"], dres=s["dres"])
        return {"dx": dx, "dw": dw, "db": db}
    x = _unpack(s["q"], s["e"], c["cols"]) if c["kept"] else s["x"].float()
    h = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy.float()
    u = g * s["w"]
    dx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(dy.dtype), "dw": (g * h).sum(0), "db": g.sum(0)}


def _run_keep(s):
    c, x = s["case"], s["x"]
    if own:
        return _api().checkpoint8(x).restore(act=c["act"])
    return _act(_unpack(*_pack(x), c["cols"]), c["act"]).to(x.dtype)


def _run_linear(s):
    c, x = s["case"], s["x"]
    if own:
        y, kept = _api().linear(x, s["w"], s["b"], act=c["act"], residual=s["res"], checkpoint=c["checkpoint"])
        return {"y": y, "kept": kept.restore()} if c["checkpoint"] else {"y": y}
    z = x.float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(x.dtype)}
    if c["checkpoint"]:
        out["kept"] = _unpack(*_pack(z), c["out"]).to(x.dtype)
    return out


def _run_linear_grad(s):
    c, dy, w = s["case"], s["dy"], s["w"]
    if own:
        a = _api()
        x = a.Checkpoint8(s["xq"], s["xe"], c["in"], dy.dtype) if c["kept"] else s["x"]
        z = None
        if c["act"] != "none":
            z = a.Checkpoint8(s["zq"], s["ze"], c["out"], dy.dtype) if c["kept"] else s["z"]
        into = s["earlier"].clone() if c["add"] else None
        dx, dw, db = a.linear_backward(dy, x, w, z=z, act=c["act"], dw=into, accumulate=c["add"], dw_dtype=_TYPES[c["grad"]])
        return {"dx": dx, "dw": dw, "db": db}
    x = _unpack(s["xq"], s["xe"], c["in"]) if c["kept"] else s["x"].float()
    dz = dy.float()
    if c["act"] != "none":
        z = _unpack(s["zq"], s["ze"], c["out"]) if c["kept"] else s["z"].float()
        dz = dz * _slope(z, c["act"])
    dw = dz.t() @ x
    if c["add"]:
        dw = s["earlier"] + dw
    return {"dx": (dz @ w.float()).to(dy.dtype), "dw": dw.to(_TYPES[c["grad"]]), "db": dz.sum(0)}


def _api():
    from matrix_aware_optimizers_02_b200 import api

    return api


_RUN = {"norm": _run_norm, "norm_grad": _run_norm_grad, "keep": _run_keep, "linear": _run_linear, "linear_grad": _run_linear_grad}


def run(state):
    return _RUN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    t = 4 if case["type"] == "fp32" else 2
    op = case["op"]
    if op in ("norm", "norm_grad", "keep"):
        rows, cols = case["rows"], case["cols"]
        n, held = rows * cols, rows * (cols + _blocks(cols))
        if op == "norm":  # read x, write y; where kept: write 8 bits, read them, write the values
            return {"bytes": 2 * t * n + 8 * cols + 8 * rows + ((2 * held + t * n) if case["checkpoint"] else 0), "flops": 8 * n}
        if op == "norm_grad":
            return {"bytes": (held if case["kept"] else t * n) + (3 if case["residual"] else 2) * t * n + 12 * cols + 8 * rows, "flops": 14 * n}
        return {"bytes": 2 * t * n + 2 * held, "flops": 8 * n}
    rows, n, m = case["rows"], case["in"], case["out"]
    if op == "linear":
        held = rows * (m + _blocks(m))
        b = t * (rows * n + m * n + rows * m) + (4 * m if case["bias"] else 0) + (t * rows * m if case["residual"] else 0)
        return {"bytes": b + ((2 * held + t * rows * m) if case["checkpoint"] else 0), "flops": 2 * rows * n * m}
    grad = 4 if case["grad"] == "fp32" else 2
    x = rows * (n + _blocks(n)) if case["kept"] else t * rows * n
    z = 0 if case["act"] == "none" else (rows * (m + _blocks(m)) if case["kept"] else t * rows * m)
    return {"bytes": x + z + t * (rows * m + m * n + rows * n) + grad * m * n * (3 if case["add"] else 1) + 4 * m, "flops": 4 * rows * n * m}


# ------------------------------------------------------------------ 64 bits
def _values64(x):
    """What an 8-bit checkpoint of x (64 bits) stands for, in 64 bits, from the format's definition."""
    rows, cols = x.shape
    out = torch.zeros((rows, _blocks(cols) * 32), dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    out = out.view(rows, -1, 32)
    top = out.abs().max(2, keepdim=True).values
    power = torch.where(top > 0, torch.frexp(top)[1] - 7, torch.full_like(top, -126, dtype=torch.int32)).clamp(min=-126)
    step = torch.ldexp(torch.ones_like(top), power)
    return (torch.round(out / step).clamp(-127, 127) * step).reshape(rows, -1)[:, :cols]


def _held64(q, e, cols):
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=q.device), e.double() - 127).repeat_interleave(32, 1)
    return (q.double() * step)[:, :cols]


def _act64(z, name):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "relu2":
        return torch.where(z > 0, z, 0.0) ** 2
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if name == "silu" else z


def _slope64(z, name):
    with torch.enable_grad():
        v = z.detach().clone().requires_grad_(True)
        return torch.autograd.grad(_act64(v, name).sum(), v)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, n = s["x"].double(), case["cols"]
        mean = x.sum(1) / n
        rstd = ((x - mean[:, None]).square().sum(1) / n + _EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * s["w"].double() + s["b"].double()
        out = {"y": y, "mean": mean, "rstd": rstd}
        if case["checkpoint"]:  # of the values that y holds in its type
            out["kept"] = _values64(y.to(s["x"].dtype).double())
        return out
    if op == "norm_grad":
        x = _held64(s["q"], s["e"], case["cols"]) if case["kept"] else s["x"].double()
        w, dy, n = s["w"].double(), s["dy"].double(), case["cols"]
        rstd = s["rstd"].double()[:, None]
        h = (x - s["mean"].double()[:, None]) * rstd
        wdy = dy * w
        dx = rstd / n * (n * wdy - wdy.sum(1)[:, None] - h * (wdy * h).sum(1)[:, None])
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, h), "db": dy.sum(0)}
    if op == "keep":
        return _act64(_values64(s["x"].double()), case["act"])
    w = s["w"].double()
    if op == "linear":
        z = torch.einsum("ti,oi->to", s["x"].double(), w)
        if s["b"] is not None:
            z += s["b"].double()
        y = _act64(z, case["act"])
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y, "kept": _values64(z)} if case["checkpoint"] else {"y": y}
    dz = s["dy"].double()
    if case["act"] != "none":
        dz = dz * _slope64(_held64(s["zq"], s["ze"], case["out"]) if case["kept"] else s["z"].double(), case["act"])
    x = _held64(s["xq"], s["xe"], case["in"]) if case["kept"] else s["x"].double()
    dw = torch.einsum("to,ti->oi", dz, x)
    if case["add"]:
        dw += s["earlier"].double()
    return {"dx": torch.einsum("to,oi->ti", dz, w), "dw": dw, "db": dz.sum(0)}

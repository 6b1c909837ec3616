"""The trained-layer operators in 64 bits, written from their definitions (torch, any device)."""

from __future__ import annotations

import math

import torch

# half a step of a type, relative to the value
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")
F32 = 2.0 ** -24  # half a step of fp32
TC = 2.0 ** -23   # an add that truncates to fp32 is off by at most one step


def act(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "relu2":
        return torch.relu(z) ** 2
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * torch.relu(z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def power_of_two(k):
    """2^k in 64 bits, exactly (torch.pow is not, for every k): the exponent field alone."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def pack(x):
    """(q, e) of the 8-bit checkpoint of x, in 64 bits."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    v = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, nb, 32)
    a = v.abs().amax(2)
    bad = ~torch.isfinite(a)
    power = torch.frexp(torch.where(bad | (a == 0), torch.ones_like(a), a))[1].long() - 1  # floor(log2 a)
    e = torch.where(a == 0, torch.ones_like(power), (power + 121).clamp(min=1))
    step = power_of_two(e - 127)
    q = torch.round(v / step.unsqueeze(2)).clamp(-127, 127)
    q = torch.where(bad.unsqueeze(2), torch.zeros_like(q), q)
    e = torch.where(bad, torch.full_like(e, 255), e)
    return q.view(rows, nb * 32).to(torch.int8), e.to(torch.uint8)


def unpack(q, e, cols):
    """What (q, e) stands for, in 64 bits."""
    e = e.long()
    step = power_of_two(e - 127)
    step = torch.where(e == 255, torch.full_like(step, math.nan), torch.where(e == 0, torch.zeros_like(step), step))
    return (q.double() * step.repeat_interleave(32, 1))[:, :cols]


def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = ((x - mean[:, None]) ** 2).mean(1).add(eps).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None] * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd, dres=None):
    dy, x, w, mean, rstd = dy.double(), x.double(), w.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    u = dy * w
    dx = rstd * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * h).sum(0), dy.sum(0)


def close(got, want, tol, what):
    """Every element within tol (a tensor or a number); NaN and infinities in the same places."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(want.shape)}"
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities differ"
    err = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    tol = torch.as_tensor(tol, dtype=torch.float64, device=want.device).expand_as(want)
    over = torch.where(fine, err - tol, torch.full_like(err, -1.0))
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {got.reshape(-1)[i].item()!r} for {want.reshape(-1)[i].item()!r}, off by "
                             f"{err.reshape(-1)[i].item():.3e}, at most {tol.reshape(-1)[i].item():.3e} allowed "
                             f"({int((over > 0).sum())} of {over.numel()} over)")

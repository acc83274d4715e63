"""Plain implementations of the 8-bit projection operators, for the tests: the quantisation rule in
float and in 64 bits, the RMSNorm's defined roundings, and the product in 64 bits."""

import torch


def up(x, a):
    return -(-x // a) * a


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def block_exponents(y, rows):
    """Per block of `rows` x 128 of y [n, k]: the smallest e >= -127 with max finite |y| <= 448 * 2^e, 0 for zeros."""
    n, k = y.shape
    a = y.double().abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a))
    a = torch.nn.functional.pad(a, (0, up(k, 128) - k, 0, up(n, rows) - n))
    amax = a.view(up(n, rows) // rows, rows, up(k, 128) // 128, 128).amax(dim=(1, 3))
    mant, ex = torch.frexp(amax)                       # 448 = 0.875 * 2^9
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(min=-127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def spread(e, rows, n, k):
    """Block exponents as one per element of [n, k]."""
    return e.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :k]


def quantise(y, rows):
    """(codes as uint8 [n, k], scale bytes [n / rows, k / 128]) of float y."""
    n, k = y.shape
    e = block_exponents(y, rows)
    v = (y.double() * pow2(-spread(e, rows, n, k))).float()      # exact: a power of two
    v = torch.where(torch.isfinite(v), v, torch.full_like(v, float("nan")))
    return v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def values(q, scale, rows):
    """The values in 64 bits that codes [n, k] and scale bytes stand for (255: NaN)."""
    n, k = q.shape
    f = pow2(scale[:, :up(k, 128) // 128].int() - 127)
    f = torch.where(scale[:, :up(k, 128) // 128] == 255, torch.full_like(f, float("nan")), f)
    return q.view(torch.float8_e4m3fn).double() * spread(f, rows, n, k)


def rmsnorm(x, residual, gain, eps):
    """(h, y) with the operator's roundings: h in x's type, rstd once from 64 bits, y in float."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    ms = h.double().square().mean(dim=1, keepdim=True)
    rstd = (1.0 / torch.sqrt(ms + eps)).float()
    y = h.float() * rstd
    return h, y if gain is None else y * gain

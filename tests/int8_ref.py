"""8-bit integer matrices and products on them in 64 bits, for the tests.

codes: 127 x / amax to the nearest integer, ties to even, decided without
rounding: 127 x and amax are multiples of a common power of two, and twice the
remainder is compared with amax.
"""
import torch

import train_ref


def quantize(x):
    """x [rows, cols] -> (codes int8, scales float32); rows holding a NaN or an infinity get 0 and NaN."""
    b = x.double()
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, torch.zeros_like(b), b)
    amax = b.abs().amax(-1, keepdim=True)
    unit = torch.where(amax > 0, amax, torch.ones_like(amax))
    low = torch.floor(127.0 * b / unit)
    low = low + (127.0 * b - low * unit >= unit).double() - (127.0 * b - low * unit < 0).double()  # the exact floor
    twice = 2.0 * (127.0 * b - low * unit)
    q = low + ((twice > unit) | ((twice == unit) & (low.remainder(2.0) == 1.0))).double()
    s = (amax / 127.0).float()
    return q.to(torch.int8), torch.where(bad, torch.full_like(s, float("nan")), s).squeeze(-1)


def product(q, s, w, sw):
    """(value, bound) of s_r sw_n <q_r, w_n>: the products are exact, their float32
    sums too below 2^24 (above, the chain's bound), and two roundings scale them."""
    a, b = q.double(), w.double().t()
    v = a @ b
    size = a.abs() @ b.abs()
    slack = torch.where(size < 2.0 ** 24, torch.zeros_like(size), (a.shape[1] / 16 + 8) * train_ref.F32 * size)
    scale = s.double().unsqueeze(-1) * sw.double()
    return v * scale, slack * scale + 3 * 2.0 ** -24 * (v * scale).abs()


def down(q, s, w, sw):
    return train_ref.rounded(*product(q, s, w, sw))


def up(q, s, wg, sg, wu, su):
    """silu(g) u: the slope of silu is at most 1.1; the sigmoid's float32 form is off
    by at most (|g| + 8) 2^-23 of itself."""
    g, dg = product(q, s, wg, sg)
    u, du = product(q, s, wu, su)
    a = g * train_ref.sigmoid(g)
    da = 1.1 * dg + a.abs() * (g.abs() + 8) * train_ref.F32
    return train_ref.rounded(a * u, da * (u.abs() + du) + a.abs() * du + 3 * train_ref.F32 * (a * u).abs())

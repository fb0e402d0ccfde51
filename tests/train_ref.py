"""The experts' gated feed-forward and its backward pass in 64 bits, for the
tests: results, and for each a bound on what float32 sums and the roundings of
the outputs may change.

A sum of K products on the tensor cores is a chain of float32 additions, at most
K / 16 + 8 of them on any product's way, each off by at most 2^-23 of what it
adds up, which is at most the sum of the products' magnitudes.  A result in bf16
is off by at most 2^-8 of itself for its rounding.
"""
import numpy as np
import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -23


def sigmoid(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def product(a, b):
    """a @ b in float64 and the bound of its float32 sums."""
    return a @ b, (a.shape[-1] / 16 + 8) * F32 * (a.abs() @ b.abs())


def rounded(value, slack):
    """A bf16 result's value and bound."""
    return value, slack + BF16 * (value.abs() + slack) + 1e-38


def layout(counts):
    """(padded offsets [E + 1], capacity's shape (T, k, E))"""
    off = np.concatenate(([0], np.cumsum((np.asarray(counts) + 127) // 128 * 128)))
    return off.astype(np.int32), max(1, int(np.sum(counts)))


def forward(x, wg, wu, wd):
    """One expert: {name: (value, bound)} of g and u (inputs float64)."""
    return {"g": rounded(*product(x, wg)), "u": rounded(*product(x, wu))}


def down_backward(dy, wd, g, u):
    """dg, du.  The sigmoid is formed in float32 with a relative error of at most
    (|g| + 8) 2^-23 (the exponent's product rounded, exp and the division a few
    ulps), which reaches s (1 + g (1 - s)) as at most (1 + |g|) s (|g| + 12) 2^-22."""
    dh, slack = product(dy, wd.t())
    s = sigmoid(g)
    f = s * (1.0 + g * (1.0 - s))
    f_off = (1.0 + g.abs()) * s * (g.abs() + 12.0) * 2.0 ** -22
    gs_off = g.abs() * s * (g.abs() + 12.0) * 2.0 ** -22
    dg, du = dh * u * f, dh * g * s
    return {"dg": rounded(dg, u.abs() * (slack * (f.abs() + f_off) + dh.abs() * f_off) + 4 * F32 * dg.abs()),
            "du": rounded(du, slack * ((g * s).abs() + gs_off) + dh.abs() * gs_off + 4 * F32 * du.abs())}


def up_backward(dg, du, wg, wu):
    a = product(torch.cat((dg, du), -1), torch.cat((wg, wu), -1).t())
    return {"dx": rounded(*a)}


def weight_backward(x, h, dg, du, dy):
    return {"dwg": rounded(*product(x.t(), dg)), "dwu": rounded(*product(x.t(), du)),
            "dwd": rounded(*product(h.t(), dy))}


def check(got, want, what):
    value, bound = want
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d values off; first %s: %r, expected %r, off by %.3g of %.3g"
                             % (what, int(bad.sum()), bad.numel(), at, float(got[at]), float(value[at]),
                                float(err[at]), float(bound[at])))


def layer(logits, x, wg, wu, wd, k, picks=None):
    """The whole layer in float64 (autograd flows through it), its picks held."""
    if picks is None:
        picks = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(logits.gather(1, picks), -1)
    out = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        t, j = (picks == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g, u = x[t] @ wg[e], x[t] @ wu[e]
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u) @ wd[e] * w[t, j].unsqueeze(-1))
    return out

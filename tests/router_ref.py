"""The router's gradient of the layer in 64 bits, with a bound for every element.

With w the softmax of a token's picked logits and dw_j = <dout, Y_j>,
  dlogits[t, id_j] = w_j (dw_j - sum_l w_l dw_l)
is a difference of products, and its error is w_j (e_j - sum_l w_l e_l) with e_j that
of dw_j, which is w_j ((1 - w_j) e_j - sum over the other l of w_l e_l): at most
w_j ((1 - w_j) |e_j| + sum over the other l of w_l |e_l|).

e_j comes from two roundings to bf16, each by at most 2^-8 of its value: of h, which
reaches dw_j through the vector Wd dout, and of Y_j.  They are sums of as many
independent errors around zero, so (Hoeffding) six times 2^-8 of the norm of the terms
is passed with probability 2 exp(-18) < 4e-8 each, for the some 20000 sums of the
tests together less than 1e-3.  What the float32 sums and the float32 weights of the
routing add is bounded term by term.
"""
import torch

import train_ref

SIGMAS = 6.0
ULP = 2.0 ** -24


def picks_of(logits, k):
    return torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]


def gradient(logits, x, wg, wu, wd, dout, k):
    """dlogits [T, E] and its bound; float64 inputs that are the kernels' exactly."""
    T, E = logits.shape
    H, I = wg.shape[1], wg.shape[2]
    picks = picks_of(logits, k)
    leaf = logits.clone().requires_grad_()
    out = train_ref.layer(leaf, x, wg, wu, wd, k, picks)
    want, = torch.autograd.grad((out * dout).sum(), leaf)
    w = torch.softmax(logits.gather(1, picks), -1)
    dw, e = torch.zeros_like(w), torch.zeros_like(w)
    for n in range(E):
        t, j = (picks == n).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        g, g_off = train_ref.product(x[t], wg[n])
        u, u_off = train_ref.product(x[t], wu[n])
        a = g * train_ref.sigmoid(g)
        h = a * u
        # silu's slope is at most 1.1, its sigmoid off by at most (|g| + 12) 2^-22 of itself
        a_off = 1.1 * g_off + a.abs() * (g.abs() + 12.0) * 2.0 ** -22
        h_off = a_off * (u.abs() + u_off) + a.abs() * u_off + 4 * ULP * h.abs()
        y, y_off = train_ref.product(h, wd[n])
        back = dout[t] @ wd[n].t()  # how an error of h reaches dw
        d = dout[t]
        dw[t, j] = (y * d).sum(-1)
        random = ((y * d) ** 2).sum(-1) + ((h * back) ** 2).sum(-1)
        # a lane adds at most H / 32 products one by one, then 5 + 8 sums join the parts
        fixed = (h_off * back.abs()).sum(-1) + (y_off * d.abs()).sum(-1) + (H / 32 + 16) * ULP * (y * d).abs().sum(-1)
        e[t, j] = SIGMAS * train_ref.BF16 * random.sqrt() + 1.02 * fixed
    mean = (w * dw.abs()).sum(-1, keepdim=True)
    # float32 weights: exp, their sum and the division, 32 units in the last place
    off = w * ((1 - 2 * w) * e + (w * e).sum(-1, keepdim=True)) + 64 * ULP * w * (dw.abs() + 3 * mean)
    return want, torch.zeros_like(want).scatter_(1, picks, off)


def check(got, want, off, what="dlogits"):
    """Every element within its bound (0 where nothing was picked), and the bound says
    something: where a token has several picks it is well below the gradient."""
    several = (off > 0).sum(-1) > 1
    if several.any():
        assert float(off[several].norm()) <= 0.25 * float(want[several].norm()), "the bound says nothing"
    train_ref.check(got, (torch.where(off > 0, want, 0.0), off), what)

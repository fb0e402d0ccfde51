"""The check of the router's gradient, on the CPU: it takes the gradient itself and
refuses what a wrong kernel might give."""
import random

import pytest

torch = pytest.importorskip("torch")
import router_ref  # noqa: E402


def inputs(s, seed, skew=0.0):
    T, H, I, E, k = s
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    bias = -skew * torch.log(torch.arange(1, E + 1).float())
    return [t.double() for t in (normal(T, E) + bias, normal(T, H).bfloat16(), (normal(E, H, I) / H ** 0.5).bfloat16(),
                                 (normal(E, H, I) / H ** 0.5).bfloat16(), (normal(E, I, H) / I ** 0.5).bfloat16(),
                                 normal(T, H).bfloat16())]


def layer_in_bf16(i, k):
    """dlogits as the kernels form them: h and Y rounded to bf16, the rest in 32 bits."""
    logits, x, wg, wu, wd, dout = i
    picks = router_ref.picks_of(logits, k)
    w = torch.softmax(logits.gather(1, picks), -1).float()
    dw = torch.zeros_like(w)
    for e in range(wg.shape[0]):
        t, j = (picks == e).nonzero(as_tuple=True)
        g, u = (x[t] @ wg[e]).float(), (x[t] @ wu[e]).float()
        h = (g * torch.sigmoid(g) * u).bfloat16()
        y = (h.double() @ wd[e]).bfloat16()
        dw[t, j] = (y.float() * dout[t].float()).sum(-1)
    dl = w * (dw - (w * dw).sum(-1, keepdim=True))
    return torch.zeros(logits.shape).scatter_(1, picks, dl)


SHAPES = [((1, 256, 384, 8, 3), 0.0), ((128, 256, 512, 8, 2), 0.0), ((333, 384, 256, 16, 4), 0.0),
          ((64, 1152, 256, 64, 8), 0.0), ((200, 384, 384, 16, 5), 3.0)]


@pytest.mark.parametrize("s,skew", SHAPES, ids=str)
def test_it_takes_the_gradient_and_refuses_others(s, skew):
    k = s[4]
    i = inputs(s, 1, skew)
    want, off = router_ref.gradient(*i, k)
    got = layer_in_bf16(i, k)
    router_ref.check(got, want, off)
    wrong = {"zero": torch.zeros_like(got), "negative": -got, "half": got / 2}
    rows = random.Random(0).sample(range(s[0]), min(3, s[0]))
    for r in rows:
        missing = got.clone()
        missing[r] = 0
        wrong["token %d missing" % r] = missing
        shifted = got.clone()
        shifted[r] = got[r].roll(1)
        wrong["token %d at its neighbours' experts" % r] = shifted
    one = got.clone()
    one.view(-1)[one.abs().argmax()] = 0
    wrong["its largest element missing"] = one
    for name, bad in wrong.items():
        with pytest.raises(AssertionError):
            router_ref.check(bad, want, off, name)


def test_one_pick_has_no_gradient():
    i = inputs((40, 128, 128, 4, 1), 2)
    want, off = router_ref.gradient(*i, 1)
    assert float(want.abs().max()) < 1e-12
    router_ref.check(layer_in_bf16(i, 1), want, off)

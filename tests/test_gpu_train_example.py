"""The example that trains a layer and serves it in 8-bit integers: it runs, and the
gradients that its torch function gives are the 64-bit layer's."""
import os
import sys

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import train_ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    need_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_layer
    finally:
        sys.path.pop(0)
    return train_layer


def test_it_runs(example):
    history, off = example.main(tokens=300, steps=3)
    assert len(history) == 3
    for loss, grads in history:
        assert loss == loss and all(bool(g.isfinite().all()) and bool(g.any()) for g in grads)
    assert off <= 0.05  # what 8 bits may cost: see test_gpu_int8.test_forward


def test_its_gradients(example):
    """Through the function, a router before it and two layers in a row (each keeps
    its own workspace until its backward)."""
    s = (200, 256, 384, 8, 2)
    T, H, I, E, k = s
    gen = torch.Generator(device="cuda").manual_seed(4)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x = normal(T, H).bfloat16()
    routers = [normal(T, E) for _ in range(2)]
    weights = [[(normal(E, K, N) / K ** 0.5).bfloat16() for K, N in ((H, I), (H, I), (I, H))] for _ in range(2)]
    dout = normal(T, H).bfloat16()
    leaves = [t.requires_grad_() for t in (x, *routers, *weights[0], *weights[1])]
    mid = example.ExpertLayer.apply(s, routers[0], x, *weights[0])
    out = example.ExpertLayer.apply(s, routers[1], mid, *weights[1])
    got = torch.autograd.grad(out, leaves, dout)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    m = train_ref.layer(wide[1], wide[0], *wide[3:6], k)
    o = train_ref.layer(wide[2], m, *wide[6:9], k)
    want = torch.autograd.grad(o, wide, dout.double())
    # the roundings of one layer's pass (see test_gpu_train) twice over
    most = 14 * train_ref.BF16
    for i, (g, w) in enumerate(zip(got, want)):
        norm = float(w.norm())
        if i in (1, 2):  # differences of products: on their scale
            o_, d_ = (m, torch.autograd.grad(train_ref.layer(wide[2], m, *wide[6:9], k), m, dout.double(), retain_graph=True)[0]) \
                if i == 1 else (o, dout.double())
            norm = float((d_.norm(dim=-1) * o_.detach().norm(dim=-1)).norm()) * 2 * k
        assert float((g.double() - w).norm()) <= most * norm, i

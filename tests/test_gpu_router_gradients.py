"""The router's gradient of the layer and of the example's torch function, element by
element, and the layer's gradients against differences along the 64-bit gradient of a
part of the tokens or experts, so that what is missing in a part shows."""
import os
import random
import sys

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import router_ref  # noqa: E402
import train_ref  # noqa: E402
from test_gpu_train import Layer, layer_inputs  # noqa: E402

NAMES = ("logits", "X", "wg", "wu", "wd")
SHAPES = [(1, 128, 128, 1, 1), (1, 256, 384, 8, 3), (128, 256, 512, 8, 2), (333, 384, 256, 16, 4),
          (700, 640, 384, 3, 1), (64, 1152, 256, 64, 8), (40, 256, 128, 256, 16)]


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


def run(moe, s, i):
    lay = Layer(moe, s)
    lay.forward(i)
    lay.backward(i)
    assert lay.status() == (0, 0)
    return lay


@pytest.mark.parametrize("s", SHAPES, ids=str)
def test_every_element(moe, s):
    i = layer_inputs(*s)
    lay = run(moe, s, i)
    want = router_ref.gradient(*(i[n].double() for n in (*NAMES, "dout")), s[4])
    router_ref.check(lay.dlogits, *want)


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(moe, seed):
    rng = random.Random(100 + seed)
    E = rng.choice([2, 3, 17, 64, 256])
    k = rng.randint(2, min(E, 16))
    s = (int(2 ** rng.uniform(0, 8)), 128 * rng.randint(1, 9), 128 * rng.randint(1, 6), E, k)
    i = layer_inputs(*s, seed=seed)
    i["logits"] += rng.choice([0.0, 3.0]) * -torch.log(torch.arange(1, E + 1, device="cuda").float())
    lay = run(moe, s, i)
    want = router_ref.gradient(*(i[n].double() for n in (*NAMES, "dout")), k)
    router_ref.check(lay.dlogits, *want)


@pytest.mark.parametrize("s", SHAPES[2:4], ids=str)
def test_parts_against_differences(moe, s):
    """A part's direction is the 64-bit layer's gradient there.  The gradient's product
    with it against the central difference along it: off by at most the sum of the
    elements' bounds for the logits, and by the part's share of the layer's seven
    roundings for the rest (see test_gpu_train)."""
    T, H, I, E, k = s
    i = layer_inputs(*s, seed=4)
    lay = run(moe, s, i)
    wide = {n: i[n].double() for n in NAMES}
    dout = i["dout"].double()
    picks = router_ref.picks_of(wide["logits"], k)
    off = router_ref.gradient(*wide.values(), dout, k)[1]
    leaves = [wide[n].clone().requires_grad_() for n in NAMES]
    true = torch.autograd.grad((train_ref.layer(*leaves, k, picks) * dout).sum(), leaves)
    for n, got, grad in zip(NAMES, (lay.dlogits, lay.dX, lay.dwg, lay.dwu, lay.dwd), true):
        for part in range(8):
            v = torch.zeros_like(grad)
            v[part::8] = grad[part::8]
            v /= v.norm()
            eps, f = 1e-4, []
            for step in (eps, -eps):
                moved = [wide[m] + step * v if m == n else wide[m] for m in NAMES]
                f.append(float((train_ref.layer(*moved, k, picks) * dout).sum()))
            diff = (f[0] - f[1]) / (2 * eps)
            along = float((got.double() * v).sum())
            most = float((off * v.abs()).sum()) if n == "logits" else 7 * train_ref.BF16 * abs(diff)
            assert most <= 0.25 * abs(diff), (n, part)
            assert abs(along - diff) <= most + 1e-6 * abs(diff), (n, part, along, diff)


def test_the_function_in_the_example(moe):
    """Two layers in a row: each router's gradient is that of its own layer, on the
    tokens and the output gradient that the function itself passed on."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        from train_layer import ExpertLayer
    finally:
        sys.path.pop(0)
    s = (200, 256, 384, 8, 2)
    a, b = layer_inputs(*s, seed=1), layer_inputs(*s, seed=2)
    first, second = ([t.requires_grad_() for t in (i["logits"], i["wg"], i["wu"], i["wd"])] for i in (a, b))
    x = a["X"].requires_grad_()
    mid = ExpertLayer.apply(s, first[0], x, *first[1:])
    out = ExpertLayer.apply(s, second[0], mid, *second[1:])
    d1, d2, dmid = torch.autograd.grad(out, [first[0], second[0], mid], b["dout"])
    for got, leaf, tokens, weights, dout in ((d1, first[0], x, first[1:], dmid),
                                             (d2, second[0], mid, second[1:], b["dout"])):
        want = router_ref.gradient(*(t.detach().double() for t in (leaf, tokens, *weights, dout)), s[4])
        router_ref.check(got, *want)

"""Training steps and 8-bit forwards queued without waiting, with inputs that change in
place, of random shapes, on two streams at once, and together as they are used: a
layer trained for some steps, its weights quantised, the 8-bit layer run on them."""
import random

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import train_ref  # noqa: E402
from test_gpu_train import Layer, layer_inputs  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


def quantized(moe, w):
    E, K, N = w.shape
    pair = moe.alloc_int8(E * N, K)
    moe.moe_quantize_weights_int8(w, E, K, N, *pair)
    return pair


@pytest.mark.parametrize("s", [(1, 256, 256, 4, 2), (200, 384, 256, 16, 4), (2000, 512, 384, 8, 2)], ids=str)
def test_steps_queued_over_the_same_buffers(moe, s):
    """Inputs copied into place between steps on the stream, nothing waited for: each
    step's results are those of the step alone."""
    sets = [layer_inputs(*s, seed=i) for i in range(3)]
    lay = Layer(moe, s)
    w8 = [t for n in ("wg", "wu", "wd") for t in quantized(moe, sets[0][n])]
    ws8, out8 = moe.alloc_int8_workspace(s), torch.empty_like(lay.out)
    held = {n: t.clone() for n, t in sets[0].items()}

    def step():
        lay.forward(held)
        lay.backward(held)
        moe.moe_forward_int8(s, held["logits"], held["X"], *w8, out8, ws8)
        return [t.clone() for t in (*lay.results(), out8)]

    want = []
    for i in sets:
        for n in held:
            held[n].copy_(i[n])
        want.append(step())
        torch.cuda.synchronize()
    order = [0, 1, 2, 1, 0, 2, 2, 0] * 3
    got = []
    for i in order:
        for n in held:
            held[n].copy_(sets[i][n])
        got.append(step())
    torch.cuda.synchronize()
    for i, g in zip(order, got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i]))
    assert lay.status() == (0, 0) and moe.last_device_status(ws8) == 0


def test_two_streams_at_once(moe):
    s = (600, 512, 384, 8, 2)
    inputs = [layer_inputs(*s, seed=i) for i in (1, 2)]
    layers = [Layer(moe, s) for _ in inputs]
    want = []
    for lay, i in zip(layers, inputs):
        lay.forward(i)
        lay.backward(i)
        want.append([t.clone() for t in lay.results()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(5):
        for lay, i, st in zip(layers, inputs, streams):
            with torch.cuda.stream(st):
                lay.forward(i)
                lay.backward(i)
    torch.cuda.synchronize()
    for lay, w in zip(layers, want):
        assert all(torch.equal(x, y) for x, y in zip(lay.results(), w))
        assert lay.status() == (0, 0)


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(moe, seed):
    """The layer's gradients and its 8-bit output on shapes of the whole range, skewed
    routers among them (bounds as in test_gpu_train and test_gpu_int8)."""
    rng = random.Random(seed)
    E = rng.choice([1, 2, 3, 17, 64, 256])
    k = rng.randint(1, min(E, 16))
    s = (int(2 ** rng.uniform(0, 10)), 128 * rng.randint(1, 9), 128 * rng.randint(1, 6), E, k)
    i = layer_inputs(*s, seed=seed)
    i["logits"] += rng.choice([0.0, 3.0]) * -torch.log(torch.arange(1, E + 1, device="cuda").float())
    lay = Layer(moe, s)
    lay.forward(i)
    lay.backward(i)
    assert lay.status() == (0, 0)
    leaves = [i[n].double().requires_grad_() for n in ("logits", "X", "wg", "wu", "wd")]
    out = train_ref.layer(*leaves, k)
    grads = torch.autograd.grad((out * i["dout"].double()).sum(), leaves)
    for name, got, want in zip(("out", "dX", "dwg", "dwu", "dwd"), (lay.out, lay.dX, lay.dwg, lay.dwu, lay.dwd),
                               (out.detach(), *grads[1:])):
        assert float((got.double() - want).norm()) <= 7 * train_ref.BF16 * float(want.norm()), (s, name)
    scale = (i["dout"].double().norm(dim=-1) * out.detach().norm(dim=-1)).norm() * 2 * k
    assert float((lay.dlogits.double() - grads[0]).norm()) <= 7 * train_ref.BF16 * float(scale), s
    w8 = [t for n in ("wg", "wu", "wd") for t in quantized(moe, i[n])]
    ws8, out8 = moe.alloc_int8_workspace(s), torch.empty_like(lay.out)
    moe.moe_forward_int8(s, i["logits"], i["X"], *w8, out8, ws8)
    assert moe.last_device_status(ws8) == 0
    assert float((out8.double() - out.detach()).norm()) <= 0.05 * float(out.detach().norm()), s


def test_trained_then_served_in_8_bits(moe):
    """Some steps of gradient descent on the layer's weights (each step's gradients
    against the 64-bit layer's), then the 8-bit layer on what they left."""
    s = (256, 256, 384, 8, 2)
    T, H, I, E, k = s
    i = layer_inputs(*s, seed=11)
    target = layer_inputs(*s, seed=12)["X"]
    lay = Layer(moe, s)
    for step in range(3):
        lay.forward(i)
        i["dout"] = ((lay.out.float() - target.float()) / T).bfloat16()
        lay.backward(i)
        leaves = [i[n].double().requires_grad_() for n in ("logits", "X", "wg", "wu", "wd")]
        out = train_ref.layer(*leaves, k)
        grads = torch.autograd.grad((out * i["dout"].double()).sum(), leaves)
        for name, got, want in zip(("wg", "wu", "wd"), (lay.dwg, lay.dwu, lay.dwd), grads[2:]):
            assert float((got.double() - want).norm()) <= 7 * train_ref.BF16 * float(want.norm()), (step, name)
        for name, grad in (("wg", lay.dwg), ("wu", lay.dwu), ("wd", lay.dwd)):
            i[name] = (i[name].float() - 0.5 * grad.float()).bfloat16()
    assert lay.status() == (0, 0)
    lay.forward(i)
    w8 = [t for n in ("wg", "wu", "wd") for t in quantized(moe, i[n])]
    ws8, out8 = moe.alloc_int8_workspace(s), torch.empty_like(lay.out)
    moe.moe_forward_int8(s, i["logits"], i["X"], *w8, out8, ws8)
    assert moe.last_device_status(ws8) == 0
    assert float((out8.float() - lay.out.float()).norm()) <= 0.05 * float(lay.out.float().norm())

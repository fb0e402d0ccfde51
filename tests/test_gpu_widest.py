"""The training and 8-bit calls at the ends of the supported sizes: the widest rows and
weights (32768), and the layer with the most tokens, experts and picks at once."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import test_gpu_int8 as int8  # noqa: E402
import test_gpu_train as train  # noqa: E402
import train_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    yield m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("size", [(32768, 128), (128, 32768), (32640, 256)], ids=lambda s: "%dx%d" % s)
def test_widest_rows(moe, size):
    counts = [5, 0, 130]
    for test in (train.test_down_backward, train.test_up_backward, train.test_weight_backward, train.test_up_train):
        test(moe, counts, size)
    for up in (True, False):
        int8.test_products(moe, up, counts, size)
        int8.test_products(moe, up, [1, 1], size)
    E, N = 2, size[1]
    int8.test_quantize_weights(moe, (E, size[0], N))


def test_most_tokens_experts_and_picks(moe):
    """2^22 tokens of 16 of 256 experts: 2^26 rows.  Output and gradients of tokens from
    all over the batch against the 64-bit layer on those tokens (a token's are its own),
    each on the scale of its norm (the roundings of test_gpu_train), and the 8-bit
    layer's."""
    T, H, I, E, k = s = (1 << 22, 128, 128, 256, 16)
    i = train.layer_inputs(*s)
    lay = train.Layer(moe, s)
    lay.forward(i)
    lay.backward(i)
    assert lay.status() == (0, 0)
    rows = torch.cat([torch.arange(a, a + 8, device="cuda") for a in (0, 12345, T // 2 - 4, T - 8)])
    w = [i[n].double() for n in ("wg", "wu", "wd")]
    logits, x = i["logits"][rows].double(), i["X"][rows].double().requires_grad_()
    out = ref.layer(logits, x, *w, k)
    dx, = torch.autograd.grad((out * i["dout"][rows].double()).sum(), x)
    for name, got, want in (("out", lay.out[rows], out.detach()), ("dX", lay.dX[rows], dx)):
        assert float((got.double() - want).norm()) <= 7 * ref.BF16 * float(want.norm()), name
    import router_ref
    router_ref.check(lay.dlogits[rows], *router_ref.gradient(logits, x.detach(), *w, i["dout"][rows].double(), k))
    # one expert's weight gradients, from the rows as the forward and backward left them
    picks = router_ref.picks_of(i["logits"], k)
    t, j = (picks == E - 1).nonzero(as_tuple=True)
    del picks
    p = torch.softmax(i["logits"][t].double().sort(-1, descending=True).values[:, :k], -1)
    xe, dy = i["X"][t].double(), i["dout"][t].double() * p.gather(1, j.unsqueeze(1))
    g, u = xe @ w[0][-1], xe @ w[1][-1]
    sg = ref.sigmoid(g)
    dh = dy @ w[2][-1].t()
    wants = (xe.t() @ (dh * u * sg * (1 + g * (1 - sg))), xe.t() @ (dh * g * sg), (g * sg * u).t() @ dy)
    for name, got, want in zip(("dwg", "dwu", "dwd"), (lay.dwg[-1], lay.dwu[-1], lay.dwd[-1]), wants):
        assert float((got.double() - want).norm()) <= 7 * ref.BF16 * float(want.norm()), name
    del xe, dy, g, u, sg, dh
    lay.g = lay.u = lay.bws = None
    w8 = [t for n in ("wg", "wu", "wd") for t in int8.quantized(moe, i[n])]
    ws8 = moe.alloc_int8_workspace(s)
    moe.moe_forward_int8(s, i["logits"], i["X"], *w8, lay.out, ws8)
    assert moe.last_device_status(ws8) == 0
    assert float((lay.out[rows].double() - out.detach()).norm()) <= 0.05 * float(out.detach().norm())

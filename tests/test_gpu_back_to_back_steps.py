"""The layer's step calls, bf16 and MXFP4, queued back to back over one set of
buffers, and calls whose inputs are written in place between them: each kernel
may be resident while earlier ones of the queue still run, and has to see what
the last one before it wrote."""
import pytest

from gpu_util import need_gpu
from test_gpu_back_to_back import queue

pytestmark = pytest.mark.gpu

SHAPES = [(8, 256, 256, 8, 2), (200, 512, 384, 16, 4), (1500, 256, 256, 4, 2), (640, 4096, 256, 8, 3)]


def weights(s, gen):
    import torch
    import combine_moe_route_04_gb300 as moe
    T, H, I, E, k = s
    w = [(torch.randn((E, K, N), generator=gen, device="cuda") / K ** 0.5).bfloat16()
         for K, N in ((H, I), (H, I), (I, H))]
    q = []
    for x in w:
        codes, scales = moe.alloc_mxfp4(E * x.shape[2], x.shape[1])
        moe.moe_quantize_weights_mxfp4(x, E, x.shape[1], x.shape[2], codes, scales)
        q += [codes, scales]
    return w, q


def sources(s, gen):
    import torch
    T, H, I, E, k = s
    return [(torch.randn((T, E), generator=gen, device="cuda") - torch.arange(E, device="cuda") * 0.3 * i,
             torch.randn((T, H), generator=gen, device="cuda").bfloat16()) for i in range(3)]


class Layer:
    """The step calls of one shape over one set of buffers."""

    def __init__(self, s, mxfp4, gen):
        import torch
        import combine_moe_route_04_gb300 as moe
        T, H, I, E, k = s
        self.s, self.moe, self.mxfp4 = s, moe, mxfp4
        self.mr = moe.capacity(s)[1]
        self.w, self.q = weights(s, gen)
        self.r = moe.alloc_route_outputs(s)
        self.ws = moe.alloc_workspace(s)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        # padding rows are not written by every call: fixed values there
        self.h, self.Y = torch.zeros((self.mr, I), **bf16), torch.zeros((self.mr, H), **bf16)
        self.x4 = [t.zero_() for t in moe.alloc_mxfp4(self.mr, H)]
        self.h4 = [t.zero_() for t in moe.alloc_mxfp4(self.mr, I)]

    def route(self, logits):
        r = self.r
        self.moe.moe_route(self.s, logits, r["topk_ids"], r["topk_w"], r["counts"], r["off_pad"], r["block_expert"],
                           r["num_blocks"], r["gather_idx"], r["scatter_idx"], self.ws)

    def up(self, x):
        m, r = self.moe, self.r
        if self.mxfp4:
            m.moe_quantize_permute_mxfp4(self.s, x, r["scatter_idx"], *self.x4, self.ws)
            m.moe_grouped_gemm_up_mxfp4(self.s, *self.x4, r["counts"], r["off_pad"], *self.q[:4], self.h, self.ws)
            m.moe_quantize_mxfp4(self.h, self.mr, self.s[2], *self.h4)
        else:
            m.moe_grouped_gemm_up(self.s, x, r["scatter_idx"], r["counts"], r["off_pad"], *self.w[:2], self.h, self.ws)

    def down(self, h=None):
        m, r = self.moe, self.r
        if self.mxfp4:
            m.moe_grouped_gemm_down_mxfp4(self.s, *(h or self.h4), r["counts"], r["off_pad"], *self.q[4:], self.Y,
                                          self.ws)
        else:
            m.moe_grouped_gemm_down(self.s, self.h if h is None else h, r["counts"], r["off_pad"], self.w[2], self.Y,
                                    self.ws)

    def combine(self, out):
        self.moe.moe_combine(self.s, self.Y, self.r["scatter_idx"], self.r["topk_w"], out, self.ws)


def differing(views, want):
    import torch
    return [i for i in range(len(views)) if not torch.equal(views[i], want[i % len(want)])][:10]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("s", SHAPES)
def test_steps_over_one_set_of_buffers(s, mxfp4, graph):
    torch = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(s[0])
    layer, src, n = Layer(s, mxfp4, gen), sources(s, gen), 60

    def step(i, out):
        logits, x = src[i % 3]
        layer.route(logits)
        layer.up(x)
        layer.down()
        layer.combine(out)

    outs = torch.zeros((n + 3, s[0], s[1]), dtype=torch.bfloat16, device="cuda")
    views = [outs[i] for i in range(n)]
    want = [outs[n + i] for i in range(3)]
    for i in range(3):
        step(i, want[i])
        torch.cuda.synchronize()
    queue(lambda: [step(i, views[i]) for i in range(n)], graph)
    assert layer.moe.last_device_status(layer.ws) == 0
    assert all(w.abs().sum() > 0 for w in want)
    assert not differing(views, want)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("s", SHAPES)
def test_down_and_combine_over_one_y(s, mxfp4, graph):
    """down, combine, down, combine ...: nothing between the combine that reads Y
    and the product that writes it anew."""
    torch = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(s[0] + 1)
    layer, n = Layer(s, mxfp4, gen), 120
    layer.route(sources(s, gen)[0][0])
    hs = []
    for _ in range(3):
        h = torch.randn((layer.mr, s[2]), generator=gen, device="cuda").bfloat16()
        if mxfp4:
            q = layer.moe.alloc_mxfp4(layer.mr, s[2])
            layer.moe.moe_quantize_mxfp4(h, layer.mr, s[2], *q)
            h = q
        hs.append(h)
    outs = torch.zeros((n + 3, s[0], s[1]), dtype=torch.bfloat16, device="cuda")
    views, want = [outs[i] for i in range(n)], [outs[n + i] for i in range(3)]

    def step(i, out):
        layer.down(hs[i % 3])
        layer.combine(out)

    for i in range(3):
        step(i, want[i])
        torch.cuda.synchronize()
    queue(lambda: [step(i, views[i]) for i in range(n)], graph)
    assert layer.moe.last_device_status(layer.ws) == 0
    assert not differing(views, want)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("s", SHAPES)
def test_forward_of_tokens_and_logits_written_in_place(s, mxfp4, graph):
    """X and the logits are rewritten between forwards, X by a kernel of this
    library (which lets the forward launch early), the logits by torch."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, I, E, k = s
    gen = torch.Generator(device="cuda").manual_seed(T + 2)
    (w, q), src, n = weights(s, gen), sources(s, gen), 60
    ws = moe.alloc_mxfp4_workspace(s) if mxfp4 else moe.alloc_workspace(s)
    packed = []
    for _, x in src:
        packed.append(moe.alloc_mxfp4(T, H))
        moe.moe_quantize_mxfp4(x, T, H, *packed[-1])
    X, L = torch.zeros_like(src[0][1]), torch.zeros_like(src[0][0])
    outs = torch.zeros((n + 3, T, H), dtype=torch.bfloat16, device="cuda")
    views, want = [outs[i] for i in range(n)], [outs[n + i] for i in range(3)]

    def step(i, out):
        L.copy_(src[i % 3][0])
        moe.moe_dequantize_mxfp4(*packed[i % 3], T, H, X)
        if mxfp4:
            moe.moe_forward_mxfp4(s, L, X, *q, out, ws)
        else:
            moe.moe_forward(s, L, X, *w, out, ws)

    for i in range(3):
        step(i, want[i])
        torch.cuda.synchronize()
    queue(lambda: [step(i, views[i]) for i in range(n)], graph)
    assert moe.last_device_status(ws) == 0
    assert not differing(views, want)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,E,k", [(16, 8, 2), (600, 37, 3), (3000, 256, 8)])
def test_balance_of_logits_and_mask_written_in_place(T, E, k, graph):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (T, 128, 128, E, k)
    gen = torch.Generator(device="cuda").manual_seed(T)
    n = 100
    src = []
    for i in range(3):
        logits = torch.randn((T, E), generator=gen, device="cuda") * (1 + i)
        src.append((logits, logits.topk(k, dim=1).indices.int().contiguous(),
                    torch.rand(T, generator=gen, device="cuda") < 0.3 * (1 + i)))
    L, ids, mask = (torch.zeros_like(t) for t in src[0])
    counts, num = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, grad = torch.zeros(E, device="cuda"), torch.tensor([1.0, 0.5], device="cuda")
    losses, d = torch.zeros(2, device="cuda"), torch.zeros((T, E), device="cuda")
    ws = moe.alloc_balance_workspace(s)
    got = torch.zeros((n + 3, T * E + 2), device="cuda")
    views, want = [got[i] for i in range(n)], [got[n + i] for i in range(3)]

    def step(i, out):
        for a, b in zip((L, ids, mask), src[i % 3]):
            a.copy_(b)
        moe.moe_balance_loss(s, L, ids, mask, counts, num, P, losses, ws)
        moe.moe_balance_loss_backward(s, L, mask, counts, num, grad, d)
        out[:2].copy_(losses)
        out[2:].copy_(d.view(-1))

    for i in range(3):
        step(i, want[i])
        torch.cuda.synchronize()
    queue(lambda: [step(i, views[i]) for i in range(n)], graph)
    assert moe.last_device_status(ws) == 0
    assert not differing(views, want)

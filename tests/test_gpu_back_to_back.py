"""MXFP4 and balance calls queued back to back on the same buffers with changing
inputs: every kernel may be launched while earlier ones of the chain still run,
and has to see what the last one before it wrote."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROUNDS = 300


def queue(calls, graph):
    """Runs calls() from the host, or as one replay of a CUDA graph, which leaves no
    gaps between the kernels."""
    torch = need_gpu()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        g.replay()
    else:
        calls()
    torch.cuda.synchronize()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("rows,cols", [(8, 256), (40, 1024), (700, 2048), (4096, 4096)])
def test_quantize_and_back_over_one_pair_of_buffers(rows, cols, graph):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = ROUNDS if rows < 4096 else 40
    src = [torch.randn((rows, cols), generator=g, device="cuda").bfloat16() * 4.0 ** i for i in range(3)]
    codes, scales = moe.alloc_mxfp4(rows, cols)
    want = []
    for x in src:
        moe.moe_quantize_mxfp4(x, rows, cols, codes, scales)
        out = torch.empty_like(x)
        moe.moe_dequantize_mxfp4(codes, scales, rows, cols, out)
        torch.cuda.synchronize()
        want.append(out)
    outs = torch.zeros((n, rows, cols), dtype=torch.bfloat16, device="cuda")
    views = [outs[i] for i in range(n)]

    def calls():
        for i in range(n):
            moe.moe_quantize_mxfp4(src[i % 3], rows, cols, codes, scales)
            moe.moe_dequantize_mxfp4(codes, scales, rows, cols, views[i])

    queue(calls, graph)
    bad = [i for i in range(n) if not torch.equal(views[i], want[i % 3])]
    assert not bad, bad[:10]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,E,k", [(16, 8, 2), (600, 37, 3), (3000, 256, 8), (30000, 64, 4)])
def test_balance_over_one_set_of_buffers(T, E, k, graph):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (T, 128, 128, E, k)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = ROUNDS if T < 30000 else 60
    src = []
    for i in range(3):
        logits = torch.randn((T, E), generator=g, device="cuda") * (1 + i) + torch.arange(E, device="cuda") * 0.02 * i
        src.append((logits, logits.topk(k, dim=1).indices.int().contiguous(),
                    torch.rand(T, generator=g, device="cuda") < 0.3 * (1 + i)))
    counts, num = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, grad = torch.zeros(E, device="cuda"), torch.tensor([1.0, 0.5], device="cuda")
    ws = moe.alloc_balance_workspace(s)

    def step(i, losses, d):
        logits, ids, mask = src[i % 3]
        moe.moe_balance_loss(s, logits, ids, mask, counts, num, P, losses, ws)
        moe.moe_balance_loss_backward(s, logits, mask, counts, num, grad, d)

    want = []
    for i in range(3):
        losses, d = torch.zeros(4, device="cuda"), torch.zeros((T, E), device="cuda")
        step(i, losses, d)
        torch.cuda.synchronize()
        want.append((losses, d))
    losses = torch.zeros((n, 4), device="cuda")
    d = torch.zeros((n, T, E), device="cuda")
    views = [(losses[i], d[i]) for i in range(n)]
    if (T * E) % 4:
        d = torch.zeros((n, T * E + 4), device="cuda")
        views = [(losses[i], d[i][:T * E]) for i in range(n)]
        assert all(v[1].data_ptr() % 16 == 0 for v in views)
    queue(lambda: [step(i, *views[i]) for i in range(n)], graph)
    assert moe.last_device_status(ws) == 0
    bad = [i for i in range(n) if not (torch.equal(views[i][0], want[i % 3][0])
                                       and torch.equal(views[i][1].reshape(T, E), want[i % 3][1]))]
    assert not bad, bad[:10]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", [(8, 256, 256, 8, 2), (200, 512, 384, 16, 4), (1500, 256, 256, 4, 2)])
def test_forwards_over_one_workspace(T, H, I, E, k, graph):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (T, H, I, E, k)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = 100
    q = []
    for K, N in ((H, I), (H, I), (I, H)):
        w = (torch.randn((E, K, N), generator=g, device="cuda") / K ** 0.5).bfloat16()
        codes, scales = moe.alloc_mxfp4(E * N, K)
        moe.moe_quantize_weights_mxfp4(w, E, K, N, codes, scales)
        q += [codes, scales]
    src = [(torch.randn((T, E), generator=g, device="cuda") - torch.arange(E, device="cuda") * 0.3 * i,
            torch.randn((T, H), generator=g, device="cuda").bfloat16()) for i in range(3)]
    ws = moe.alloc_mxfp4_workspace(s)
    want = []
    for logits, x in src:
        out = torch.empty_like(x)
        moe.moe_forward_mxfp4(s, logits, x, *q, out, ws)
        torch.cuda.synchronize()
        want.append(out)
    outs = torch.zeros((n, T, H), dtype=torch.bfloat16, device="cuda")
    views = [outs[i] for i in range(n)]
    queue(lambda: [moe.moe_forward_mxfp4(s, *src[i % 3], *q, views[i], ws) for i in range(n)], graph)
    assert moe.last_device_status(ws) == 0
    bad = [i for i in range(n) if not torch.equal(views[i], want[i % 3])]
    assert not bad, bad[:10]

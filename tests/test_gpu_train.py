"""The backward pass of the experts' products, of the combine and of the layer
against 64-bit references, on ragged counts, with padding rows that hold NaN and
outputs whose padding must stay as it was."""
import numpy as np
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import train_ref as ref  # noqa: E402

MARK = -7.5  # what output padding holds before and after


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


class Rows:
    """Random rows in expert order for the given counts."""

    def __init__(self, moe, counts, H, I, seed=0, scale=1.0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.counts, self.H, self.I, self.E = list(counts), H, I, len(counts)
        off, T = ref.layout(counts)
        self.s = moe.shape(T, H, I, self.E, 1)
        self.R = moe.capacity(self.s)[1]
        self.off = off
        self.d_counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.d_off = torch.from_numpy(off).cuda()
        self.real = torch.zeros(self.R, dtype=torch.bool, device="cuda")
        for e, c in enumerate(counts):
            self.real[off[e]:off[e] + c] = True
        self.x = self.rows(H)
        self.g, self.u = self.rows(I, 2.0), self.rows(I)
        self.h = self.rows(I)
        self.dy = self.rows(H, scale)
        self.dg, self.du = self.rows(I), self.rows(I)
        self.wg, self.wu = self.weights(H, I), self.weights(H, I)
        self.wd = self.weights(I, H)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def rows(self, cols, scale=1.0):
        v = (self.normal(self.R, cols) * scale).bfloat16()
        v[~self.real] = float("nan")
        return v

    def weights(self, K, N):
        return (self.normal(self.E, K, N) / K ** 0.5).bfloat16()

    def out(self, cols):
        return torch.full((self.R, cols), MARK, dtype=torch.bfloat16, device="cuda")

    def spans(self):
        for e, c in enumerate(self.counts):
            yield e, slice(int(self.off[e]), int(self.off[e]) + c)

    def done(self, moe, *outs):
        assert moe.last_device_status(self.ws) == 0
        assert int(self.ws[:256].sum()) == 0  # counters cleared for the next call
        for o in outs:
            assert (o[~self.real] == MARK).all(), "padding rows were written"


COUNTS = [
    [1],
    [5, 0, 1],
    [128],
    [16, 32, 48],
    [129, 127, 0, 64, 65],
    [255, 256, 257, 0, 3],
    [0, 0, 300, 0],
    [513, 31, 15, 17],
    [1000],
]
SIZES = [(128, 128), (256, 384), (640, 256), (384, 640)]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_down_backward(moe, counts, size):
    r = Rows(moe, counts, *size)
    dg, du = r.out(r.I), r.out(r.I)
    moe.moe_grouped_gemm_down_backward(r.s, r.dy, r.d_counts, r.d_off, r.wd, r.g, r.u, dg, du, r.ws)
    r.done(moe, dg, du)
    for e, at in r.spans():
        want = ref.down_backward(*(t.double() for t in (r.dy[at], r.wd[e], r.g[at], r.u[at])))
        ref.check(dg[at], want["dg"], "dg of expert %d" % e)
        ref.check(du[at], want["du"], "du of expert %d" % e)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_up_backward(moe, counts, size):
    r = Rows(moe, counts, *size)
    dx = r.out(r.H)
    moe.moe_grouped_gemm_up_backward(r.s, r.dg, r.du, r.d_counts, r.d_off, r.wg, r.wu, dx, r.ws)
    r.done(moe, dx)
    for e, at in r.spans():
        want = ref.up_backward(*(t.double() for t in (r.dg[at], r.du[at], r.wg[e], r.wu[e])))
        ref.check(dx[at], want["dx"], "dX of expert %d" % e)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_weight_backward(moe, counts, size):
    r = Rows(moe, counts, *size)
    dw = [torch.full_like(w, MARK) for w in (r.wg, r.wu, r.wd)]
    moe.moe_grouped_gemm_weight_backward(r.s, r.x, r.h, r.dg, r.du, r.dy, r.d_counts, r.d_off, *dw, r.ws)
    r.done(moe)
    for e, at in r.spans():
        want = ref.weight_backward(*(t[at].double() for t in (r.x, r.h, r.dg, r.du, r.dy)))
        for name, w in zip(("dwg", "dwu", "dwd"), dw):
            ref.check(w[e], want[name], "%s of expert %d" % (name, e))


# row counts around the ends of MMA steps (16), of stages (64) and of what stays in
# shared memory for a run (320), long ones between
RUN_COUNTS = [0, 1, 7, 16, 17, 63, 64, 65, 130, 0, 255, 256, 257, 300, 319, 320, 321, 15, 700, 335, 384, 2]


@pytest.mark.parametrize("size", [(256, 1280), (640, 384), (128, 2176), (1152, 256)], ids=lambda s: "%dx%d" % s)
def test_weight_backward_in_runs(moe, size):
    """Gradient tiles enough that a cluster takes several of a row tile in turn, over
    one copy of their second operand."""
    counts = [RUN_COUNTS[(5 * e + e // 22) % len(RUN_COUNTS)] for e in range(256)]
    test_weight_backward(moe, counts, size)


# more experts than a warp has lanes: the last of 97, every one of 256, the last of 256
MANY = [[3] + [0] * 95 + [200], [(37 * e) % 150 for e in range(256)], [0] * 255 + [300]]


@pytest.mark.parametrize("counts", MANY, ids=["97", "256", "last"])
def test_many_experts(moe, counts):
    for test in (test_down_backward, test_up_backward, test_weight_backward, test_up_train):
        test(moe, counts, (128, 256))


@pytest.mark.parametrize("case", [([1500], 2048, 256), ([3001], 256, 1664), ([2003], 1408, 1408)], ids=str)
def test_one_expert_of_many_rows(moe, case):
    """A dense block: windows of other sizes than powers of two."""
    counts, H, I = case
    test_down_backward(moe, counts, (H, I))
    test_up_backward(moe, counts, (H, I))
    test_weight_backward(moe, counts, (H, I))


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%d" % s)
def test_up_train(moe, counts, size):
    r = Rows(moe, counts, *size)
    g, u, h, h0 = r.out(r.I), r.out(r.I), r.out(r.I), r.out(r.I)
    moe.moe_grouped_gemm_up_train(r.s, r.x, r.d_counts, r.d_off, r.wg, r.wu, g, u, h, r.ws)
    r.done(moe, g, u, h)
    for e, at in r.spans():
        want = ref.forward(r.x[at].double(), r.wg[e].double(), r.wu[e].double(), None)
        ref.check(g[at], want["g"], "g of expert %d" % e)
        ref.check(u[at], want["u"], "u of expert %d" % e)
    ws = moe.alloc_workspace(r.s)
    moe.moe_grouped_gemm_up_rows(r.s, r.x, r.d_counts, r.d_off, r.wg, r.wu, h0, ws)
    assert torch.equal(h.view(torch.int16), h0.view(torch.int16))


def test_no_rows_at_all(moe):
    """A shape whose rows went elsewhere: nothing written but zero weight gradients."""
    r = Rows(moe, [0, 0, 0], 256, 128)
    outs = [r.out(r.I), r.out(r.I), r.out(r.H)]
    dw = [torch.full_like(w, MARK) for w in (r.wg, r.wu, r.wd)]
    moe.moe_grouped_gemm_down_backward(r.s, r.dy, r.d_counts, r.d_off, r.wd, r.g, r.u, outs[0], outs[1], r.ws)
    moe.moe_grouped_gemm_up_backward(r.s, r.dg, r.du, r.d_counts, r.d_off, r.wg, r.wu, outs[2], r.ws)
    moe.moe_grouped_gemm_weight_backward(r.s, r.x, r.h, r.dg, r.du, r.dy, r.d_counts, r.d_off, *dw, r.ws)
    r.done(moe, *outs)
    assert all(not w.any() for w in dw)


def routed(moe, T, H, E, k, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = moe.shape(T, H, 128, E, k)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    o = moe.alloc_route_outputs(s)
    ws = moe.alloc_workspace(s)
    moe.moe_route(s, logits, o["topk_ids"], o["topk_w"], o["counts"], o["off_pad"], o["block_expert"],
                  o["num_blocks"], o["gather_idx"], o["scatter_idx"], ws)
    return s, logits, o, gen


@pytest.mark.parametrize("shape", [(1, 128, 1, 1), (1, 4096, 64, 8), (3, 256, 5, 5), (64, 384, 37, 3), (1003, 1408, 256, 16),
                                   (4096, 640, 8, 2), (77, 128, 33, 9)], ids=str)
def test_combine_backward(moe, shape):
    T, H, E, k = shape
    s, logits, o, gen = routed(moe, T, H, E, k)
    R = moe.capacity(s)[1]
    rows = o["scatter_idx"].long()
    real = torch.zeros(R, dtype=torch.bool, device="cuda")
    real[rows.flatten()] = True
    Y = torch.randn((R, H), generator=gen, device="cuda").bfloat16()
    Y[~real] = float("nan")
    dout = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    dY = torch.full((R, H), MARK, dtype=torch.bfloat16, device="cuda")
    dlogits = torch.full((T, E), MARK, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_combine_backward(s, Y, o["scatter_idx"], o["topk_ids"], o["topk_w"], dout, dY, dlogits, ws)
    assert moe.last_device_status(ws) == 0
    assert (dY[~real] == MARK).all()
    w, d = o["topk_w"].double(), dout.double()
    ref.check(dY[rows], ref.rounded(w.unsqueeze(-1) * d.unsqueeze(1), 2.0 ** -24 * (w.unsqueeze(-1) * d.unsqueeze(1)).abs()), "dY")
    y = Y[rows].double()
    dw = (y * d.unsqueeze(1)).sum(-1)
    # a lane adds at most H / 32 products one by one, then 5 + 8 sums join the parts
    dw_off = (H / 32 + 16) * 2.0 ** -24 * (y * d.unsqueeze(1)).abs().sum(-1)
    mean = (w * dw).sum(-1, keepdim=True)
    mean_off = (w * (dw_off + (k + 1) * 2.0 ** -24 * dw.abs())).sum(-1, keepdim=True)
    dl = w * (dw - mean)
    dl_off = w * (dw_off + mean_off + 4 * 2.0 ** -24 * (dw.abs() + mean.abs()))
    want = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, o["topk_ids"].long(), dl)
    off = torch.zeros_like(want).scatter_(1, o["topk_ids"].long(), dl_off)
    ref.check(dlogits, (want, off), "dlogits")


@pytest.mark.parametrize("shape", [(1, 128, 1, 1), (64, 384, 37, 3), (1003, 1408, 256, 16)], ids=str)
def test_permute_backward(moe, shape):
    T, H, E, k = shape
    s, _, o, gen = routed(moe, T, H, E, k)
    R = moe.capacity(s)[1]
    dXp = torch.randn((R, H), generator=gen, device="cuda").bfloat16()
    dX = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_permute_backward(s, dXp, o["scatter_idx"], dX, ws)
    assert moe.last_device_status(ws) == 0
    v = dXp[o["scatter_idx"].long()].double()
    ref.check(dX, ref.rounded(v.sum(1), k * 2.0 ** -24 * v.abs().sum(1)), "dX")


def layer_inputs(T, H, I, E, k, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    return dict(logits=normal(T, E), X=normal(T, H).bfloat16(), wg=(normal(E, H, I) / H ** 0.5).bfloat16(),
                wu=(normal(E, H, I) / H ** 0.5).bfloat16(), wd=(normal(E, I, H) / I ** 0.5).bfloat16(),
                dout=normal(T, H).bfloat16())


class Layer:
    """moe_forward_train and moe_backward with their buffers."""

    def __init__(self, moe, s):
        self.moe, self.s = moe, s
        T, H, I, E, k = s
        self.R = moe.capacity(s)[1]
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.g, self.u = torch.empty((self.R, I), **bf), torch.empty((self.R, I), **bf)
        self.out, self.dX = torch.empty((T, H), **bf), torch.empty((T, H), **bf)
        self.dwg, self.dwu, self.dwd = torch.empty((E, H, I), **bf), torch.empty((E, H, I), **bf), torch.empty((E, I, H), **bf)
        self.dlogits = torch.empty((T, E), device="cuda")
        self.ws, self.bws = moe.alloc_workspace(s), moe.alloc_backward_workspace(s)

    def forward(self, i):
        self.moe.moe_forward_train(self.s, i["logits"], i["X"], i["wg"], i["wu"], i["wd"], self.g, self.u, self.out, self.ws)

    def backward(self, i):
        self.moe.moe_backward(self.s, i["wg"], i["wu"], i["wd"], self.g, self.u, i["dout"], self.dX, self.dwg, self.dwu,
                              self.dwd, self.dlogits, self.ws, self.bws)

    def results(self):
        return [self.out, self.dX, self.dwg, self.dwu, self.dwd, self.dlogits]

    def status(self):
        return self.moe.last_device_status(self.ws), self.moe.last_device_status(self.bws)


SHAPES = [(1, 128, 128, 1, 1), (1, 256, 384, 8, 3), (128, 256, 512, 8, 2), (333, 384, 256, 16, 4), (700, 640, 384, 3, 1)]


@pytest.mark.parametrize("s", SHAPES, ids=str)
def test_layer_against_64_bits(moe, s):
    """The layer's output and gradients.  Along the way to a result at most seven
    values are rounded to bf16 (g, u, h, Y or dY, dg or du, dX of a row, the
    result), each by at most 2^-8 of itself, so that the norm of the difference is
    at most 7 x 2^-8 of a norm without cancellation; dlogits are compared on the
    scale of the products' norm that they are differences of."""
    T, H, I, E, k = s
    i = layer_inputs(*s)
    lay = Layer(moe, s)
    lay.forward(i)
    lay.backward(i)
    assert lay.status() == (0, 0)
    leaves = [i[n].double().requires_grad_() for n in ("logits", "X", "wg", "wu", "wd")]
    out = ref.layer(*leaves, k)
    grads = torch.autograd.grad((out * i["dout"].double()).sum(), leaves)
    most = 7 * ref.BF16
    for name, got, want in zip(("out", "dlogits", "dX", "dwg", "dwu", "dwd"),
                               (lay.out, lay.dlogits, lay.dX, lay.dwg, lay.dwu, lay.dwd), (out.detach(), *grads)):
        norm = want.norm()
        if name == "dlogits":
            # each is w (dw - mean) with dw = <dout, Y>, Y rounded: |error| <= w 2 max_j |dout| |Y_j| 2 roundings
            norm = (i["dout"].double().norm(dim=-1) * out.detach().norm(dim=-1)).norm() * 2 * k
        assert float((got.double() - want).norm()) <= most * float(norm), name


@pytest.mark.parametrize("s", SHAPES[2:4], ids=str)
def test_layer_against_differences(moe, s):
    """Each gradient's product with a direction against the central difference of
    the 64-bit layer along it.  The direction is the gradient's own (plus noise of
    a tenth), so nothing cancels and the roundings above bound the error."""
    T, H, I, E, k = s
    i = layer_inputs(*s, seed=3)
    lay = Layer(moe, s)
    lay.forward(i)
    lay.backward(i)
    leaves = {n: i[n].double() for n in ("logits", "X", "wg", "wu", "wd")}
    picks = torch.sort(leaves["logits"], dim=-1, descending=True, stable=True).indices[:, :k]
    dout = i["dout"].double()
    gen = torch.Generator(device="cuda").manual_seed(9)
    for n, got in (("logits", lay.dlogits), ("X", lay.dX), ("wg", lay.dwg), ("wu", lay.dwu), ("wd", lay.dwd)):
        v = got.double()
        v = v / v.norm()
        noise = torch.randn(v.shape, generator=gen, device="cuda", dtype=torch.float64)
        v = v + 0.1 * noise / noise.norm()
        eps = 1e-4
        f = []
        for step in (eps, -eps):
            moved = [leaves[m] + step * v if m == n else leaves[m] for m in ("logits", "X", "wg", "wu", "wd")]
            f.append(float((ref.layer(*moved, k, picks) * dout).sum()))
        diff = (f[0] - f[1]) / (2 * eps)
        along = float((got.double() * v).sum())
        assert abs(along - diff) <= 7 * ref.BF16 * abs(diff), (n, along, diff)


@pytest.mark.parametrize("s", SHAPES, ids=str)
def test_layer_is_its_steps(moe, s):
    """moe_forward_train gives moe_forward's bits and moe_backward the step calls'."""
    T, H, I, E, k = s
    i = layer_inputs(*s, seed=1)
    lay = Layer(moe, s)
    lay.forward(i)
    out = torch.empty_like(lay.out)
    ws = moe.alloc_workspace(s)
    moe.moe_forward(s, i["logits"], i["X"], i["wg"], i["wu"], i["wd"], out, ws)
    assert torch.equal(out.view(torch.int16), lay.out.view(torch.int16))
    lay.backward(i)
    o = moe.alloc_route_outputs(s)
    moe.moe_route(s, i["logits"], o["topk_ids"], o["topk_w"], o["counts"], o["off_pad"], o["block_expert"],
                  o["num_blocks"], o["gather_idx"], o["scatter_idx"], ws)
    rows = o["scatter_idx"].long()

    def buf(cols):
        return torch.full((lay.R, cols), float("nan"), dtype=torch.bfloat16, device="cuda")

    xp, g, u, h, y, dy, dg, du, dxp = (buf(c) for c in (H, I, I, I, H, H, I, I, H))
    xp[rows] = i["X"].unsqueeze(1)
    c, off = o["counts"], o["off_pad"]
    moe.moe_grouped_gemm_up_train(s, xp, c, off, i["wg"], i["wu"], g, u, h, ws)
    moe.moe_grouped_gemm_down(s, h, c, off, i["wd"], y, ws)
    dX, dlogits = torch.empty_like(lay.dX), torch.empty_like(lay.dlogits)
    dw = [torch.empty_like(t) for t in (lay.dwg, lay.dwu, lay.dwd)]
    moe.moe_combine_backward(s, y, o["scatter_idx"], o["topk_ids"], o["topk_w"], i["dout"], dy, dlogits, ws)
    moe.moe_grouped_gemm_down_backward(s, dy, c, off, i["wd"], g, u, dg, du, ws)
    moe.moe_grouped_gemm_up_backward(s, dg, du, c, off, i["wg"], i["wu"], dxp, ws)
    moe.moe_grouped_gemm_weight_backward(s, xp, h, dg, du, dy, c, off, *dw, ws)
    moe.moe_permute_backward(s, dxp, o["scatter_idx"], dX, ws)
    assert moe.last_device_status(ws) == 0 and lay.status() == (0, 0)
    for a, b in zip((dX, *dw), (lay.dX, lay.dwg, lay.dwu, lay.dwd)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(dlogits, lay.dlogits)


def test_layer_repeats_and_replays(moe):
    """The same bits twice, on another stream, and from a captured graph replayed on new inputs."""
    s = SHAPES[3]
    a, b = layer_inputs(*s, seed=5), layer_inputs(*s, seed=6)
    lay = Layer(moe, s)

    def run(i):
        lay.forward(i)
        lay.backward(i)
        return [t.clone() for t in lay.results()]

    first, other = run(a), run(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = run(a)
    torch.cuda.current_stream().wait_stream(stream)
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    held = {n: t.clone() for n, t in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.forward(held)
        lay.backward(held)
    for inputs, want in ((b, other), (a, first), (b, other)):
        for n in held:
            held[n].copy_(inputs[n])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(lay.results(), want):
            assert torch.equal(x, y)
    assert lay.status() == (0, 0)

"""Quantisation to 8-bit integers and the products on them against 64-bit references."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import int8_ref as ref  # noqa: E402
import train_ref  # noqa: E402

MARK = -7.5


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


def generator(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def special_rows(rows, cols, gen):
    """Normal rows, and among them: zeros, ties (multiples of amax / 254), one value
    alone, the largest and smallest magnitudes, NaN, infinities."""
    x = torch.randn((rows, cols), generator=gen, device="cuda").bfloat16()
    n = torch.randint(-254, 255, (cols,), generator=gen, device="cuda").float()
    special = [torch.zeros(cols, device="cuda"), n / 2, n * 2.0 ** 100, n * 2.0 ** -120, n * 2.0 ** -133,
               n.sign() * 2.0 ** (n.abs() % 12), (n == n.max()).float() * 3.0,
               torch.where(n == n.max(), torch.full_like(n, 3.3e38), n * 1e36)]
    for i, s in enumerate(special):
        if i < rows:
            x[i] = s.bfloat16()
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        if len(special) + i < rows:
            x[len(special) + i, (7 * i) % cols] = v
    return x


def same_scales(got, want):
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("shape", [(1, 128), (12, 128), (13, 384), (64, 4096), (301, 1024), (15, 1152), (33, 8192), (14, 8320),
                                   (12, 32768), (2049, 640)], ids=str)
def test_quantize_rows(moe, shape):
    rows, cols = shape
    x = special_rows(rows, cols, generator())
    codes, scales = torch.full((rows + 1, cols), 99, dtype=torch.int8, device="cuda"), torch.full((rows + 1,), MARK, device="cuda")
    moe.moe_quantize_int8(x, rows, cols, codes, scales)
    q, s = ref.quantize(x)
    assert torch.equal(codes[:rows], q)
    assert same_scales(scales[:rows], s)
    assert (codes[rows] == 99).all() and scales[rows] == MARK  # nothing behind the last row
    out = torch.full((rows + 1, cols), MARK, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_int8(codes, scales, rows, cols, out)
    want = (q.float() * s.unsqueeze(-1)).bfloat16()
    assert torch.equal(out[:rows].isnan(), want.isnan())
    assert torch.equal(out[:rows][~want.isnan()], want[~want.isnan()])
    assert (out[rows] == MARK).all()


def test_every_quotient_of_a_row(moe):
    """All 8-bit significands against all of amax's, over the exponents that matter."""
    m = torch.arange(128, 256, device="cuda").float()
    x = torch.stack([torch.cat([m * 2.0 ** -e for e in range(1, 11)]) for _ in range(128)])  # [128, 1280], below 128
    x[:, 0] = m  # each row's amax: 128 .. 255
    x = x.bfloat16().contiguous()
    codes, scales = moe.alloc_int8(128, 1280)
    moe.moe_quantize_int8(x, 128, 1280, codes, scales)
    q, s = ref.quantize(x)
    assert torch.equal(codes, q) and torch.equal(scales, s)


@pytest.mark.parametrize("shape", [(1, 128, 128), (3, 384, 256), (2, 640, 128), (1, 4096, 192 * 2), (2, 2304, 128), (1, 4224, 128),
                                   (2, 8320, 128)], ids=str)
def test_quantize_weights(moe, shape):
    E, K, N = shape
    w = special_rows(E * N, K, generator(1)).reshape(E, N, K).transpose(1, 2).contiguous()
    codes, scales = moe.alloc_int8(E * N, K)
    moe.moe_quantize_weights_int8(w, E, K, N, codes, scales)
    q, s = ref.quantize(w.transpose(1, 2).reshape(E * N, K))
    assert torch.equal(codes, q) and same_scales(scales, s)


@pytest.mark.parametrize("shape", [(40, 384, 512), (24, 1152, 256), (20, 2176, 1024), (80, 128, 256), (9, 4224, 1280), (3, 8320, 2560), (1, 12416, 256), (2, 12800, 512)], ids=str)
def test_quantize_weights_of_many_columns(moe, shape):
    """Columns enough to fill the device, where a cluster of fewer CTAs takes them."""
    test_quantize_weights(moe, shape)


@pytest.mark.parametrize("shape", [(1, 128, 1, 1), (50, 384, 7, 3), (300, 9216, 64, 16)], ids=str)
def test_quantize_permute(moe, shape):
    T, H, E, k = shape
    s = moe.shape(T, H, 128, E, k)
    o, ws = moe.alloc_route_outputs(s), moe.alloc_workspace(s)
    logits = torch.randn((T, E), generator=generator(2), device="cuda")
    moe.moe_route(s, logits, o["topk_ids"], o["topk_w"], o["counts"], o["off_pad"], o["block_expert"], o["num_blocks"],
                  o["gather_idx"], o["scatter_idx"], ws)
    x = special_rows(T, H, generator(3))
    R = moe.capacity(s)[1]
    codes, scales = torch.full((R, H), 99, dtype=torch.int8, device="cuda"), torch.full((R,), MARK, device="cuda")
    moe.moe_quantize_permute_int8(s, x, o["scatter_idx"], codes, scales, ws)
    assert moe.last_device_status(ws) == 0
    q, z = ref.quantize(x)
    rows = o["scatter_idx"].long()
    assert torch.equal(codes[rows], q.unsqueeze(1).expand(T, k, H))
    assert same_scales(scales[rows].flatten(), z.unsqueeze(1).expand(T, k).flatten())
    left = torch.ones(R, dtype=torch.bool, device="cuda")
    left[rows.flatten()] = False
    assert (codes[left] == 99).all() and (scales[left] == MARK).all()


class Rows:
    """Random codes and scales in expert order; padding holds other codes and NaN scales."""

    def __init__(self, moe, counts, K, N, up, seed=0, codes=None):
        gen = generator(seed)
        off, T = train_ref.layout(counts)
        self.counts, self.off, self.E, self.up = list(counts), off, len(counts), up
        self.s = moe.shape(T, K if up else N, N if up else K, self.E, 1)
        self.R = moe.capacity(self.s)[1]
        self.d_counts, self.d_off = torch.tensor(counts, dtype=torch.int32, device="cuda"), torch.from_numpy(off).cuda()
        self.real = torch.zeros(self.R, dtype=torch.bool, device="cuda")
        for e, at in self.spans():
            self.real[at] = True

        def ints(rows):
            if codes is not None:
                return torch.full((rows, K), codes, dtype=torch.int8, device="cuda")
            return torch.randint(-128, 128, (rows, K), generator=gen, device="cuda").to(torch.int8)

        def scales(rows):
            return (torch.rand(rows, generator=gen, device="cuda") + 0.5) / (127 * 40 * (K / 256) ** 0.5 / 2 ** 0.5)

        self.q, self.z = ints(self.R), scales(self.R) * 2
        self.z[~self.real] = float("nan")
        self.w = [(ints(self.E * N), scales(self.E * N)) for _ in range(2 if up else 1)]
        self.out = torch.full((self.R, N), MARK, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.N = N

    def spans(self):
        for e, c in enumerate(self.counts):
            yield e, slice(int(self.off[e]), int(self.off[e]) + c)

    def run(self, moe):
        w = [t for pair in self.w for t in pair]
        fn = moe.moe_grouped_gemm_up_int8 if self.up else moe.moe_grouped_gemm_down_int8
        fn(self.s, self.q, self.z, self.d_counts, self.d_off, *w, self.out, self.ws)
        assert moe.last_device_status(self.ws) == 0
        assert int(self.ws.sum()) == 0

    def check(self):
        assert (self.out[~self.real] == MARK).all(), "padding rows were written"
        for e, at in self.spans():
            n = slice(e * self.N, (e + 1) * self.N)
            want = (ref.up if self.up else ref.down)(self.q[at], self.z[at], *[t[n] for pair in self.w for t in pair])
            train_ref.check(self.out[at], want, "expert %d" % e)


COUNTS = [[1], [2], [0, 1, 1], [3] + [0] * 18 + [6], [5, 0, 1], [16, 32, 48], [129, 127, 0, 64, 65], [255, 256, 257, 0, 3], [0, 0, 300, 0], [1000, 33]]


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)) if len(c) < 9 else "few-of-%d" % len(c))
@pytest.mark.parametrize("size", [(128, 128), (256, 384), (640, 256), (384, 640)], ids=lambda s: "%dx%d" % s)
def test_products(moe, up, counts, size):
    r = Rows(moe, counts, *size, up)
    r.run(moe)
    r.check()


# more experts than a warp has lanes: the last of 97, every one of 256, the last of 256
MANY = [[3] + [0] * 95 + [200], [(37 * e) % 150 for e in range(256)], [0] * 255 + [70]]


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("counts", MANY, ids=["97", "256", "last"])
def test_products_of_many_experts(moe, up, counts):
    test_products(moe, up, counts, (128, 256))


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("codes", [127, -128, 1])
def test_products_of_extreme_codes(moe, up, codes):
    """Sums past 2^24 (8192 x 127^2 and 8192 x 2^14), and exact ones."""
    r = Rows(moe, [3, 130], 8192, 256, up, codes=codes)
    r.run(moe)
    r.check()


def test_nan_scales_reach_their_rows_and_columns_alone(moe):
    r = Rows(moe, [40, 3], 256, 256, False)
    r.z[5] = float("nan")
    r.w[0][1][256 + 9] = float("nan")  # column 9 of the second expert
    r.run(moe)
    bad = r.out.isnan()
    want = torch.zeros_like(bad)
    want[5] = True
    want[128:131, 9] = True
    assert torch.equal(bad, want)


def quantized(moe, w):
    E, K, N = w.shape
    pair = moe.alloc_int8(E * N, K)
    moe.moe_quantize_weights_int8(w, E, K, N, *pair)
    return pair


def layer(s, seed=0):
    T, H, I, E, k = s
    gen = generator(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    return (normal(T, E), normal(T, H).bfloat16(), (normal(E, H, I) / H ** 0.5).bfloat16(),
            (normal(E, H, I) / H ** 0.5).bfloat16(), (normal(E, I, H) / I ** 0.5).bfloat16())


SHAPES = [(1, 128, 128, 1, 1), (1, 256, 384, 8, 3), (128, 256, 512, 8, 2), (333, 384, 256, 16, 4), (700, 640, 384, 3, 1)]


@pytest.mark.parametrize("s", SHAPES, ids=str)
def test_forward(moe, s):
    """moe_forward_int8 gives its steps' bits, and the bf16 layer's output as far as
    8 bits go: x, the weights and h are off by at most amax / 254 an element, which
    at amax below 5.5 of their deviation is at most 2.2% of their norm each, and five
    such errors that do not depend on one another add up to 5%."""
    T, H, I, E, k = s
    logits, x, wg, wu, wd = layer(s)
    w = [t for m in (wg, wu, wd) for t in quantized(moe, m)]
    out = torch.empty_like(x)
    ws = moe.alloc_int8_workspace(s)
    moe.moe_forward_int8(s, logits, x, *w, out, ws)
    assert moe.last_device_status(ws) == 0
    o, bws = moe.alloc_route_outputs(s), moe.alloc_workspace(s)
    moe.moe_route(s, logits, o["topk_ids"], o["topk_w"], o["counts"], o["off_pad"], o["block_expert"], o["num_blocks"],
                  o["gather_idx"], o["scatter_idx"], bws)
    R = moe.capacity(s)[1]
    xq, hq = moe.alloc_int8(R, H), moe.alloc_int8(R, I)
    h, y = torch.zeros((R, I), dtype=torch.bfloat16, device="cuda"), torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_quantize_permute_int8(s, x, o["scatter_idx"], *xq, bws)
    moe.moe_grouped_gemm_up_int8(s, *xq, o["counts"], o["off_pad"], *w[:4], h, bws)
    moe.moe_quantize_int8(h, R, I, *hq)
    moe.moe_grouped_gemm_down_int8(s, *hq, o["counts"], o["off_pad"], *w[4:], y, bws)
    steps = torch.empty_like(out)
    moe.moe_combine(s, y, o["scatter_idx"], o["topk_w"], steps, bws)
    assert moe.last_device_status(bws) == 0
    assert torch.equal(out.view(torch.int16), steps.view(torch.int16))
    full = torch.empty_like(out)
    moe.moe_forward(s, logits, x, wg, wu, wd, full, bws)
    assert float((out.float() - full.float()).norm()) <= 0.05 * float(full.float().norm())


def test_forward_repeats_and_replays(moe):
    s = SHAPES[3]
    a, b = layer(s, 1), layer(s, 2)
    w = [t for m in a[2:] for t in quantized(moe, m)]
    out, ws = torch.empty_like(a[1]), moe.alloc_int8_workspace(s)

    def run(i):
        moe.moe_forward_int8(s, i[0], i[1], *w, out, ws)
        return out.clone()

    first, other = run(a), run(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = run(a)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(first, again)
    held = [t.clone() for t in a[:2]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_int8(s, *held, *w, out, ws)
    for inputs, want in ((b, other), (a, first), (b, other)):
        for h, v in zip(held, inputs):
            h.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert moe.last_device_status(ws) == 0

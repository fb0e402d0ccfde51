"""The backward products and the 8-bit products on counters, counts and offsets that
are not what they should be: reported, inside the buffers, and the next call sound."""
import numpy as np
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import train_ref  # noqa: E402

BOUNDS = 7
MARK = -7.5
UP, DOWN = 16, 32                     # the products' counters among the workspace's 32-bit words


class Product:
    """One product's buffers, its call, its outputs and where its counter lies."""

    def __init__(self, which, counts, H, I, seed=0):
        need_gpu()
        import combine_moe_route_04_gb300 as moe
        self.moe, self.which, self.counts = moe, which, counts
        gen = torch.Generator(device="cuda").manual_seed(seed)
        off, T = train_ref.layout(counts)
        E = len(counts)
        self.s = moe.shape(T, H, I, E, 1)
        R = self.R = moe.capacity(self.s)[1]
        self.c = torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.o = torch.from_numpy(off).cuda()
        self.words = torch.zeros(64, dtype=torch.int32, device="cuda")
        self.ws = self.words.view(torch.uint8)

        def rows(cols):
            return torch.randn((R, cols), generator=gen, device="cuda").bfloat16()

        def weights(K, N):
            return (torch.randn((E, K, N), generator=gen, device="cuda") / K ** 0.5).bfloat16()

        def ints(n, K):
            return torch.randint(-127, 128, (n, K), generator=gen, device="cuda").to(torch.int8), \
                torch.rand(n, generator=gen, device="cuda") / K

        def out(*shape):
            return torch.full(shape, MARK, dtype=torch.bfloat16, device="cuda")

        c, o, ws = self.c, self.o, self.ws
        self.at = UP
        if which == "down_backward":
            self.outs = [out(R, I), out(R, I)]
            a = [rows(H), c, o, weights(I, H), rows(I), rows(I), *self.outs, ws]
            self.fn = moe.moe_grouped_gemm_down_backward
        elif which == "up_backward":
            self.outs, self.at = [out(R, H)], DOWN
            a = [rows(I), rows(I), c, o, weights(H, I), weights(H, I), *self.outs, ws]
            self.fn = moe.moe_grouped_gemm_up_backward
        elif which == "weight_backward":
            self.outs = [out(E, H, I), out(E, H, I), out(E, I, H)]
            a = [rows(H), rows(I), rows(I), rows(I), rows(H), c, o, *self.outs, ws]
            self.fn = moe.moe_grouped_gemm_weight_backward
        elif which == "up_int8":
            self.outs = [out(R, I)]
            a = [*ints(R, H), c, o, *ints(E * I, H), *ints(E * I, H), *self.outs, ws]
            self.fn = moe.moe_grouped_gemm_up_int8
        else:
            self.outs, self.at = [out(R, H)], DOWN
            a = [*ints(R, I), c, o, *ints(E * H, I), *self.outs, ws]
            self.fn = moe.moe_grouped_gemm_down_int8
        self.args = a

    def call(self):
        for t in self.outs:
            t.fill_(MARK)
        self.fn(self.s, *self.args)
        return self.moe.last_device_status(self.ws), [t.clone() for t in self.outs]


PRODUCTS = ["down_backward", "up_backward", "weight_backward", "up_int8", "down_int8"]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def big(which):
    """More tiles than clusters, so that clusters draw more than once."""
    return Product(which, [300, 5, 0, 129], 8192 + 128, 4096 + 128)


@pytest.mark.parametrize("which", PRODUCTS)
def test_a_tile_counter_that_was_not_cleared(which):
    p = big(which)
    status, want = p.call()
    assert status == 0
    for left in (1, 3, 75, 76, 77, 500, 1 << 20, -1, -2):
        p.words[p.at] = left
        assert p.call()[0] == BOUNDS, left
        status, got = p.call()                        # cleared again
        assert status == 0 and same(got, want), left
    assert not p.words.any()


@pytest.mark.parametrize("which", PRODUCTS)
def test_an_arrival_count_that_was_not_cleared(which):
    p = big(which)
    want = p.call()[1]
    for left in (1, 2):
        p.words[p.at + 1] = left
        assert p.call()[0] == BOUNDS, left
        p.words[p.at:p.at + 2] = 0
        status, got = p.call()
        assert status == 0 and same(got, want), left


@pytest.mark.parametrize("which", PRODUCTS)
@pytest.mark.parametrize("counts", [[40, 5, 0, 129], [1, 1]], ids=["tiles", "few-rows"])
def test_counts_and_offsets_out_of_range(which, counts):
    """An expert whose rows are not inside its blocks and the buffers is reported and
    left out; the others' results are those of the sound call."""
    p = Product(which, counts, 256, 384)
    status, want = p.call()
    assert status == 0
    off, E = p.o.clone(), len(counts)
    per_expert = which == "weight_backward"
    for bad_count, bad_off in [(1 << 30, None), (-5, None), (129, None), (None, -128), (None, 1 << 30)]:
        p.c[1], p.o[1] = counts[1], off[1]
        if bad_count is not None:
            p.c[1] = bad_count
        else:
            p.o[1] = bad_off
        status, got = p.call()
        assert status == BOUNDS, (bad_count, bad_off)
        for g, w in zip(got, want):
            if per_expert:
                assert torch.equal(g[2:], w[2:])
                assert (g[1] == MARK).all()
            else:
                first = int(off[2])
                assert torch.equal(g[first:], w[first:])
                assert (g[int(off[1]):first] == MARK).all()
    p.c[1], p.o[1] = counts[1], off[1]
    status, got = p.call()
    assert status == 0 and same(got, want)


@pytest.mark.parametrize("which", PRODUCTS)
def test_counts_that_fit_alone_but_not_together(which):
    """Every expert is said to fill the buffers; no expert's padded rows allow it, so
    nothing is loaded or stored and the buffers can be small."""
    p = Product(which, [1] * 256, 128, 128)
    p.c.fill_(p.R)
    status, got = p.call()
    assert status == BOUNDS
    assert all((g == MARK).all() for g in got)


def test_rows_and_ids_out_of_range_in_the_combine_backward():
    need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, E, k = 9, 256, 4, 2
    s = moe.shape(T, H, 128, E, k)
    R = moe.capacity(s)[1]
    gen = torch.Generator(device="cuda").manual_seed(0)
    y = torch.randn((R, H), generator=gen, device="cuda").bfloat16()
    dout = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    rows = torch.randperm(R, generator=gen, device="cuda")[:T * k].reshape(T, k).int()
    ids = torch.tensor([[0, 1], [1, 2], [2, 3]] * 3, dtype=torch.int32, device="cuda")
    w = torch.rand((T, k), generator=gen, device="cuda")

    def call(rows, ids):
        dy, dl = torch.full_like(y, MARK), torch.full((T, E), MARK, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        moe.moe_combine_backward(s, y, rows, ids, w, dout, dy, dl, ws)
        return moe.last_device_status(ws), dy, dl

    status, dy, dl = call(rows, ids)
    assert status == 0
    for bad in (-1, R, 1 << 30):
        r = rows.clone()
        r[4, 1] = bad
        status, gy, gl = call(r, ids)
        assert status == BOUNDS
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[rows[4, 1].long()] = False
        assert torch.equal(gy[keep], dy[keep]) and (gy[~keep] == MARK).all()
        other = torch.arange(T, device="cuda") != 4
        assert torch.equal(gl[other], dl[other])
    for bad in (-1, E, 1 << 30):
        i = ids.clone()
        i[2, 0] = bad
        status, gy, gl = call(rows, i)
        assert status == BOUNDS and torch.equal(gy, dy)
        want = dl.clone()
        want[2, ids[2, 0].long()] = 0
        assert torch.equal(gl, want)
    same_id = ids.clone()
    same_id[5] = 3                                    # both picks of a token name one expert: their sum
    status, _, gl = call(rows, same_id)
    assert status == 0
    assert abs(float(gl[5, 3]) - float(dl[5, ids[5].long()].double().sum())) <= 2.0 ** -23 * float(dl[5].abs().sum())


def test_quantize_permute_reports_rows_out_of_range():
    need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = moe.shape(5, 256, 128, 2, 1)
    R = moe.capacity(s)[1]
    x = torch.randn((5, 256), device="cuda").bfloat16()
    rows = torch.tensor([[0], [1], [R], [-1], [130]], dtype=torch.int32, device="cuda")
    codes, scales = moe.alloc_int8(R, 256)
    codes.fill_(99)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_permute_int8(s, x, rows, codes, scales, ws)
    assert moe.last_device_status(ws) == BOUNDS
    written = (codes != 99).any(-1).nonzero().flatten().tolist()
    assert written == [0, 1, 130]

"""The bf16 products on tile counters that were not cleared: whatever is left in one,
the call reports it (tiles may have been left out), stays inside its buffers, and the
next call is sound.  One kernel has them all: gate/up, the same that keeps g and u,
down, and in a forward the second after the first."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import train_ref  # noqa: E402
from test_gpu_train import Layer, layer_inputs  # noqa: E402

BOUNDS = 7
MARK = -7.5
UP, DOWN = 16, 32                     # the products' counters among the workspace's 32-bit words


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


class Product:
    """One product over more tiles than there are clusters, so that clusters draw more than once."""

    def __init__(self, moe, which):
        self.moe = moe
        counts, K, N = [300, 5, 0, 129], 256, 256 * 33 if which != "down" else 512 * 33
        E, gen = len(counts), torch.Generator(device="cuda").manual_seed(0)
        off, T = train_ref.layout(counts)
        self.s = s = moe.shape(T, K, N, E, 1) if which != "down" else moe.shape(T, N, K, E, 1)
        R = moe.capacity(s)[1]
        c, o = torch.tensor(counts, dtype=torch.int32, device="cuda"), torch.from_numpy(off).cuda()
        self.ws = moe.alloc_workspace(s)
        self.words = self.ws[:256].view(torch.int32)
        self.at = DOWN if which == "down" else UP

        def normal(*shape):
            return torch.randn(shape, generator=gen, device="cuda").bfloat16()

        def out():
            return torch.full((R, N), MARK, dtype=torch.bfloat16, device="cuda")

        assert 4 * 33 > torch.cuda.get_device_properties(0).multi_processor_count // 2 + 3
        if which == "down":
            self.outs = [out()]
            self.fn, self.args = moe.moe_grouped_gemm_down, [normal(R, K), c, o, normal(E, K, N), *self.outs]
        else:
            self.outs = [out()] if which == "up" else [out(), out(), out()]
            self.fn = moe.moe_grouped_gemm_up_rows if which == "up" else moe.moe_grouped_gemm_up_train
            self.args = [normal(R, K), c, o, normal(E, K, N), normal(E, K, N), *self.outs]

    def call(self):
        for t in self.outs:
            t.fill_(MARK)
        self.fn(self.s, *self.args, self.ws)
        return self.moe.last_device_status(self.ws), [t.clone() for t in self.outs]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("which", ["up", "up_train", "down"])
def test_a_tile_counter_that_was_not_cleared(moe, which):
    p = Product(moe, which)
    status, want = p.call()
    assert status == 0 and not p.words.any()
    for left in (1, 3, 56, 75, 76, 77, 131, 132, 133, 500, 1 << 20, -1, -2):
        p.words[p.at] = left
        assert p.call()[0] == BOUNDS, left
        status, got = p.call()                        # cleared again
        assert status == 0 and same(got, want), left
    assert not p.words.any()


@pytest.mark.parametrize("which", ["up", "up_train", "down"])
def test_an_arrival_count_that_was_not_cleared(moe, which):
    p = Product(moe, which)
    want = p.call()[1]
    for left in (1, 2):
        p.words[p.at + 1] = left
        assert p.call()[0] == BOUNDS, left
        p.words[p.at:p.at + 2] = 0
        status, got = p.call()
        assert status == 0 and same(got, want), left


@pytest.mark.parametrize("which", ["up", "up_train", "down"])
def test_no_rows_and_nothing_to_report(moe, which):
    p = Product(moe, which)
    p.args[1].zero_()
    for _ in range(2):
        status, got = p.call()
        assert status == 0 and all((g == MARK).all() for g in got) and not p.words.any()


@pytest.mark.parametrize("train", [False, True], ids=["forward", "forward_train"])
@pytest.mark.parametrize("at", [UP, DOWN], ids=["gate_up", "down"])
def test_a_forward_with_a_tile_counter_that_was_not_cleared(moe, train, at):
    """The product that follows waits for the windows that the first left out: it ends
    with the first one's report, not with a wait that ran out."""
    s = (600, 256, 256 * 25, 4, 1) if at == UP else (600, 512 * 25, 256, 4, 1)
    i = layer_inputs(*s)
    lay = Layer(moe, s)
    words = lay.ws[:256].view(torch.int32)

    def call():
        lay.out.zero_()
        if train:
            lay.forward(i)
        else:
            moe.moe_forward(s, i["logits"], i["X"], i["wg"], i["wu"], i["wd"], lay.out, lay.ws)
        return moe.last_device_status(lay.ws), lay.out.clone()

    status, want = call()
    assert status == 0
    for left in (1, 3, 20, 500, -1):
        words[at] = left
        assert call()[0] == BOUNDS, left
        words[UP:UP + 2], words[DOWN:DOWN + 2] = 0, 0
        status, got = call()
        assert status == 0 and torch.equal(got, want), left

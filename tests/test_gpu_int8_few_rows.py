"""The 8-bit products' two ways (integer dot products for few rows, tensor cores for
more) on the same rows: the same bits while every float32 sum is exact, and within
the products' bound of the definition where sums pass 2^24."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_int8 import Rows, test_forward  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    return m


def both_ways(moe, up, K, codes=None):
    """Two rows of one expert alone, and the same beside another expert's 300."""
    few, many = (Rows(moe, counts, K, 384, up, codes=codes) for counts in ([2], [2, 300]))
    few.q[:2], few.z[:2] = many.q[:2], many.z[:2]
    for a, b in zip(few.w, many.w):
        for x, y in zip(a, b):
            x.copy_(y[:x.shape[0]])
    for r in (few, many):
        r.run(moe)
        r.check()
    return few.out[:2], many.out[:2]


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("K,codes", [(128, None), (640, None), (1024, None), (1024, 127), (1024, -128)], ids=str)
def test_the_same_bits_where_sums_are_exact(moe, up, K, codes):
    a, b = both_ways(moe, up, K, codes)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# rows up to the most that are taken as few, several in an expert, and one more
COUNTS = [[8] + [0] * 15, [1] + [0] * 18 + [7], [5, 0, 3] + [0] * 253, [4, 4] + [0] * 30, [1] * 8 + [0] * 8,
          [9] + [0] * 17]


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "%d-rows-of-%d" % (sum(c), len(c)))
@pytest.mark.parametrize("size", [(128, 128), (384, 640)], ids=lambda s: "%dx%d" % s)
def test_rows_of_single_experts(moe, up, counts, size):
    r = Rows(moe, counts, *size, up)
    r.run(moe)
    r.check()


def test_the_layer_at_the_most_rows(moe):
    """Three tokens of eight experts each, as few and one row more as many."""
    for s in [(3, 256, 384, 64, 8), (5, 256, 384, 64, 5)]:
        test_forward(moe, s)


@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
@pytest.mark.parametrize("K,codes", [(8192, None), (8192, 127), (32768, -128)], ids=str)
def test_long_sums_keep_their_bound(moe, up, K, codes):
    both_ways(moe, up, K, codes)

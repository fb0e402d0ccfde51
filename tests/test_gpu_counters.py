"""Workspace counters that were not cleared: the call that finds one dirty reports
it, however little is left in it, and stays inside its buffers."""
import numpy as np
import pytest

import mxfp4_ref as ref
from gpu_util import need_gpu, to_dev
from test_gpu_mxfp4 import operands, shape_for, upload

pytestmark = pytest.mark.gpu

BOUNDS = 7
UP, DOWN = 16, 32                     # the products' counters among the workspace's 32-bit words


def product(which, wide):
    """(call, output, workspace words, tiles) of one product over a few experts, with
    more tiles than the GPU has SMs (CTAs then draw more than once)."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    counts, K, N = [300, 5, 0, 129], 128, 16384
    H, I, mats = (K, N, 2) if which == UP else (N, K, 1)
    r, ws, off, real = operands(counts, K, N, mats, 3)
    s = shape_for(counts, H, I, wide)
    mr = moe.capacity(s)[1]
    codes, scales = upload(r, off, mr)
    w = [t for c, z in ws for t in (to_dev(ref.pack(c)), to_dev(ref.tile(z)))]
    out = torch.zeros((mr, N), dtype=torch.bfloat16, device="cuda")
    words = torch.zeros(64, dtype=torch.int32, device="cuda")
    fn = moe.moe_grouped_gemm_up_mxfp4 if which == UP else moe.moe_grouped_gemm_down_mxfp4
    c, o = to_dev(np.array(counts, np.int32)), to_dev(off.astype(np.int32))
    windows = sum(-(-n // (192 if wide else 128)) for n in counts)
    tiles = windows * (N // 128 if which == UP else -(-N // 256))
    assert tiles > torch.cuda.get_device_properties(0).multi_processor_count + 3
    return lambda: fn(s, codes, scales, c, o, *w, out, words.view(torch.uint8)), out, words, tiles


@pytest.mark.parametrize("which", [UP, DOWN])
@pytest.mark.parametrize("wide", [False, True])
def test_a_product_reports_what_its_tile_counter_held(which, wide):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    call, out, words, tiles = product(which, wide)
    call()
    assert moe.last_device_status(words.view(torch.uint8)) == 0
    want = out.clone()
    for left in (1, 3, tiles - 1, tiles, tiles + 1, 1 << 20, -1):
        words[which] = left
        call()
        assert moe.last_device_status(words.view(torch.uint8)) == BOUNDS, left
        out.zero_()
        call()                                        # cleared again: nothing to report, every tile computed
        assert moe.last_device_status(words.view(torch.uint8)) == 0, left
        assert torch.equal(out, want), left


@pytest.mark.parametrize("which", [UP, DOWN])
@pytest.mark.parametrize("wide", [False, True])
def test_a_product_reports_what_its_arrival_count_held(which, wide):
    """The count of CTAs that have drawn their last tile: a leftover in it, small
    enough for the last one to be found, is reported by the call that finds it."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    call, out, words, tiles = product(which, wide)
    call()
    want = out.clone()
    assert words[which:which + 2].tolist() == [0, 0]
    for left in (1, 2):
        words[which + 1] = left
        call()
        assert moe.last_device_status(words.view(torch.uint8)) == BOUNDS, left
        words[which:which + 2] = 0
        out.zero_()
        call()
        assert moe.last_device_status(words.view(torch.uint8)) == 0, left
        assert torch.equal(out, want), left


@pytest.mark.parametrize("which", [UP, DOWN])
def test_a_product_without_rows_has_nothing_to_report(which):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s, n = (64, 256, 256, 3, 1), 256
    mr = moe.capacity(s)[1]
    rows, w = moe.alloc_mxfp4(mr, n), moe.alloc_mxfp4(3 * n, n)
    out = torch.full((mr, n), -7.0, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        if which == UP:
            moe.moe_grouped_gemm_up_mxfp4(s, *rows, zero, zero, *w, *w, out, ws)
        else:
            moe.moe_grouped_gemm_down_mxfp4(s, *rows, zero, zero, *w, out, ws)
        assert moe.last_device_status(ws) == 0
        assert bool((out == -7.0).all())
        assert not ws.any()

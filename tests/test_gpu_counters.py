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


@pytest.mark.parametrize("T,E,k", [(3000, 64, 4), (700, 255, 3), (50000, 8, 2)])
def test_the_balance_loss_reports_what_its_counter_held(T, E, k):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (T, 128, 128, E, k)
    gen = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    ids = logits.topk(k, dim=1).indices.int().contiguous()
    counts, num = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, losses = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    ws = moe.alloc_balance_workspace(s)
    word = ws[:256].view(torch.int32)[60:61]          # the CTAs' counter

    def call():
        for t in (counts, num, P, losses):
            t.fill_(-5)
        moe.moe_balance_loss(s, logits, ids, None, counts, num, P, losses, ws)
        return moe.last_device_status(ws), [t.clone() for t in (counts, num, P, losses)]

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    status, want = call()
    assert status == 0 and word.item() == 0 and want[1].item() == T
    for left in (1, 2, 5, 9):                         # in the count: reported, and no harm done
        word.fill_(left)
        status, got = call()
        assert status == BOUNDS and same(got, want), left
        assert word.item() == 0
    for left in (1 << 10, 7 << 10, 1 << 20, 1 << 31, 0x12345678, -1):
        word.fill_(left - (1 << 32) if left >= 1 << 31 else left)
        assert call()[0] == BOUNDS, left
        word.zero_()
        status, got = call()
        assert status == 0 and same(got, want), left


def test_the_balance_loss_waits_for_its_slowest_cta():
    """A leftover of one, and one CTA with nearly all of the work: the CTA before it
    must not take itself for the last."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, E, k = 1 << 18, 256, 4
    s = (T, 128, 128, E, k)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    logits = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids = logits.topk(k, dim=1).indices.int().contiguous()
    mask = (torch.arange(T, device="cuda") // 64) % sms == 0      # CTA b takes the b-th 64 tokens of every 64 sms
    counts, num = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, losses = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    ws = moe.alloc_balance_workspace(s)
    word = ws[:256].view(torch.int32)[60:61]
    part = ws[256:]

    def call():
        for t in (counts, num, P, losses, part):
            t.zero_()
        moe.moe_balance_loss(s, logits, ids, mask, counts, num, P, losses, ws)
        return moe.last_device_status(ws), [t.clone() for t in (counts, num, P, losses)]

    status, want = call()
    assert status == 0 and want[1].item() == mask.sum().item()
    for _ in range(5):
        word.fill_(1)
        status, got = call()
        assert status == BOUNDS
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert word.item() == 0


@pytest.mark.parametrize("which", [UP, DOWN])
@pytest.mark.parametrize("wide", [False, True])
def test_counts_that_fit_alone_but_not_together_are_reported(which, wide):
    """Every expert is said to fill the buffers, of a shape whose tiles would then
    number past 32 bits.  The counts alone decide that nothing is loaded or stored
    (every expert's padded rows are empty, too), so the buffers can be small."""
    torch = need_gpu()
    import ctypes
    import combine_moe_route_04_gb300 as moe
    H, I = (128, 32768) if which == UP else (32768, 128)
    s = moe.shape(1 << 22, H, I, 256, 16 if wide else 1)       # 262144 or 16384 rows per expert
    if not wide:
        s.T = 256 * 256                                          # 256 rows per expert: the shorter windows
    mr = moe.capacity(s)[1]
    N = I if which == UP else H
    tiles = 256 * ((mr - 1) // (192 if wide else 128) + 1) * (N // 128 if which == UP else -(-N // 256))
    assert tiles >= 1 << 31 or not wide
    counts = torch.full((256,), mr, dtype=torch.int32, device="cuda")
    off = torch.zeros(257, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    small = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    p = small.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    a = [ctypes.byref(s), p, p, counts.data_ptr(), off.data_ptr()] + [p] * (4 if which == UP else 2) \
        + [p, ws.data_ptr(), stream]
    fn = moe.load().moe_grouped_gemm_up_mxfp4 if which == UP else moe.load().moe_grouped_gemm_down_mxfp4
    for _ in range(2):
        assert fn(*a) == 0
        assert moe.last_device_status(ws) == BOUNDS
        assert bool((small == 7).all()) and not ws.any()

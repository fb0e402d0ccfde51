"""MXFP4 and balance calls on buffers whose element offsets pass 2^32 (or 2^31):
the far end is checked against the same values handled on their own."""
import numpy as np
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_quantize_and_back_past_32_bits():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    rows, cols, tail = (1 << 20) + 77, 4096 + 128, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn((tail, cols), generator=g, device="cuda").bfloat16()
    x[: 128] = torch.randn((128, cols), generator=g, device="cuda").bfloat16()
    assert x.numel() > 1 << 32
    codes, scales = moe.alloc_mxfp4(rows, cols)
    moe.moe_quantize_mxfp4(x, rows, cols, codes, scales)
    back = torch.full((rows, cols), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(codes, scales, rows, cols, back)
    for part in (slice(0, 128), slice(rows - tail, rows)):
        y = x[part].clone()
        n = y.shape[0]
        c, s = moe.alloc_mxfp4(n, cols)
        moe.moe_quantize_mxfp4(y, n, cols, c, s)
        assert torch.equal(codes[part], c)
        want = torch.empty_like(y)
        moe.moe_dequantize_mxfp4(c, s, n, cols, want)
        assert torch.equal(back[part], want) and want.abs().sum() > 0
    assert not back[128:rows - tail].any()


def test_weights_past_32_bits():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    E, K, N = 130, 8192, 4096
    w = torch.zeros((E, K, N), dtype=torch.bfloat16, device="cuda")
    w[-1] = torch.randn((K, N), device="cuda").bfloat16()
    assert w.numel() > 1 << 32
    codes, scales = moe.alloc_mxfp4(E * N, K)
    moe.moe_quantize_weights_mxfp4(w, E, K, N, codes, scales)
    c, s = moe.alloc_mxfp4(N, K)
    moe.moe_quantize_mxfp4(w[-1].t().contiguous(), N, K, c, s)
    assert torch.equal(codes[-N:], c) and torch.equal(scales[-s.numel():], s)
    assert not codes[:-N].any()


def test_down_product_past_32_bits():
    """2^20 rows of 4224 columns: the last expert's rows as a call of their own gives them."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, I, E, k = (1 << 20) - 100, 4096 + 128, 256, 3, 1
    s = (T, H, I, E, k)
    mr = moe.capacity(s)[1]
    g = torch.Generator(device="cuda").manual_seed(2)
    counts = torch.tensor([T - 700, 0, 700], dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    assert int(off[2]) * H > 1 << 32
    h = torch.randn((mr, I), generator=g, device="cuda").bfloat16()
    hc, hs = moe.alloc_mxfp4(mr, I)
    moe.moe_quantize_mxfp4(h, mr, I, hc, hs)
    w = torch.randn((E, I, H), generator=g, device="cuda").bfloat16()
    wc, wsc = moe.alloc_mxfp4(E * H, I)
    moe.moe_quantize_weights_mxfp4(w, E, I, H, wc, wsc)
    Y = torch.full((mr, H), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_gemm_down_mxfp4(s, hc, hs, counts.cuda(), off.cuda(), wc, wsc, Y, ws)
    assert moe.last_device_status(ws) == 0
    first, n = int(off[2]), 700
    small = (n, H, I, 1, 1)
    smr = moe.capacity(small)[1]
    c1, s1 = moe.alloc_mxfp4(smr, I)
    moe.moe_quantize_mxfp4(h[first:first + smr].contiguous(), smr, I, c1, s1)
    w1, ws1 = moe.alloc_mxfp4(H, I)
    moe.moe_quantize_weights_mxfp4(w[2:3].contiguous(), 1, I, H, w1, ws1)
    want = torch.zeros((smr, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_down_mxfp4(small, c1, s1, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    torch.tensor([0, smr], dtype=torch.int32, device="cuda"), w1, ws1, want, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(Y[first:first + n], want[:n]) and want[:n].abs().sum() > 0
    assert bool((Y[first + n:] == -7.0).all())


def test_balance_at_the_largest_shape():
    """2^22 tokens of 256 experts: 4.3 GB of logits.  Every row is one of 64, so the
    definition needs only those in float64."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, E, k = 1 << 22, 256, 4
    rng = np.random.default_rng(5)
    base = (rng.standard_normal((64, E)) * 2).astype(np.float32)
    ids = np.argsort(-base, axis=1, kind="stable")[:, :k].astype(np.int32)
    logits = torch.from_numpy(base).cuda().repeat(T // 64, 1)
    picks = torch.from_numpy(ids).cuda().repeat(T // 64, 1)
    s = (T, 128, 128, E, k)
    counts, n = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, losses = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda")
    d = torch.full((T, E), 9.0, device="cuda")
    ws = moe.alloc_balance_workspace(s)
    moe.moe_balance_loss(s, logits, picks, None, counts, n, P, losses, ws)
    moe.moe_balance_loss_backward(s, logits, None, counts, n, torch.tensor([1.0, 1.0], device="cuda"), d)
    assert moe.last_device_status(ws) == 0
    x = base.astype(np.float64)
    ex = np.exp(x - x.max(1, keepdims=True))
    p = ex / ex.sum(1, keepdims=True)
    lse = x.max(1) + np.log(ex.sum(1))
    f = np.bincount(ids.ravel(), minlength=E) / (64 * k)
    assert n.item() == T and np.array_equal(counts.cpu().numpy(), np.bincount(ids.ravel(), minlength=E) * (T // 64))
    # sums of 2^22 / 152 / 32 terms per lane, each rounded: 2^-24 sqrt of that, and the terms' own error
    rel = 2.0 ** -24 * ((T / 152 / 32) ** 0.5 + 100)
    assert np.all(np.abs(P.cpu().numpy() - p.mean(0)) <= rel * p.mean(0))
    want = np.array([E * (f * p.mean(0)).sum(), (lse ** 2).mean()])
    assert np.all(np.abs(losses.cpu().numpy() - want) <= 2 * rel * want)
    wd = p * (E / T * (f - (p * f).sum(1, keepdims=True)) + 2 / T * lse[:, None])
    mag = p * (E / T * (np.abs(f - 1 / E) + (p * np.abs(f - 1 / E)).sum(1, keepdims=True))
               + 2 / T * np.abs(lse[:, None]))
    for at in (0, T // 2, T - 64):
        assert np.all(np.abs(d[at:at + 64].cpu().numpy() - wd) <= 2.0 ** -24 * 200 * mag)

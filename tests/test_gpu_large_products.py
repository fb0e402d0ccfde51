"""The MXFP4 gate/up product and the MXFP4 forward where element offsets of h pass
2^32: the far end is checked against a small call on the same rows."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def quantized(w):
    import combine_moe_route_04_gb300 as moe
    E, K, N = w.shape
    codes, scales = moe.alloc_mxfp4(E * N, K)
    moe.moe_quantize_weights_mxfp4(w, E, K, N, codes, scales)
    return codes, scales


def test_gate_up_product_past_32_bits():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, I, E = (1 << 20) - 100, 256, 4096 + 128, 3
    s = (T, H, I, E, 1)
    mr = moe.capacity(s)[1]
    g = torch.Generator(device="cuda").manual_seed(4)
    counts = torch.tensor([T - 700, 0, 700], dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    assert int(off[2]) * I > 1 << 32
    x = torch.randn((mr, H), generator=g, device="cuda").bfloat16()
    xq = moe.alloc_mxfp4(mr, H)
    moe.moe_quantize_mxfp4(x, mr, H, *xq)
    w = [(torch.randn((E, H, I), generator=g, device="cuda") / 16).bfloat16() for _ in range(2)]
    q = [t for v in w for t in quantized(v)]
    h = torch.full((mr, I), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_gemm_up_mxfp4(s, *xq, counts.cuda(), off.cuda(), *q, h, ws)
    assert moe.last_device_status(ws) == 0
    first, n = int(off[2]), 700
    small = (n, H, I, 1, 1)
    smr = moe.capacity(small)[1]
    x1 = moe.alloc_mxfp4(smr, H)
    moe.moe_quantize_mxfp4(x[first:first + smr].contiguous(), smr, H, *x1)
    q1 = [t for v in w for t in quantized(v[2:3].contiguous())]
    want = torch.zeros((smr, I), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_up_mxfp4(small, *x1, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                  torch.tensor([0, smr], dtype=torch.int32, device="cuda"), *q1, want, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(h[first:first + n], want[:n]) and want[:n].abs().sum() > 0
    assert bool((h[first + n:] == -7.0).all())
    assert bool((h[T - 700:first] == -7.0).all())


def test_forward_past_32_bits():
    """2^20 routed rows of 4224 columns in 4 bits: each token's result is that of a
    forward of a few hundred tokens."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, I, E, k, n = 1 << 19, 256, 4096 + 128, 4, 2, 400
    assert T * k * I > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn((T, E), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    q = [t for K, N in ((H, I), (H, I), (I, H))
         for t in quantized((torch.randn((E, K, N), generator=g, device="cuda") / K ** 0.5).bfloat16())]
    s = (T, H, I, E, k)
    ws = moe.alloc_mxfp4_workspace(s)
    out = torch.zeros_like(x)
    moe.moe_forward_mxfp4(s, logits, x, *q, out, ws)
    assert moe.last_device_status(ws) == 0
    small = (n, H, I, E, k)
    sws = moe.alloc_mxfp4_workspace(small)
    for at in (0, T // 2, T - n):
        want = torch.zeros((n, H), dtype=torch.bfloat16, device="cuda")
        moe.moe_forward_mxfp4(small, logits[at:at + n].contiguous(), x[at:at + n].contiguous(), *q, want, sws)
        assert moe.last_device_status(sws) == 0
        assert torch.equal(out[at:at + n], want) and want.abs().sum() > 0

"""The backward products, the combine's gradient and the 8-bit calls where element
offsets pass 2^31 and 2^32: the far end against a small call on the same rows."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T, N, E = (1 << 20) - 100, 4096 + 128, 3
COUNTS = [T - 700, 0, 700]


@pytest.fixture(scope="module")
def moe():
    need_gpu()
    import combine_moe_route_04_gb300 as m
    yield m
    torch.cuda.empty_cache()


def layout():
    counts = torch.tensor(COUNTS, dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    assert int(off[2]) * N > 1 << 32
    return counts.cuda(), off.cuda(), int(off[2])


def normal(gen, *shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda")
    return out


def small(moe, H, I):
    s = (700, H, I, 1, 1)
    R = moe.capacity(s)[1]
    return s, R, torch.tensor([700], dtype=torch.int32, device="cuda"), torch.tensor([0, R], dtype=torch.int32, device="cuda")


def test_backward_products_of_wide_hidden_rows(moe):
    """dg, du and the weights' gradients with 2^20 rows of 4224 columns on the side of I."""
    H = 128
    s = (T, H, N, E, 1)
    R = moe.capacity(s)[1]
    counts, off, first = layout()
    gen = torch.Generator(device="cuda").manual_seed(1)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dy, x, wd = normal(gen, R, H), normal(gen, R, H), normal(gen, E, N, H)
    g, u = normal(gen, R, N), normal(gen, R, N)
    dg, du = torch.full_like(g, -7.5), torch.full_like(u, -7.5)
    moe.moe_grouped_gemm_down_backward(s, dy, counts, off, wd, g, u, dg, du, ws)
    s1, R1, c1, o1 = small(moe, H, N)
    at = slice(first, first + R1)
    dg1, du1 = torch.zeros((R1, N), dtype=torch.bfloat16, device="cuda"), torch.zeros((R1, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_down_backward(s1, dy[at], c1, o1, wd[2], g[at], u[at], dg1, du1, ws)
    assert moe.last_device_status(ws) == 0
    for big, little in ((dg, dg1), (du, du1)):
        assert torch.equal(big[first:first + 700], little[:700]) and little[:700].any()
        assert (big[first + 700:] == -7.5).all() and (big[T - 700:first] == -7.5).all()
    wg, wu = normal(gen, E, H, N), normal(gen, E, H, N)
    dx, dx1 = torch.full_like(dy, -7.5), torch.zeros_like(dy[at])
    moe.moe_grouped_gemm_up_backward(s, dg, du, counts, off, wg, wu, dx, ws)
    moe.moe_grouped_gemm_up_backward(s1, dg1, du1, c1, o1, wg[2], wu[2], dx1, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(dx[first:first + 700], dx1[:700]) and (dx[first + 700:] == -7.5).all()
    big = [torch.zeros_like(w) for w in (wg, wu, wd)]
    little = [torch.zeros_like(w[:1]) for w in (wg, wu, wd)]
    moe.moe_grouped_gemm_weight_backward(s, x, g, dg, du, dy, counts, off, *big, ws)
    moe.moe_grouped_gemm_weight_backward(s1, x[at], g[at], dg1, du1, dy[at], c1, o1, *little, ws)
    assert moe.last_device_status(ws) == 0
    for b, l in zip(big, little):
        assert torch.equal(b[2], l[0]) and not b[1].any() and b[0].any()


def test_wide_token_rows(moe):
    """dX, the combine's gradients and the 8-bit down product with 2^20 rows of 4224 columns on the side of H."""
    I = 128
    s = (T, N, I, E, 1)
    R = moe.capacity(s)[1]
    counts, off, first = layout()
    gen = torch.Generator(device="cuda").manual_seed(2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dg, du, wg, wu = normal(gen, R, I), normal(gen, R, I), normal(gen, E, N, I), normal(gen, E, N, I)
    dx = torch.full((R, N), -7.5, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_up_backward(s, dg, du, counts, off, wg, wu, dx, ws)
    s1, R1, c1, o1 = small(moe, N, I)
    at = slice(first, first + R1)
    want = torch.zeros((R1, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_up_backward(s1, dg[at], du[at], c1, o1, wg[2], wu[2], want, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(dx[first:first + 700], want[:700]) and (dx[first + 700:] == -7.5).all()
    # the combine's gradients: a token's row far out
    y = dx
    dout = normal(gen, T, N)
    rows = torch.cat((torch.arange(T - 700), torch.arange(first, first + 700))).int().cuda().reshape(T, 1)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 0.5, device="cuda")
    dy, dl = torch.full_like(y, -7.5), torch.full((T, E), -7.5, device="cuda")
    moe.moe_combine_backward(s, y, rows, ids, w, dout, dy, dl, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(dy[first:first + 700], dout[T - 700:] * 0.5)
    assert (dy[first + 700:] == -7.5).all() and not dl[:, 1:].any()
    dX = torch.empty_like(dout)
    moe.moe_permute_backward(s, dy, rows, dX, ws)
    assert moe.last_device_status(ws) == 0 and torch.equal(dX, dout * 0.5)
    del dout, dX, dy, dl
    # 8 bits: rows quantised and multiplied
    codes, scales = moe.alloc_int8(R, N)
    moe.moe_quantize_int8(y, R, N, codes, scales)
    c1q, s1q = moe.alloc_int8(R1, N)
    moe.moe_quantize_int8(y[at], R1, N, c1q, s1q)
    assert torch.equal(codes[at], c1q) and torch.equal(scales[at], s1q)
    back = torch.empty_like(y)
    moe.moe_dequantize_int8(codes, scales, R, N, back)
    b1 = torch.empty_like(y[at])
    moe.moe_dequantize_int8(c1q, s1q, R1, N, b1)
    assert torch.equal(back[at], b1)
    hq, hz = torch.randint(-127, 128, (R, I), generator=gen, device="cuda").to(torch.int8), torch.rand(R, generator=gen, device="cuda")
    wq, wz = torch.randint(-127, 128, (E * N, I), generator=gen, device="cuda").to(torch.int8), torch.rand(E * N, generator=gen, device="cuda")
    back.fill_(-7.5)
    moe.moe_grouped_gemm_down_int8(s, hq, hz, counts, off, wq, wz, back, ws)
    moe.moe_grouped_gemm_down_int8(s1, hq[at], hz[at], c1, o1, wq[2 * N:], wz[2 * N:], b1, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(back[first:first + 700], b1[:700]) and (back[first + 700:] == -7.5).all()
    # and the gate/up product, whose operand they are
    s2, s3 = (T, N, 128, E, 1), (700, N, 128, 1, 1)
    g = [torch.randint(-127, 128, (E * 128, N), generator=gen, device="cuda").to(torch.int8) for _ in range(2)]
    z = [torch.rand(E * 128, generator=gen, device="cuda") / N for _ in range(2)]
    h, h1 = torch.full((R, 128), -7.5, dtype=torch.bfloat16, device="cuda"), torch.zeros((R1, 128), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_up_int8(s2, codes, scales, counts, off, g[0], z[0], g[1], z[1], h, ws)
    moe.moe_grouped_gemm_up_int8(s3, c1q, s1q, c1, o1, g[0][256:], z[0][256:], g[1][256:], z[1][256:], h1, ws)
    assert moe.last_device_status(ws) == 0
    assert torch.equal(h[first:first + 700], h1[:700]) and (h[first + 700:] == -7.5).all()


def test_training_forward_of_wide_hidden_rows(moe):
    """g, u and h past 2^32 elements."""
    H = 128
    s = (T, H, N, E, 1)
    R = moe.capacity(s)[1]
    counts, off, first = layout()
    gen = torch.Generator(device="cuda").manual_seed(3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x, wg, wu = normal(gen, R, H), normal(gen, E, H, N), normal(gen, E, H, N)
    outs = [torch.full((R, N), -7.5, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_grouped_gemm_up_train(s, x, counts, off, wg, wu, *outs, ws)
    s1, R1, c1, o1 = small(moe, H, N)
    want = [torch.zeros((R1, N), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_grouped_gemm_up_train(s1, x[first:first + R1], c1, o1, wg[2], wu[2], *want, ws)
    assert moe.last_device_status(ws) == 0
    for b, l in zip(outs, want):
        assert torch.equal(b[first:first + 700], l[:700]) and l[:700].any()
        assert (b[first + 700:] == -7.5).all() and (b[T - 700:first] == -7.5).all()

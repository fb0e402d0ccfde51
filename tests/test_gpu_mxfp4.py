"""MXFP4: quantisation to the bit, the grouped products against float64, and the
layer's forward against its own steps."""
import numpy as np
import pytest

import mxfp4_ref as ref
from gpu_util import f32, host_u16, need_gpu, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def bf16_bits(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def hard_rows(rows, cols, seed):
    """bf16 bits with what rounding can go wrong on: ties, zeros of both signs,
    subnormals, the largest values, blocks of one value and of mixed scales."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    b = x.reshape(rows, -1, 32)
    kind = rng.integers(0, 8, b.shape[:2])
    b[kind == 0] = 0.0
    b[kind == 1] = -0.0
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 4.0])
    t = rng.choice(ties, b.shape) * rng.choice([-1.0, 1.0], b.shape)
    b[kind == 2] = t[kind == 2]
    bits = bf16_bits(x)
    v = bits.reshape(rows, -1, 32)
    tiny = rng.integers(0, 0x0300, v.shape).astype(np.uint16) | (rng.integers(0, 2, v.shape).astype(np.uint16) << 15)
    v[kind == 3] = tiny[kind == 3]                       # subnormals and the smallest normals
    huge = rng.integers(0x7E00, 0x7F80, v.shape).astype(np.uint16)
    v[kind == 4] = huge[kind == 4]
    return bits


def to64(bits):
    return f32(bits).astype(np.float64)


def run_quantize(bits):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    rows, cols = bits.shape
    codes, scales = moe.alloc_mxfp4(rows, cols)
    scales.fill_(77)
    moe.moe_quantize_mxfp4(to_dev_bf16(bits), rows, cols, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (127, 1408), (128, 1024), (129, 640), (300, 2176),
                                       (5, 32768)])
def test_quantize_and_back_to_the_bit(rows, cols):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    bits = hard_rows(rows, cols, rows + cols)
    codes, scales = run_quantize(bits)
    want_c, want_s, want_v = ref.quantize(to64(bits))
    assert np.array_equal(scales.cpu().numpy(), want_s)   # padding rows' scales are 0
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(codes, scales, rows, cols, back)
    assert np.array_equal(to64(host_u16(back)), want_v)


def test_blocks_with_nan_or_infinity_read_as_nan():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    bits = hard_rows(4, 256, 3)
    bits[0, 5], bits[1, 40], bits[2, 255], bits[3, 64] = 0x7FC0, 0x7F80, 0xFF80, 0xFFFF
    codes, scales = run_quantize(bits)
    want_c, want_s, want_v = ref.quantize(to64(bits))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    back = torch.empty((4, 256), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(codes, scales, 4, 256, back)
    got = to64(host_u16(back))
    assert np.array_equal(got, want_v, equal_nan=True)
    assert np.isnan(got).sum() == 4 * 32


def test_dequantize_every_code_under_every_scale():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    rng = np.random.default_rng(0)
    c = rng.integers(0, 16, (256, 128)).astype(np.uint8)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)
    back = torch.empty((256, 128), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(to_dev(ref.pack(c)), to_dev(ref.tile(s)), 256, 128, back)
    want = ref.values(c, s)
    want[np.abs(want) > 3.3895313892515355e38] *= np.inf   # bf16's largest
    assert np.array_equal(to64(host_u16(back)), want, equal_nan=True)


@pytest.mark.parametrize("E,K,N", [(1, 128, 128), (2, 384, 256), (3, 256, 640), (5, 1408, 128)])
def test_weights_quantize_as_their_transpose(E, K, N):
    need_gpu()
    import combine_moe_route_04_gb300 as moe
    bits = hard_rows(E * N, K, E + K + N)
    bits[0, 3], bits[-1, K - 1] = 0x7F80, 0x7FC1
    w = np.ascontiguousarray(bits.reshape(E, N, K).transpose(0, 2, 1))
    codes, scales = moe.alloc_mxfp4(E * N, K)
    moe.moe_quantize_weights_mxfp4(to_dev_bf16(w), E, K, N, codes, scales)
    want_c, want_s, _ = ref.quantize(to64(bits))
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s)


# ------------------------------------------------------------------ products
def operands(counts, K, N, mats, seed, garbage=True):
    """Rows in expert order and weights as MXFP4, on the host: padding rows hold
    garbage codes under NaN scales.  Values are N(0, 1) and N(0, 1/K)."""
    rng = np.random.default_rng(seed)
    counts = np.asarray(counts)
    off = np.concatenate(([0], np.cumsum((counts + 127) // 128 * 128)))
    E = len(counts)
    x = rng.standard_normal((off[-1], K))
    s = ref.scale_bytes(x)
    c = ref.codes_of(x, s)
    real = np.zeros(off[-1], bool)
    for e in range(E):
        real[off[e]:off[e] + counts[e]] = True
    if garbage:
        s[~real] = 255
        c[~real] = 15
    rows = (c, s)
    ws = []
    for _ in range(mats):
        w = rng.standard_normal((E * N, K)) / np.sqrt(K)
        sw = ref.scale_bytes(w)
        ws.append((ref.codes_of(w, sw), sw))
    return rows, ws, off, real


def padded(a, rows, fill):
    out = np.full((rows,) + a.shape[1:], fill, a.dtype)
    out[:a.shape[0]] = a
    return out


def matmul64(rows, w, off, counts, N):
    """(x w^T, |x| |w|^T) per real row."""
    x, wv = np.nan_to_num(ref.values(*rows)), ref.values(*w)
    y = np.zeros((off[-1], N))
    mag = np.zeros((off[-1], N))
    for e, n in enumerate(counts):
        a, b = x[off[e]:off[e] + n], wv[e * N:(e + 1) * N]
        y[off[e]:off[e] + n] = a @ b.T
        mag[off[e]:off[e] + n] = np.abs(a) @ np.abs(b).T
    return y, mag


def bounds(K, y, mag):
    """float32 accumulation of K products, each sum off by at most an ulp of a
    partial sum: K 2^-23 of the absolute products."""
    return K * 2.0 ** -23 * mag


COUNTS = [
    [1], [0, 1, 0], [63, 64, 65, 0], [128, 127, 129], [192, 193, 191], [0, 0, 400, 5], [257, 16, 17, 15],
    [1025, 0, 577, 769, 1] + 8 * [0],
]


def shape_for(counts, H, I, wide=False):
    """A shape whose capacity holds these counts (T k rows over E experts); wide:
    one with over 256 rows per expert, for which the products cut other windows."""
    T = max(1, sum(counts))
    return (max(T, 257 * len(counts)) if wide else T, H, I, len(counts), 1)


def upload(rows, off, max_rows):
    c, s = rows
    return to_dev(padded(ref.pack(c), max_rows, 0xFF)), to_dev(ref.tile(padded(s, max_rows, 255)))


def up_call(counts, H, I, seed, rows=None, wide=False):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    r, ws, off, real = operands(counts, H, I, 2, seed)
    if rows is not None:
        r = rows(r, off)
    s = shape_for(counts, H, I, wide)
    mr = moe.capacity(s)[1]
    xc, xs = upload(r, off, mr)
    h = torch.full((mr, I), -7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dev = [t for c, sc in ws for t in (to_dev(ref.pack(c)), to_dev(ref.tile(sc)))]
    moe.moe_grouped_gemm_up_mxfp4(s, xc, xs, to_dev(np.array(counts, np.int32)), to_dev(off.astype(np.int32)), *dev,
                                  h, status)
    assert moe.last_device_status(status) == 0
    return to64(host_u16(h)), r, ws, off, real


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,I", [(128, 128), (384, 256), (1024, 384)])
def test_up_product_against_64_bits(counts, H, I, wide):
    got, r, ws, off, real = up_call(counts, H, I, sum(counts) + H, wide=wide)
    g, gm = matmul64(r, ws[0], off, counts, I)
    u, um = matmul64(r, ws[1], off, counts, I)
    sig = 1.0 / (1.0 + np.exp(-g))
    want = g * sig * u
    eg, eu = bounds(H, g, gm), bounds(H, u, um)
    # |silu'| <= 1.1; the sigmoid's fast exp and divide are within 2^-19 of it
    tol = 1.1 * eg * np.abs(u) + np.abs(g * sig) * eu + 1.1 * eg * eu + (2.0 ** -19 + 2.0 ** -8) * np.abs(want) + 1e-30
    assert np.all(np.abs(got[:off[-1]] - want)[real] <= tol[real])
    assert np.all(got[:off[-1]][~real] == -7.0) and np.all(got[off[-1]:] == -7.0)   # padding rows stay unwritten


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,I", [(128, 128), (384, 256), (640, 1152)])
def test_down_product_against_64_bits(counts, H, I, wide):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    r, ws, off, real = operands(counts, I, H, 1, sum(counts) + H)
    s = shape_for(counts, H, I, wide)
    mr = moe.capacity(s)[1]
    hc, hs = upload(r, off, mr)
    Y = torch.full((mr, H), -7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_gemm_down_mxfp4(s, hc, hs, to_dev(np.array(counts, np.int32)), to_dev(off.astype(np.int32)),
                                    to_dev(ref.pack(ws[0][0])), to_dev(ref.tile(ws[0][1])), Y, status)
    assert moe.last_device_status(status) == 0
    got = to64(host_u16(Y))
    want, mag = matmul64(r, ws[0], off, counts, H)
    tol = bounds(I, want, mag) + 2.0 ** -8 * np.abs(want) + 1e-30
    assert np.all(np.abs(got[:off[-1]] - want)[real] <= tol[real])
    assert np.all(got[:off[-1]][~real] == -7.0) and np.all(got[off[-1]:] == -7.0)


@pytest.mark.parametrize("seed", range(10))
def test_products_of_random_shapes(seed):
    """Random expert counts (empty ones among them), sizes and windows, both products."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    rng = np.random.default_rng(100 + seed)
    E = int(rng.integers(1, 40))
    counts = (rng.integers(0, 1 + int(np.exp(rng.uniform(0, 6.2))), E) * (rng.random(E) < 0.8)).tolist()
    H, I = (128 * int(rng.integers(1, 7)) for _ in range(2))
    wide = bool(rng.integers(0, 2))
    got, r, ws, off, real = up_call(counts, H, I, seed, wide=wide)
    g, gm = matmul64(r, ws[0], off, counts, I)
    u, um = matmul64(r, ws[1], off, counts, I)
    sig = 1.0 / (1.0 + np.exp(-g))
    want = g * sig * u
    eg, eu = bounds(H, g, gm), bounds(H, u, um)
    tol = 1.1 * eg * np.abs(u) + np.abs(g * sig) * eu + 1.1 * eg * eu + (2.0 ** -19 + 2.0 ** -8) * np.abs(want) + 1e-30
    assert np.all(np.abs(got[:off[-1]] - want)[real] <= tol[real])
    assert np.all(got[:off[-1]][~real] == -7.0)
    s = shape_for(counts, H, I, wide)
    mr = moe.capacity(s)[1]
    r, ws, off, real = operands(counts, I, H, 1, 50 + seed)
    hc, hs = upload(r, off, mr)
    Y = torch.full((mr, H), -7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (s, hc, hs, to_dev(np.array(counts, np.int32)), to_dev(off.astype(np.int32)), to_dev(ref.pack(ws[0][0])),
            to_dev(ref.tile(ws[0][1])), Y, status)
    moe.moe_grouped_gemm_down_mxfp4(*args)
    got = to64(host_u16(Y))
    want, mag = matmul64(r, ws[0], off, counts, H)
    tol = bounds(I, want, mag) + 2.0 ** -8 * np.abs(want) + 1e-30
    assert np.all(np.abs(got[:off[-1]] - want)[real] <= tol[real])
    moe.moe_grouped_gemm_down_mxfp4(*args)
    assert moe.last_device_status(status) == 0
    assert np.array_equal(to64(host_u16(Y)), got)      # the same bits again


def test_a_tile_counter_that_was_not_cleared_is_reported():
    """As for the bf16 products: the call that finds it dirty says so, the next is sound."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    counts, H, I = [300, 5, 0, 129], 256, 512
    r, ws, off, real = operands(counts, I, H, 1, 3)
    s = shape_for(counts, H, I)
    mr = moe.capacity(s)[1]
    hc, hs = upload(r, off, mr)
    Y = torch.zeros((mr, H), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (s, hc, hs, to_dev(np.array(counts, np.int32)), to_dev(off.astype(np.int32)), to_dev(ref.pack(ws[0][0])),
            to_dev(ref.tile(ws[0][1])), Y, status)
    moe.moe_grouped_gemm_down_mxfp4(*args)
    assert moe.last_device_status(status) == 0
    want = Y.clone()
    status.view(torch.int32)[32] = 1 << 20            # the down product's counter
    moe.moe_grouped_gemm_down_mxfp4(*args)
    assert moe.last_device_status(status) == 7
    Y.zero_()
    moe.moe_grouped_gemm_down_mxfp4(*args)
    assert moe.last_device_status(status) == 0
    assert torch.equal(Y, want)


def test_scales_far_apart_and_a_nan_block():
    """Every row and block with a scale of its own; one block of one row NaN:
    that row, and only it, is NaN."""
    counts, H, I = [70, 3], 512, 128

    def spread(r, off):
        c, s = r
        rng = np.random.default_rng(1)
        s = np.where(s == 255, 255, s.astype(int) + rng.integers(-12, 13, s.shape)).astype(np.uint8)
        s[65, 9] = 255
        return c, s

    got, r, ws, off, real = up_call(counts, H, I, 5, spread)
    assert np.isnan(got[65]).all()
    real[65] = False
    assert np.isfinite(got[:off[-1]][real]).all()
    g, gm = matmul64(r, ws[0], off, counts, I)
    u, um = matmul64(r, ws[1], off, counts, I)
    sig = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    want = g * sig * u
    eg, eu = bounds(H, g, gm), bounds(H, u, um)
    tol = 1.1 * eg * np.abs(u) + np.abs(g * sig) * eu + 1.1 * eg * eu \
        + (2.0 ** -18 * (1 + np.abs(g)) + 2.0 ** -8) * np.abs(want) + 1e-30
    assert np.all(np.abs(got[:off[-1]] - want)[real] <= tol[real])


# ------------------------------------------------------------------ the layer
def layer_inputs(T, H, I, E, k, seed, skew=0.0):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((T, E), generator=g, device="cuda") - skew * torch.log(torch.arange(1, E + 1, device="cuda"))
    X = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    q = []
    for K, N in ((H, I), (H, I), (I, H)):
        w = (torch.randn((E, K, N), generator=g, device="cuda") / K ** 0.5).bfloat16()
        codes, scales = moe.alloc_mxfp4(E * N, K)
        moe.moe_quantize_weights_mxfp4(w, E, K, N, codes, scales)
        q += [codes, scales]
    return logits, X, q


def steps(s, logits, X, q):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, H, I, E, k = s
    mr = moe.capacity(s)[1]
    bufs = moe.alloc_route_outputs(s)
    ws = moe.alloc_workspace(s)
    moe.moe_route(s, logits, bufs["topk_ids"], bufs["topk_w"], bufs["counts"], bufs["off_pad"], bufs["block_expert"],
                  bufs["num_blocks"], bufs["gather_idx"], bufs["scatter_idx"], ws)
    xc, xs = moe.alloc_mxfp4(mr, H)
    moe.moe_quantize_permute_mxfp4(s, X, bufs["scatter_idx"], xc, xs, ws)
    h = torch.zeros((mr, I), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_up_mxfp4(s, xc, xs, bufs["counts"], bufs["off_pad"], *q[:4], h, ws)
    hc, hs = moe.alloc_mxfp4(mr, I)
    moe.moe_quantize_mxfp4(h, mr, I, hc, hs)
    Y = torch.zeros((mr, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_down_mxfp4(s, hc, hs, bufs["counts"], bufs["off_pad"], *q[4:], Y, ws)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_combine(s, Y, bufs["scatter_idx"], bufs["topk_w"], out, ws)
    assert moe.last_device_status(ws) == 0
    return out, (xc, xs, bufs)


SHAPES = [(1, 128, 128, 1, 1, 0.0), (5, 256, 128, 8, 8, 0.0), (128, 256, 512, 8, 2, 0.0), (333, 640, 384, 7, 3, 0.0),
          (700, 384, 256, 16, 4, 3.0), (1500, 256, 256, 4, 2, 0.5), (64, 1152, 640, 256, 16, 0.0)]


@pytest.mark.parametrize("T,H,I,E,k,skew", SHAPES)
def test_forward_is_its_steps_to_the_bit(T, H, I, E, k, skew):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (T, H, I, E, k)
    logits, X, q = layer_inputs(*s, seed=T + H, skew=skew)
    want, (xc, xs, bufs) = steps(s, logits, X, q)
    out = torch.empty_like(want)
    ws = moe.alloc_mxfp4_workspace(s)
    for _ in range(2):
        out.fill_(3.0)
        moe.moe_forward_mxfp4(s, logits, X, *q, out, ws)
        assert moe.last_device_status(ws) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    # quantise + permute = quantise, then take the rows
    codes, scales = moe.alloc_mxfp4(T, H)
    moe.moe_quantize_mxfp4(X, T, H, codes, scales)
    at = bufs["scatter_idx"].long().flatten()
    assert torch.equal(xc[at], codes.repeat_interleave(k, 0))
    back = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(codes, scales, T, H, back)
    perm = torch.empty((xc.shape[0], H), dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(xc, xs, xc.shape[0], H, perm)
    assert torch.equal(perm[at], back.repeat_interleave(k, 0))


def test_forward_on_a_stream_and_in_a_graph():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (96, 256, 256, 8, 2)
    logits, X, q = layer_inputs(*s, seed=9)
    want, _ = steps(s, logits, X, q)
    out = torch.empty_like(want)
    ws = moe.alloc_mxfp4_workspace(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.moe_forward_mxfp4(s, logits, X, *q, out, ws, stream=side)
    assert moe.last_device_status(ws, stream=side) == 0
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_mxfp4(s, logits, X, *q, out, ws)
    X.neg_()          # a replay reads what the buffers hold then
    want, _ = steps(s, logits, X, q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_forward_is_near_the_layer_in_64_bits():
    """Against the layer on the values the 4-bit operands stand for, in float64;
    h in between is quantised from the float64 h, so a value next to a rounding
    boundary may fall on the other side: the Frobenius error stays small."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = T, H, I, E, k = (200, 512, 384, 6, 2)
    logits, X, q = layer_inputs(*s, seed=4)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_mxfp4_workspace(s)
    moe.moe_forward_mxfp4(s, logits, X, *q, out, ws)
    assert moe.last_device_status(ws) == 0

    def val(codes, scales, rows, cols):
        v = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        moe.moe_dequantize_mxfp4(codes, scales, rows, cols, v)
        return to64(host_u16(v))

    wg, wu = val(q[0], q[1], E * I, H).reshape(E, I, H), val(q[2], q[3], E * I, H).reshape(E, I, H)
    wd = val(q[4], q[5], E * H, I).reshape(E, H, I)
    x = ref.quantize(to64(host_u16(X)))[2]
    lg = logits.cpu().numpy().astype(np.float64)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    w = np.exp(np.take_along_axis(lg, ids, 1))
    w /= w.sum(1, keepdims=True)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            g, u = wg[e] @ x[t], wu[e] @ x[t]
            h = ref.quantize(to64(bf16_bits((g / (1 + np.exp(-g)) * u)[None])))[2][0]
            want[t] += w[t, j] * (wd[e] @ h)
    got = to64(host_u16(out))
    assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


# ------------------------------------------------------------------ refusals
def test_refusals():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    codes, scales = moe.alloc_mxfp4(4, 256)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_quantize_mxfp4(x, 4, 200, codes, scales)          # not a multiple of 128
    assert ei.value.code == 2
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(x, 5, 256, codes, scales)          # buffers too small
    with pytest.raises(TypeError):
        moe.moe_quantize_mxfp4(x.float(), 4, 256, codes, scales)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(x.t(), 4, 256, codes, scales)      # not contiguous
    with pytest.raises(ValueError):
        moe.moe_dequantize_mxfp4(codes, scales[:-1], 4, 256, x)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(x.cpu(), 4, 256, codes, scales)
    s = (4, 256, 128, 2, 1)
    with pytest.raises(ValueError):
        moe.moe_forward_mxfp4(s, torch.zeros((4, 2), device="cuda"), x, codes, scales, codes, scales, codes, scales,
                              x, moe.alloc_mxfp4_workspace(s))


def test_counts_out_of_range_are_reported():
    """A count beyond an expert's padded rows: the kernel skips the tile and says so."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (64, 128, 128, 2, 1)
    mr = moe.capacity(s)[1]
    xc, xs = moe.alloc_mxfp4(mr, 128)
    wc, wsc = moe.alloc_mxfp4(2 * 128, 128)
    for t in (xc, xs, wc, wsc):
        t.zero_()
    h = torch.zeros((mr, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_up_mxfp4(s, xc, xs, torch.tensor([200, 1], **i32), torch.tensor([0, 128, 256], **i32), wc, wsc,
                                  wc, wsc, h, ws)
    assert moe.last_device_status(ws) == 7
    for counts, off, want in (([60, 4], [0, 128, 128 * 64], 7), ([60, 4], [0, 100, 256], 7),
                              ([60, 4], [128, 0, 128], 7), ([1 << 30, 4], [0, 128, 256], 7),
                              ([-5, 4], [0, 128, 256], 0)):
        moe.moe_grouped_gemm_up_mxfp4(s, xc, xs, torch.tensor(counts, **i32), torch.tensor(off, **i32), wc, wsc, wc,
                                      wsc, h, ws)
        assert moe.last_device_status(ws) == want
    moe.moe_grouped_gemm_up_mxfp4(s, xc, xs, torch.tensor([60, 4], **i32), torch.tensor([0, 128, 256], **i32), wc, wsc,
                                  wc, wsc, h, ws)
    assert moe.last_device_status(ws) == 0

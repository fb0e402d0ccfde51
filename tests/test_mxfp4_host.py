"""CPU checks of the MXFP4 and balance calls' host side, and hand-worked cases of
the reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import mxfp4_ref as ref


@pytest.fixture(scope="module")
def moe():
    from combine_moe_route_04_gb300 import _build
    _build.build()
    import combine_moe_route_04_gb300 as m
    m.load()
    return m


GOOD = 1 << 20   # never dereferenced: validation fails first
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


def test_sizes(moe):
    assert moe.mxfp4_sizes(1, 128) == (64, 512)
    assert moe.mxfp4_sizes(128, 256) == (128 * 128, 1024)
    assert moe.mxfp4_sizes(129, 4096) == (129 * 2048, 256 * 128)
    for rows, cols in [(0, 128), (-1, 128), (1 << 31, 128), (4, 0), (4, 64), (4, 200), (4, 32768 + 128)]:
        with pytest.raises(moe.MoEError) as ei:
            moe.mxfp4_sizes(rows, cols)
        assert ei.value.code == SHAPE
    c = ctypes.c_size_t()
    assert moe.load().moe_mxfp4_sizes(1, 128, None, ctypes.byref(c)) == INVALID


def test_workspaces(moe):
    for s in [(1, 128, 128, 1, 1), (2048, 4096, 1536, 64, 8), (1 << 22, 128, 128, 256, 16)]:
        T, H, I, E, k = s
        mr = moe.capacity(s)[1]
        need = mr * H // 2 + mr * H // 32 + mr * I // 2 + mr * I // 32 + mr * H * 2
        assert need <= moe.mxfp4_workspace_size(s) <= moe.workspace_size(s) + mr * (H + I) + (1 << 20)
        assert moe.balance_workspace_size(s) <= 1 << 20
    for f in (moe.mxfp4_workspace_size, moe.balance_workspace_size):
        with pytest.raises(moe.MoEError):
            f((4, 100, 128, 2, 1))


def calls(moe):
    """(function, arguments with every pointer GOOD, indexes of the pointers that may not be NULL)"""
    s = moe.shape(128, 256, 512, 8, 2)
    p = ctypes.byref(s)
    lib = moe.load()
    g = GOOD
    yield lib.moe_quantize_mxfp4, [g, 4, 256, g, g, None], [0, 3, 4]
    yield lib.moe_quantize_weights_mxfp4, [g, 2, 256, 128, g, g, None], [0, 4, 5]
    yield lib.moe_dequantize_mxfp4, [g, g, 4, 256, g, None], [0, 1, 4]
    yield lib.moe_quantize_permute_mxfp4, [p] + [g] * 5 + [None], range(1, 6)
    yield lib.moe_grouped_gemm_up_mxfp4, [p] + [g] * 10 + [None], range(1, 11)
    yield lib.moe_grouped_gemm_down_mxfp4, [p] + [g] * 8 + [None], range(1, 9)
    yield lib.moe_forward_mxfp4, [p] + [g] * 10 + [None], range(1, 11)
    yield lib.moe_balance_loss, [p, g, g, None] + [g] * 5 + [None], [1, 2, 4, 5, 6, 7, 8]
    yield lib.moe_balance_loss_backward, [p, g, None] + [g] * 4 + [None], [1, 3, 4, 5, 6]


def test_null_and_misaligned_pointers_refused(moe):
    seen = 0
    for fn, args, ptrs in calls(moe):
        for i in ptrs:
            for bad, code in ((None, INVALID), (GOOD + 8, MISALIGNED)):
                a = list(args)
                a[i] = bad
                assert fn(*a) == code, (fn.__name__, i)
                seen += 1
    assert seen == 2 * (3 + 3 + 3 + 5 + 10 + 8 + 10 + 7 + 5)


def test_shapes_refused(moe):
    lib = moe.load()
    bad = moe.shape(128, 200, 512, 8, 2)
    for fn, args, _ in calls(moe):
        a = list(args)
        if isinstance(a[0], int):
            continue
        a[0] = ctypes.byref(bad)
        assert fn(*a) == SHAPE, fn.__name__
        a[0] = None
        assert fn(*a) == INVALID, fn.__name__
    g = GOOD
    for rows, cols in [(0, 256), (4, 130), (4, 1 << 16)]:
        assert lib.moe_quantize_mxfp4(g, rows, cols, g, g, None) == SHAPE
        assert lib.moe_dequantize_mxfp4(g, g, rows, cols, g, None) == SHAPE
    for E, K, N in [(0, 128, 128), (257, 128, 128), (2, 100, 128), (2, 128, 0)]:
        assert lib.moe_quantize_weights_mxfp4(g, E, K, N, g, g, None) == SHAPE


def test_reference_block_by_hand():
    x = np.zeros((1, 128))
    # block 0: max 6.5 -> 2^(2 - 2) = 1: 6.5 and 7 saturate, ties go to the even code
    x[0, :12] = [6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.2, -0.3, 5.1, 0.74]
    # block 1: max 0.3 -> 2^(-2 - 2): 0.3 * 16 = 4.8 -> 4, 0.05 * 16 = 0.8 -> 1
    x[0, 32:34] = [0.3, 0.05]
    # block 3: an infinity
    x[0, 100] = np.inf
    codes, scales, values = ref.quantize(x)
    s = [scales[b % 4] for b in range(4)]
    assert s == [127, 123, 0, 255]
    assert values[0, :12].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.0, -0.5, 6.0, 0.5]
    assert values[0, 32:34].tolist() == [0.25, 0.0625]
    assert not values[0, 64:96].any() and np.isnan(values[0, 96:]).all()
    assert codes[0, :4].tolist() == [0x07, 0x22, 0x44, 0x66]
    assert ref.unpack(codes)[0, :4].tolist() == [7, 0, 2, 2]


def test_reference_scale_tiles():
    s = np.arange(256 * 8, dtype=np.int64).reshape(256, 8) % 251
    t = ref.tile(s.astype(np.uint8))
    # row 0 block 0; row 1; row 32; block 1; block 4 (next tile); row 128 (next row of tiles)
    for (r, b), at in {(0, 0): 0, (1, 0): 16, (32, 0): 4, (0, 1): 1, (0, 4): 512, (128, 0): 1024,
                       (255, 7): 1024 + 512 + 31 * 16 + 12 + 3}.items():
        assert t[at] == s[r, b]

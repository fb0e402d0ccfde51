"""CPU checks of the 8-bit integer calls' host side, and hand-worked codes of the
reference the GPU tests compare with."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    from combine_moe_route_04_gb300 import _build
    _build.build()
    import combine_moe_route_04_gb300 as m
    m.load()
    return m


GOOD = 1 << 20   # never dereferenced: validation fails first
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


def test_workspace(moe):
    for s in [(1, 128, 128, 1, 1), (2048, 4096, 1536, 64, 8), (1 << 22, 128, 128, 256, 16)]:
        mr = moe.capacity(s)[1]
        need = mr * (s[1] + s[2]) * 3 + mr * 8
        assert need <= moe.int8_workspace_size(s)
    with pytest.raises(moe.MoEError):
        moe.int8_workspace_size((4, 100, 128, 2, 1))
    assert moe.load().moe_int8_workspace_size(ctypes.byref(moe.shape(1, 128, 128, 1, 1)), None) == INVALID


def calls(moe):
    """(function, arguments with every pointer GOOD, indexes of the pointers)"""
    p = ctypes.byref(moe.shape(128, 256, 512, 8, 2))
    lib = moe.load()
    g = GOOD
    yield lib.moe_quantize_int8, [g, 4, 256, g, g, None], [0, 3, 4]
    yield lib.moe_quantize_weights_int8, [g, 2, 256, 128, g, g, None], [0, 4, 5]
    yield lib.moe_dequantize_int8, [g, g, 4, 256, g, None], [0, 1, 4]
    yield lib.moe_quantize_permute_int8, [p] + [g] * 5 + [None], range(1, 6)
    yield lib.moe_grouped_gemm_up_int8, [p] + [g] * 10 + [None], range(1, 11)
    yield lib.moe_grouped_gemm_down_int8, [p] + [g] * 8 + [None], range(1, 9)
    yield lib.moe_forward_int8, [p] + [g] * 10 + [None], range(1, 11)


def test_refusals(moe):
    for fn, args, ptrs in calls(moe):
        assert len(fn.argtypes) == len(args)
        for i in ptrs:
            for bad, code in ((None, INVALID), (GOOD + 8, MISALIGNED)):
                a = list(args)
                a[i] = bad
                assert fn(*a) == code, (fn.__name__, i)
        if not isinstance(args[0], int):
            assert fn(None, *args[1:]) == INVALID
            assert fn(ctypes.byref(moe.shape(128, 200, 512, 8, 2)), *args[1:]) == SHAPE
    lib, g = moe.load(), GOOD
    for rows, cols in [(0, 256), (-1, 256), (1 << 31, 128), (4, 130), (4, 64), (4, 1 << 16)]:
        assert lib.moe_quantize_int8(g, rows, cols, g, g, None) == SHAPE
        assert lib.moe_dequantize_int8(g, g, rows, cols, g, None) == SHAPE
    for E, K, N in [(0, 128, 128), (257, 128, 128), (2, 100, 128), (2, 128, 0)]:
        assert lib.moe_quantize_weights_int8(g, E, K, N, g, g, None) == SHAPE


def test_binding_checks_its_tensors(moe):
    torch = pytest.importorskip("torch")
    codes, scales = torch.zeros((4, 128), dtype=torch.int8), torch.zeros(4)
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_quantize_int8(x, 4, 128, codes, scales)
    with pytest.raises(TypeError):
        moe.moe_quantize_int8(x, 4, 128, None, scales)


def test_reference_codes_by_hand():
    torch = pytest.importorskip("torch")
    import int8_ref as ref
    x = torch.zeros((4, 128))
    # amax 254: the codes are x / 2, ties to even
    x[0, :9] = torch.tensor([254.0, 1.0, 3.0, 5.0, -1.0, -3.0, 2.0, -254.0, 127.0])
    x[1, :3] = torch.tensor([1.0, 0.5, -0.25])  # 127, 63.5 -> 64, -31.75 -> -32
    x[3, 5] = float("inf")
    q, s = ref.quantize(x)
    assert q[0, :9].tolist() == [127, 0, 2, 2, 0, -2, 1, -127, 64]
    assert q[1, :3].tolist() == [127, 64, -32]
    assert s[:3].tolist() == [2.0, float(torch.tensor(1 / 127)), 0.0]
    assert not q[2].any() and not q[3].any() and bool(s[3].isnan())

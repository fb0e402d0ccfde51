"""CPU checks of the training calls' host side: sizes and refusals."""
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


def test_backward_workspace(moe):
    for s in [(1, 128, 128, 1, 1), (2048, 4096, 1536, 64, 8), (1 << 22, 128, 128, 256, 16)]:
        mr = moe.capacity(s)[1]
        need = mr * s[1] * 2 + mr * s[2] * 4
        assert need + 256 <= moe.backward_workspace_size(s) <= need + 4096
    with pytest.raises(moe.MoEError):
        moe.backward_workspace_size((4, 100, 128, 2, 1))
    assert moe.load().moe_backward_workspace_size(ctypes.byref(moe.shape(1, 128, 128, 1, 1)), None) == INVALID


def calls(moe):
    """(function, number of pointers after the shape, the stream last)"""
    lib = moe.load()
    yield lib.moe_grouped_gemm_up_train, 9
    yield lib.moe_combine_backward, 8
    yield lib.moe_grouped_gemm_down_backward, 9
    yield lib.moe_grouped_gemm_up_backward, 8
    yield lib.moe_grouped_gemm_weight_backward, 11
    yield lib.moe_permute_backward, 4
    yield lib.moe_forward_train, 9
    yield lib.moe_backward, 13


def test_refusals(moe):
    good = ctypes.byref(moe.shape(128, 256, 512, 8, 2))
    for fn, n in calls(moe):
        assert len(fn.argtypes) == n + 2
        for i in range(n):
            for bad, code in ((None, INVALID), (GOOD + 8, MISALIGNED)):
                a = [GOOD] * n + [None]
                a[i] = bad
                assert fn(good, *a) == code, (fn.__name__, i)
        a = [GOOD] * n + [None]
        assert fn(None, *a) == INVALID
        for bad in [(0, 256, 512, 8, 2), (128, 200, 512, 8, 2), (128, 256, 500, 8, 2), (128, 256, 512, 8, 9)]:
            assert fn(ctypes.byref(moe.shape(*bad)), *a) == SHAPE, fn.__name__


def test_binding_checks_its_tensors(moe):
    """The binding refuses host tensors before the library is called."""
    torch = pytest.importorskip("torch")
    s = (4, 128, 128, 2, 1)
    bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    R = moe.capacity(s)[1]
    rows, w = torch.zeros((R, 128), dtype=bf), torch.zeros((2, 128, 128), dtype=bf)
    counts, off, idx = torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros((4, 1), dtype=i32)
    x, ws = torch.zeros((4, 128), dtype=bf), torch.zeros(1 << 20, dtype=u8)
    lg = torch.zeros((4, 2), dtype=f32)
    for fn, args in [(moe.moe_grouped_gemm_up_train, (rows, counts, off, w, w, rows, rows, rows, ws)),
                     (moe.moe_combine_backward, (rows, idx, idx, lg, x, rows, lg, ws)),
                     (moe.moe_grouped_gemm_down_backward, (rows, counts, off, w, rows, rows, rows, rows, ws)),
                     (moe.moe_grouped_gemm_up_backward, (rows, rows, counts, off, w, w, rows, ws)),
                     (moe.moe_grouped_gemm_weight_backward, (rows, rows, rows, rows, rows, counts, off, w, w, w, ws)),
                     (moe.moe_permute_backward, (rows, idx, x, ws)),
                     (moe.moe_forward_train, (lg, x, w, w, w, rows, rows, x, ws)),
                     (moe.moe_backward, (w, w, w, rows, rows, x, x, w, w, w, lg, ws, ws))]:
        with pytest.raises(ValueError, match="CUDA"):
            fn(s, *args)
        with pytest.raises(TypeError):
            fn(s, None, *args[1:])

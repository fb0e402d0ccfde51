"""workspace_views belongs to moe_forward's workspace: a buffer too small to be one
(an MXFP4 or balance workspace) is refused instead of giving pointers past its end."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    from combine_moe_route_04_gb300 import _build
    _build.build()
    import combine_moe_route_04_gb300 as m
    m.load()
    return m


SHAPES = [(1, 128, 128, 1, 1), (64, 256, 512, 8, 2), (300, 1408, 640, 37, 3), (128, 128, 2048, 4, 1)]


@pytest.mark.parametrize("s", SHAPES)
def test_other_workspaces_are_refused(moe, s):
    for size in (moe.mxfp4_workspace_size(s), 256, moe.workspace_size(s) - 1):
        assert size < moe.workspace_size(s)
        with pytest.raises(ValueError):
            moe.workspace_views(s, torch.empty(size, dtype=torch.uint8))


@pytest.mark.parametrize("s", SHAPES)
def test_a_forwards_workspace_is_taken(moe, s):
    n = moe.workspace_size(s)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty((n + 3) // 4, dtype=torch.int32)):
        base = (ws.data_ptr() + 15) // 16 * 16
        if base != ws.data_ptr():
            continue
        v = moe.workspace_views(s, ws)
        mr = moe.capacity(s)[1]
        assert base < v.topk_ids < base + n
        assert v.Y + 2 * mr * s[1] <= base + n and v.h + 2 * mr * s[2] <= base + n and v.Xp + 2 * mr * s[1] <= base + n
    assert moe.workspace_views(s, 1 << 20).topk_ids > 1 << 20      # an address is taken as it is

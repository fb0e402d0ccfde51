"""The balance loss, its counts and its gradient against float64."""
import numpy as np
import pytest

from gpu_util import need_gpu, to_dev

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def top_k(logits, k):
    return np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)


def ref64(logits, ids, mask, g):
    """Definition in float64: counts, n, mean_probs, losses, dlogits, and the
    gradient's magnitude before cancellation (for the tolerance)."""
    T, E = logits.shape
    k = ids.shape[1]
    x = logits.astype(np.float64)
    use = ~np.all(np.isneginf(x), axis=1)
    if mask is not None:
        use &= mask != 0
    n = int(use.sum())
    counts = np.bincount(ids[use].ravel(), minlength=E)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if n == 0:
        return counts, 0, np.zeros(E), np.zeros(2), d, mag
    with np.errstate(over="ignore", invalid="ignore"):
        top = x[use].max(1, keepdims=True)
        ex = np.exp(x[use] - top)
        p = ex / ex.sum(1, keepdims=True)
        lse = top[:, 0] + np.log(ex.sum(1))
        f = counts / (n * k)
        P = p.mean(0)
        losses = np.array([E * (f * P).sum(), (lse ** 2).mean()])
        fp = (p * f).sum(1, keepdims=True)
        d[use] = p * (g[0] * E / n * (f - fp) + g[1] * 2 / n * lse[:, None])
        c = np.abs(f - 1.0 / E)
        mag[use] = p * (abs(g[0]) * E / n * (c + (p * c).sum(1, keepdims=True))
                        + abs(g[1]) * 2 / n * np.abs(lse[:, None]))
    return counts, n, P, losses, d, mag


def run(logits, ids, mask, g, calls=1):
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    T, E = logits.shape
    s = (T, 128, 128, E, ids.shape[1])
    L, I = to_dev(logits.astype(np.float32)), to_dev(ids)
    M = None if mask is None else to_dev(mask)
    counts = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    n = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    P = torch.full((E,), -5.0, device="cuda")
    losses = torch.full((2,), -5.0, device="cuda")
    d = torch.full((T, E), -5.0, device="cuda")
    ws = moe.alloc_balance_workspace(s)
    out = []
    for _ in range(calls):
        moe.moe_balance_loss(s, L, I, M, counts, n, P, losses, ws)
        moe.moe_balance_loss_backward(s, L, M, counts, n, to_dev(np.asarray(g, np.float32)), d)
        assert moe.last_device_status(ws) == 0
        out.append([t.cpu().numpy().copy() for t in (counts, n, P, losses, d)])
    for o in out[1:]:
        for a, b in zip(out[0], o):
            assert a.tobytes() == b.tobytes()      # the same bits every time
    return out[0]


def check(logits, ids, mask, g=(1e-2, 1e-3)):
    counts, n, P, losses, d = run(logits, ids, mask, g, calls=2)
    wc, wn, wP, wl, wd, mag = ref64(logits.astype(np.float32), ids, mask, np.float32(g).astype(np.float64))
    assert np.array_equal(counts, wc) and n[0] == wn
    # A probability carries the error of exp's argument (its rounding grows with
    # the distance from the row's maximum), of exp itself and of the row's sum:
    # (|x| + 12) 2^-23 and E roundings of a sum, at most; sums over tokens add
    # about as many roundings again.
    x = logits[np.isfinite(logits)]
    spread = float(x.max() - x.min()) if x.size else 0.0
    rel = (spread + 12 + logits.shape[1] ** 0.5) * 2 * EPS * 2
    tok = (logits.shape[0] ** 0.5 + 32) * EPS
    assert np.all(np.abs(P - wP) <= (rel + tok) * np.abs(wP) + 1e-30)
    assert np.all(np.abs(losses - wl) <= 2 * (rel + tok) * np.abs(wl) + 1e-12)
    assert np.all(np.abs(d - wd) <= 4 * rel * mag + 1e-30)
    return d


CASES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (31, 8, 2), (128, 8, 2), (97, 37, 3), (513, 64, 8), (1000, 128, 8),
         (333, 256, 16),
         (77, 255, 16), (2050, 100, 4), (4099, 3, 1), (6000, 16, 1), (9001, 66, 7)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", CASES)
def test_against_64_bits(T, E, k, masked):
    rng = np.random.default_rng(T * 1000 + E)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    mask = (rng.random(T) < 0.7).astype(np.uint8) * rng.integers(1, 256, T).astype(np.uint8) if masked else None
    check(logits, top_k(logits, k), mask)


def test_nothing_takes_part():
    logits = np.ones((10, 12), np.float32)
    ids = top_k(logits, 2)
    for m in (np.zeros(10, np.uint8), None):
        x = logits if m is not None else np.full((10, 12), -np.inf, np.float32)
        counts, n, P, losses, d = run(x, ids, m, (1.0, 1.0))
        assert n[0] == 0 and not counts.any() and not P.any() and not losses.any() and not d.any()


def test_masked_tokens_may_hold_anything():
    rng = np.random.default_rng(8)
    logits = rng.standard_normal((200, 20)).astype(np.float32)
    mask = (np.arange(200) % 3 != 0).astype(np.uint8)
    ids = top_k(logits, 4)
    want = run(logits, ids, mask, (1.0, 1.0))
    logits[mask == 0] = rng.choice([np.nan, np.inf, -np.inf, 3e38], (int((mask == 0).sum()), 20))
    ids[mask == 0] = 1 << 30                       # not looked at either
    got = run(logits, ids, mask, (1.0, 1.0))
    for a, b in zip(want, got):
        assert a.tobytes() == b.tobytes()


def test_experts_at_minus_infinity_and_lowest_values():
    rng = np.random.default_rng(9)
    logits = rng.standard_normal((300, 24)).astype(np.float32)
    logits[:, 5:9] = -np.inf
    logits[10] = -np.inf                            # takes no part
    logits[11, 1:] = -np.inf                        # one expert left
    logits[12, :12] = np.finfo(np.float32).min      # lowest value: probability 0
    d = check(np.where(np.isneginf(logits), -np.inf, logits), top_k(np.nan_to_num(logits, neginf=-1e38), 3), None)
    assert not d[10].any() and not d[:, 5:9].any()


def test_a_nan_that_takes_part_shows():
    logits = np.zeros((40, 6), np.float32)
    logits[7, 2] = np.nan
    counts, n, P, losses, d = run(logits, top_k(np.zeros((40, 6)), 2), None, (1.0, 1.0))
    assert n[0] == 40 and np.isnan(losses).all() and np.isnan(d[7]).all()
    assert np.isfinite(np.delete(d, 7, 0)).all()    # the counts, so the other rows' gradients, are unharmed


def test_gradient_against_differences():
    """Central differences of the float64 loss, counts held constant."""
    rng = np.random.default_rng(3)
    T, E, k, g = 12, 9, 2, (0.7, 0.3)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = top_k(logits, k)
    mask = np.ones(T, np.uint8)
    mask[4] = 0
    d = run(logits, ids, mask, g)[4]
    x = logits.astype(np.float64)

    def loss(y):
        _, _, _, l, _, _ = ref64(y, ids, mask, g)
        return g[0] * l[0] + g[1] * l[1]

    h = 1e-5
    for t in range(T):
        for e in range(E):
            y = x.copy()
            y[t, e] += h
            a = loss(y)
            y[t, e] -= 2 * h
            assert abs(d[t, e] - (a - loss(y)) / (2 * h)) <= 2e-7


def test_expert_ids_out_of_range_are_reported():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (40, 128, 128, 6, 2)
    ids = torch.zeros((40, 2), dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    ids[3, 0], ids[9, 1] = 6, -1
    counts, n = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, losses = torch.zeros(6, device="cuda"), torch.zeros(2, device="cuda")
    ws = moe.alloc_balance_workspace(s)
    moe.moe_balance_loss(s, torch.zeros((40, 6), device="cuda"), ids, None, counts, n, P, losses, ws)
    assert moe.last_device_status(ws) == 7
    assert counts.tolist() == [39, 39, 0, 0, 0, 0]


def test_after_the_layers_routing_on_a_stream_and_in_a_graph():
    """moe_route's picks feed the loss; its counts are the routing's."""
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = T, _, _, E, k = (3000, 128, 128, 64, 8)
    logits = torch.randn((T, E), device="cuda")
    bufs = moe.alloc_route_outputs(s)
    ws, bws = moe.alloc_workspace(s), moe.alloc_balance_workspace(s)
    counts, n = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    P, losses, d = torch.zeros(E, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros((T, E), device="cuda")
    g = torch.tensor([1.0, 0.1], device="cuda")
    torch.cuda.synchronize()

    def calls(stream=None):
        moe.moe_route(s, logits, bufs["topk_ids"], bufs["topk_w"], bufs["counts"], bufs["off_pad"],
                      bufs["block_expert"], bufs["num_blocks"], bufs["gather_idx"], bufs["scatter_idx"], ws, stream)
        moe.moe_balance_loss(s, logits, bufs["topk_ids"], None, counts, n, P, losses, bws, stream)
        moe.moe_balance_loss_backward(s, logits, None, counts, n, g, d, stream)

    side = torch.cuda.Stream()
    calls(side)
    assert moe.last_device_status(ws, side) == 0 and moe.last_device_status(bws, side) == 0
    assert torch.equal(counts, bufs["counts"]) and n.item() == T
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    logits.copy_(torch.randn((T, E), device="cuda") - torch.arange(E, device="cuda") * 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(counts, bufs["counts"])
    wc, wn, wP, wl, wd, mag = ref64(logits.cpu().numpy(), bufs["topk_ids"].cpu().numpy(), None,
                                    np.float32([1.0, 0.1]).astype(np.float64))
    assert np.array_equal(counts.cpu().numpy(), wc)
    assert np.all(np.abs(losses.cpu().numpy() - wl) <= 1e-5 * wl)


def test_refusals():
    torch = need_gpu()
    import combine_moe_route_04_gb300 as moe
    s = (8, 128, 128, 4, 2)
    f = lambda *n: torch.zeros(n, device="cuda")  # noqa: E731
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = moe.alloc_balance_workspace(s)
    good = dict(s=s, logits=f(8, 4), topk_ids=i(8, 2), mask=None, counts=i(4), num_tokens=i(1), mean_probs=f(4),
                losses=f(2), ws=ws)
    moe.moe_balance_loss(**good)
    for name, bad, err in (("logits", f(8, 3), ValueError), ("logits", f(8, 4).double(), TypeError),
                           ("logits", f(4, 8).t(), ValueError), ("topk_ids", i(8, 1), ValueError),
                           ("mask", f(8), TypeError),
                           ("mask", torch.ones(7, dtype=torch.bool, device="cuda"), ValueError),
                           ("ws", ws[:-1], ValueError), ("losses", torch.zeros(2), ValueError)):
        with pytest.raises(err):
            moe.moe_balance_loss(**{**good, name: bad})
    with pytest.raises(moe.MoEError):
        moe.moe_balance_loss(**{**good, "s": (8, 128, 128, 300, 2)})
    with pytest.raises(ValueError):
        moe.moe_balance_loss_backward(s, f(8, 4), None, i(4), i(1), f(1), f(8, 4))

"""The balance loss and its gradient against float64 on rows with absent experts,
one expert left, float32's lowest value and logits far apart, with bounds that
follow each row's own spread."""
import numpy as np
import pytest

from test_gpu_balance import EPS, ref64, run, top_k

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


def bounds(logits, mask=None):
    """(relative error of a probability per row [T, 1], of a sum over tokens).

    exp's argument is off by about its own size times 2^-23 (the difference and
    its product by log2 e are rounded), the exponential, the reciprocal and the
    row's sum by some ulps: (|x| + 12 + sqrt E) 2^-22 as for the other cases, |x|
    at most 104: what lies further below the row's maximum underflows to 0, and
    its true probability is below 1e-45."""
    x = logits.astype(np.float64)
    top = np.where(np.isneginf(x).all(1), 0.0, x.max(1))[:, None]
    depth = np.where(x >= top - 104.0, top - x, 0.0).max(1, keepdims=True)
    rel = (depth + 12 + x.shape[1] ** 0.5) * 4 * EPS
    return rel, float(rel.max()) + (x.shape[0] ** 0.5 + 32) * EPS


def check(logits, ids, mask=None, g=(1e-2, 1e-3)):
    logits = logits.astype(np.float32)
    counts, n, P, losses, d = run(logits, ids, mask, g, calls=2)
    wc, wn, wP, wl, wd, mag = ref64(logits, ids, mask, np.float32(g).astype(np.float64))
    assert np.array_equal(counts, wc) and n[0] == wn and wn > 0
    rel, tot = bounds(logits)
    assert rel.max() < 1e-4 and tot < 1e-4       # the bounds mean something
    assert np.all(np.abs(P - wP) <= tot * wP + 1e-30)
    assert np.all(np.abs(losses - wl) <= 2 * tot * wl + 1e-12)
    assert np.all(np.abs(d - wd) <= 4 * rel * mag + 1e-30)
    return P, losses, d


def base(T, E, seed, scale=1.0):
    return (np.random.default_rng(seed).standard_normal((T, E)) * scale).astype(np.float32)


def ids_of(logits, k):
    return top_k(np.nan_to_num(logits, neginf=-3.4e38), k)


@pytest.mark.parametrize("E,k", [(7, 2), (24, 3), (37, 3), (64, 4), (129, 4), (255, 5), (256, 8)])
def test_absent_experts_lone_experts_and_lowest_values(E, k):
    logits = base(300, E, E)
    logits[:, 3:5] = -np.inf                         # two experts absent everywhere
    logits[10] = -np.inf                             # takes no part
    logits[11, 1:] = -np.inf                         # one expert left
    logits[12, : E // 2] = LOWEST                    # probability 0 beside ordinary logits
    logits[13, 1:] = LOWEST
    logits[14, E - 1] = -np.inf
    logits[15, :-1] = -np.inf                        # the last expert alone
    P, losses, d = check(logits, ids_of(logits, k))
    assert not d[10].any() and not d[:, 3:5].any() and not P[3:5].any()
    assert not d[12, : E // 2].any() and not d[13, 1:].any()


@pytest.mark.parametrize("E,k", [(8, 2), (37, 3), (256, 8)])
def test_logits_far_from_zero_and_from_each_other(E, k):
    """Row maxima from -60 to 60 (the z loss is then large in every row), and rows
    whose logits fall by up to 104 below their maximum."""
    rng = np.random.default_rng(E)
    logits = base(400, E, E + 1) + rng.uniform(-60, 60, (400, 1)).astype(np.float32)
    far = rng.random(400) < 0.5
    logits[far] -= rng.uniform(0, 100, (int(far.sum()), E)).astype(np.float32)
    check(logits, ids_of(logits, k))


@pytest.mark.parametrize("E,k", [(5, 2), (24, 3), (200, 4)])
def test_masked_beside_absent_experts(E, k):
    logits = base(500, E, E + 2)
    logits[::7, E // 2] = -np.inf
    logits[3::11, 1:] = LOWEST
    mask = (np.random.default_rng(E).random(500) < 0.6).astype(np.uint8)
    logits[mask == 0] = -np.inf                      # what a padded batch may hold
    ids = ids_of(logits, k)
    P, losses, d = check(logits, ids, mask)
    assert not d[mask == 0].any()


def test_every_logit_at_the_lowest_value():
    """A token whose logits are all float32's lowest takes part: its probabilities
    are equal, its log-sum-exp is that value, whose square is past float32."""
    E, k, g = 12, 2, np.float32([1e-2, 1e-3])
    logits = base(64, E, 5)
    logits[20] = LOWEST
    ids = ids_of(logits, k)
    counts, n, P, losses, d = run(logits, ids, None, g)
    wc, wn, wP, wl, wd, mag = ref64(logits, ids, None, g.astype(np.float64))
    rel, tot = bounds(logits)
    assert n[0] == 64 and np.array_equal(counts, wc)
    assert np.all(np.abs(P - wP) <= tot * wP)
    assert abs(losses[0] - wl[0]) <= 2 * tot * wl[0] and np.isposinf(losses[1])
    assert np.all(np.abs(d - wd) <= 4 * rel * mag + 1e-30)


@pytest.mark.parametrize("g", [(1.0, 0.0), (0.0, 1.0)])
def test_a_gradient_of_one_loss_alone(g):
    logits = base(50, 10, 6)
    check(logits, ids_of(logits, 2), None, g)

"""The 64-bit oracle of the block's operators: its gradients against differences
of its own forward formulas, its choices against a search over all sets."""
import itertools

import numpy as np
import pytest

from oracle import block as oracle


def difference(f, x, h=1e-6):
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        out[i] = (f(up) - f(down)) / (2 * h)
    return out


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient(sigmoid, renormalize):
    rng = np.random.default_rng(0)
    l, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 3))
    ids, _ = oracle.route_scored(l, 3, renormalize, sigmoid, scale=2.5)

    def loss(x):
        total = 0.0
        for t in range(3):
            s = oracle.scores(x[t], sigmoid)[ids[t]]
            total += (2.5 * (s / s.sum() if renormalize else s) * g[t]).sum()
        return total

    got = oracle.route_scored_backward(l, ids, g, renormalize, sigmoid, 2.5)
    assert np.allclose(got, difference(loss, l), atol=1e-8)


def test_route_choice_over_all_sets():
    """The groups and experts kept are the best of all ways to keep as many."""
    rng = np.random.default_rng(1)
    for _ in range(50):
        l, b = rng.standard_normal(12), 0.3 * rng.standard_normal(12)
        c = oracle.scores(l, True) + b
        got = oracle.choose(l, True, b, 4, 2, 2, 3)
        two = lambda g: np.sort(c[3 * g:3 * g + 3])[-2:].sum()
        pairs = itertools.combinations(range(4), 2)
        best = max(pairs, key=lambda p: two(p[0]) + two(p[1]))
        allowed = [3 * g + i for g in best for i in range(3)]
        sets = itertools.combinations(allowed, 3)
        assert set(got) == set(max(sets, key=lambda s: c[list(s)].sum()))
        assert list(c[got]) == sorted(c[got], reverse=True)


def test_route_ties_bars_and_nans():
    zero = np.zeros(6)
    assert oracle.choose(zero, True, None, 1, 1, 1, 3) == [0, 1, 2]
    assert oracle.choose(zero, True, zero, 3, 2, 2, 3) == [0, 1, 2]
    barred = np.array([0, -np.inf, 0, -np.inf, -np.inf, -np.inf])
    assert oracle.choose(barred, True, zero, 3, 2, 2, 3) == [0, 2]
    assert oracle.choose(np.full(6, -np.inf), False, None, 1, 1, 1, 2) == []
    assert oracle.choose(np.array([1.0, np.nan, 3.0]), True, np.zeros(3), 1, 1, 1, 2) == [1, 2]


@pytest.mark.parametrize("post, gates, pre, residual", [
    (True, 1, True, True), (True, 2, False, True), (False, 4, True, True), (False, 0, True, False),
    (True, 0, True, False)])
def test_norm_gradient(post, gates, pre, residual):
    rng = np.random.default_rng(2)
    T, H = 4, 5
    p = dict(x=rng.standard_normal((T, H)), residual=rng.standard_normal((T, H)),
             post=rng.standard_normal(H), gate=rng.standard_normal((gates, H)),
             pre=rng.standard_normal(H))
    for name, there in (("post", post), ("gate", gates), ("pre", pre), ("residual", residual)):
        if not there:
            p[name] = None
    dsum = rng.standard_normal((T, H))
    dy = rng.standard_normal((T, H)) if pre else None

    def loss(**changed):
        q = {**p, **changed}
        f = oracle.norm(q["x"], q["residual"], q["post"], q["gate"], 0.7, q["pre"], 1e-3)
        return (f["sum"] * dsum).sum() + (0 if dy is None else (f["y"] * dy).sum())

    got = oracle.norm_backward(p["x"], p["residual"], p["post"], p["gate"], 0.7, p["pre"], 1e-3,
                               dsum, dy)
    names = dict(x="x", residual="residual", post="post_gain", gate="gate", pre="pre_gain")
    for mine, theirs in names.items():
        if p[mine] is not None:
            assert np.allclose(got[theirs], difference(lambda v: loss(**{mine: v}), p[mine]),
                               atol=1e-6), mine


@pytest.mark.parametrize("kind", ["silu", "relu", "none"])
def test_act_gradient(kind):
    g = np.array([-30.0, -1.3, -0.4, 0.2, 5.0, 40.0])
    got = difference(lambda v: oracle.act(v, kind).sum(), g)
    assert np.allclose(oracle.act_slope(g, kind), got, atol=1e-8)


def test_checkpoint():
    v = np.array([[1.0, -0.5, 127.4 / 64, 0.0] + [0.0] * 28 + [3e-45, np.inf]])
    codes, scales, values = oracle.checkpoint(v)
    assert list(codes[0, :3]) == [64, -32, 127] and scales[0, 0] == 121
    assert scales[0, 1] == 255 and np.isnan(values[0, 32:]).all()
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 64)) * 10.0 ** rng.integers(-30, 30, (20, 1))
    _, scales, values = oracle.checkpoint(x)
    step = 2.0 ** (np.repeat(scales, 32, 1) - 127)
    assert (np.abs(values - x) <= step * np.where(np.abs(x) > 127.5 * step, 1, 0.5)).all()


def test_combine_gradient():
    rng = np.random.default_rng(4)
    rows, w, dy = rng.standard_normal((6, 3)), rng.standard_normal((3, 2)), rng.standard_normal((3, 3))
    token_row = np.array([[0, 3], [-1, 1], [5, -1]])
    drows, dw = oracle.combine_backward(dy, rows, token_row, w)
    assert np.allclose(drows, difference(lambda v: (oracle.combine(v, token_row, w) * dy).sum(), rows))
    assert np.allclose(dw, difference(lambda v: (oracle.combine(rows, token_row, v) * dy).sum(), w))

"""The oracle of the expert layer's operators against known values."""
import numpy as np
import pytest

from oracle import moe


def test_block_of_known_values():
    x = np.zeros((1, 32))
    x[0, :10] = [6, -4, 3, 2, 1.5, 1, 0.5, 0.25, 0.26, -0.1]   # the largest, 6: scale 1
    c, s = moe.mx_quantize(x)
    assert s[0, 0] == 127
    assert c[0, :10].tolist() == [7, 14, 5, 4, 3, 2, 1, 0, 1, 8]
    assert np.array_equal(moe.mx_values(c, s)[0, :7], x[0, :7])


@pytest.mark.parametrize("value, code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4),
                                         (3.5, 6), (5.0, 6), (7.9, 7)])
def test_ties_go_to_the_even_code(value, code):
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 4.0, value        # scale 1 either way
    c, s = moe.mx_quantize(x)
    assert s[0, 0] == 127 and c[0, 1] == code


def test_scale_range():
    x = np.zeros((5, 32))
    x[1, 3] = 2.0 ** -149
    x[2, 3] = np.float64(np.finfo(np.float32).max)
    x[3, 3] = np.inf
    x[4, 3] = np.nan
    _, s = moe.mx_quantize(x)
    assert s[:, 0].tolist() == [0, 0, 252, 255, 255]


def test_pack_places_scales():
    c = np.zeros((130, 256), dtype=np.uint8)
    s = np.zeros((130, 8), dtype=np.uint8)
    s[33, 5] = 9
    s[129, 0] = 7
    _, b = moe.mx_pack(c, s)
    assert b.nonzero()[0].tolist() == [512 + 1 * 16 + 1 * 4 + 1, 2 * 512 + 1 * 16]


def test_route_ties_masks_and_tables():
    inf = np.inf
    l = np.array([[1.0, 1, 1, 0], [-inf, 2, -inf, -inf], [-inf] * 4, [0, np.nan, 0, 0]])
    r = moe.route(l, 2, True)
    assert r["ids"].tolist() == [[0, 1], [1, -1], [-1, -1], [1, 0]]
    assert r["weights"][:3].tolist() == [[0.5, 0.5], [1, 0], [0, 0]]
    assert np.isnan(r["weights"][3]).all()
    assert r["expert_first"].tolist() == [0, 128, 256, 256]
    assert r["expert_rows"].tolist() == [2, 3, 0, 0]
    assert r["row_token"][128:131].tolist() == [0, 1, 3]
    capped = moe.route(l, 2, True, capacity=2)
    assert capped["expert_rows"].tolist() == [2, 2, 0, 0]
    assert capped["token_row"].tolist() == [[0, 2], [3, -1], [-1, -1], [-1, 1]]


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_is_the_derivative(renormalize):
    rng = np.random.default_rng(3)
    l, g = rng.standard_normal((6, 9)), rng.standard_normal((6, 3))
    ids = moe.route(l, 3, renormalize)["ids"]
    d = moe.route_backward(l, ids, g, renormalize)
    f = lambda x: (g * moe.route_weights(x, ids, renormalize)).sum()
    for t in range(6):
        for e in range(9):
            h = np.zeros_like(l)
            h[t, e] = 1e-5
            # central difference: error about h^2 = 1e-10 and 1e-16 / h = 1e-11
            assert abs((f(l + h) - f(l - h)) / 2e-5 - d[t, e]) < 1e-8

"""The balanced router on the GPU against the 64-bit oracle.

Choices and tables are exact.  Weights: expf is within 2 ulp (4 e, e = 2^-24), a
sigmoid has two roundings more, softmax's sum up to 37 + 32 of them, the share
and the scale three: 96 e relative.  (Where the oracle scales small sigmoids, so
does the kernel.)  Gradients: 96 e of the weights' and dot's magnitudes, and one
rounding to the logits' type.
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo
from oracle import block as oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import moe

BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(logits, top_k, renormalize=True, scoring="sigmoid", bias=None, groups=1, top_groups=1,
          group_top=1, scale=1.0, capacity=0, dweights=None):
    r = moe.route(logits, top_k, renormalize, capacity, scoring, bias, groups, top_groups,
                  group_top, scale)
    l64, sigmoid = host(logits), scoring == "sigmoid"
    scale = float(np.float32(scale))
    ids, w = oracle.route_scored(l64, top_k, renormalize, sigmoid, host(bias), groups, top_groups,
                                 group_top, scale)
    got = r.ids.cpu().numpy()
    assert np.array_equal(got, ids), (np.argwhere((got != ids).any(1))[:4], got[(got != ids).any(1)][:4],
                                      ids[(got != ids).any(1)][:4])
    off = np.abs(host(r.weights) - w)
    assert (off <= 96 * E * np.abs(w) + 2.0 ** -120).all(), (off / np.abs(w)).max() / E
    check_tables(r, ids, logits.shape[1], capacity)
    if dweights is not None:
        d = moe.route_backward(logits, r.ids, r.weights, dweights, renormalize, scoring, scale)
        assert d.dtype == logits.dtype
        want = oracle.route_scored_backward(l64, ids, host(dweights), renormalize, sigmoid, scale)
        mag = (np.abs(w) * np.abs(host(dweights))).sum(1, keepdims=True) * (1 + 1 / scale)
        bound = 96 * E * (mag + np.abs(want)) + torch.finfo(logits.dtype).eps / 2 * np.abs(want)
        assert (np.abs(host(d) - want) <= bound * (1 + 2.0 ** -8) + 2.0 ** -120).all()
    assert moe.device_status() == fo.FO_OK
    return r


def check_tables(r, ids, experts, capacity):
    """The row tables as a stable counting sort of the pairs."""
    T, k = ids.shape
    M = r.row_token.numel()
    row_token, row_slot = np.full(M, -1), np.zeros(M, dtype=int)
    token_row, first, rows, at = np.full((T, k), -1), [], [], 0
    for e in range(experts):
        pairs = np.argwhere(ids == e)
        if capacity:
            at, pairs = e * capacity, pairs[:capacity]
        for i, (t, s) in enumerate(pairs):
            row_token[at + i], row_slot[at + i], token_row[t, s] = t, s, at + i
        first.append(at)
        rows.append(len(pairs))
        at += -(-len(pairs) // 128) * 128
    for got, want in ((r.row_token, row_token), (r.row_slot, row_slot), (r.token_row, token_row),
                      (r.expert_first, first), (r.expert_rows, rows)):
        assert np.array_equal(got.cpu().numpy(), want)


def normal(rng, shape, dtype=F32, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).cuda()


SHAPES = [  # tokens, experts, top_k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 128, 8, 8, 4, 2), (5, 8, 2, 1, 1, 1), (17, 60, 6, 6, 3, 1),
    (33, 60, 6, 6, 3, 2), (40, 256, 8, 8, 4, 2), (3, 7, 7, 7, 7, 2), (20, 96, 32, 3, 2, 2),
    (9, 1024, 32, 32, 16, 2), (50, 160, 6, 8, 3, 1), (64, 72, 8, 4, 1, 2), (7, 33, 5, 11, 4, 2),
    (2, 512, 10, 16, 2, 1), (200, 32, 4, 32, 7, 2), (31, 65, 3, 5, 2, 2), (6, 64, 32, 2, 2, 2),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_route(shape, dtype):
    T, n, k, groups, top_groups, group_top = shape
    rng = np.random.default_rng(T * n)
    for scoring, spread in (("sigmoid", 0.05), ("softmax", 0.5 / n)):
        for biased in (False, True):
            for renormalize in (False, True):
                check(normal(rng, (T, n), dtype, 1.5), k, renormalize, scoring,
                      normal(rng, (n,), F32, spread) if biased else None, groups, top_groups,
                      group_top, 2.5 if biased else 1.0, 0,
                      normal(rng, (T, k)) if k > 1 or not renormalize else None)


@pytest.mark.parametrize("T, n, k, groups, capacity", [(3000, 60, 6, 6, 256), (5000, 16, 2, 4, 0),
                                                       (2049, 128, 8, 8, 128), (700, 300, 4, 1, 0)])
def test_many_tokens(T, n, k, groups, capacity):
    rng = np.random.default_rng(T)
    check(normal(rng, (T, n)), k, True, "sigmoid", normal(rng, (n,), F32, 0.05), groups,
          max(1, groups // 2), 2, 1.0, capacity, normal(rng, (T, k)))


@pytest.mark.parametrize("n, k, groups", [(64, 8, 1), (64, 8, 4), (250, 6, 5), (40, 32, 1), (32, 31, 2)])
def test_choices_that_fp32_cannot_tell(n, k, groups):
    """A bias that undoes the scores' differences but for fp32's last places: all
    of a token's choice values lie within 2^-24 of each other."""
    rng = np.random.default_rng(n)
    l = normal(rng, (1, n))
    bias = torch.from_numpy(1 - oracle.scores(host(l)[0], True)).to(F32).cuda()
    others = normal(rng, (3, n))
    logits = torch.cat((l, others, l + 2.0 ** -20, l))
    top_groups = -(-k * groups // n) if k * groups > n else max(1, groups // 2)
    for group_top in (1, 2):
        check(logits, k, True, "sigmoid", bias, groups, top_groups, group_top)
    # softmax, the same
    bias = torch.from_numpy(1 - oracle.scores(host(l)[0], False)).to(F32).cuda()
    check(logits, k, True, "softmax", bias, groups, top_groups, 2)


@pytest.mark.parametrize("top_groups", [1, 3, 4])
def test_pairs_that_fp32_cannot_tell(top_groups):
    """Few near ties in each token, at every rank and at the groups' border."""
    rng = np.random.default_rng(top_groups)
    T, n, groups = 400, 64, 4
    l = host(normal(rng, (T, n), F32, 1.5))
    l32 = l.astype(np.float32).astype(np.float64)
    bias = np.float32(0.05 * rng.standard_normal(n)).astype(np.float64)
    for t in range(T):
        a, b = rng.choice(n, 2, replace=False)
        c = oracle.scores(l32[t], True)[a] + bias[a] - bias[b]
        if 0.01 < c < 0.99:     # the logit that makes b's choice a's, to fp32
            l32[t, b] = np.float32(np.log(c / (1 - c)))
    check(torch.from_numpy(l32).to(F32).cuda(), 8, True, "sigmoid",
          torch.from_numpy(bias).to(F32).cuda(), groups, top_groups, 2)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1000.0, 30000.0])
@pytest.mark.parametrize("n, groups", [(256, 8), (64, 4), (60, 6), (1024, 32)])
def test_groups_of_choices_of_unlike_signs(n, groups, size, scoring):
    """Two groups of pairs that cancel but for their scores, which differ by a few of the
    steps of fp32 that the pair's own size has."""
    rng = np.random.default_rng(n)
    T, per, step = 300, n // groups, float(np.spacing(np.float32(size)))
    bias = np.full(n, -size)
    bias[::per] = size
    l = np.float32(rng.standard_normal((T, n)) - 6.0)
    for t in range(T):
        g, h = rng.choice(groups, 2, replace=False) * per
        if scoring == "sigmoid":
            p = rng.uniform(0.3, 0.7, 3)
            q = np.clip(p[0] + p[1] - p[2] + step * rng.uniform(-4, 4), 0.05, 0.95)
            x, i = np.log((*p, q)) - np.log1p(-np.array((*p, q))), (g, g + 1, h, h + 1)
        else:
            x = rng.uniform(0.0, 1.0, 3)
            q = max(np.exp(x[0]) + np.exp(x[1]) - np.exp(x[2]) + step * rng.uniform(-8, 8), 0.1)
            x, i = (*x, np.log(q)), (g, g + 1, h, h + 1)
        l[t, list(i)] = np.float32(x)
    check(torch.from_numpy(l).cuda(), min(4, per), True, scoring,
          torch.from_numpy(np.float32(bias)).cuda(), groups, 1, 2)


@pytest.mark.parametrize("offset", [100.0, -1000.0])
@pytest.mark.parametrize("n, groups", [(256, 8), (64, 4)])
def test_groups_of_logits_far_from_zero(n, groups, offset):
    """Two groups whose pairs differ by few steps of fp32, each of them a large part of
    a score: softmax looks at differences, not at sizes."""
    rng = np.random.default_rng(n)
    T, per, step = 600, n // groups, np.spacing(np.float32(abs(offset)))
    l = np.float32(offset - 8.0 + rng.standard_normal((T, n)))
    for t in range(T):
        for g in rng.choice(groups, 2, replace=False):
            for e in rng.choice(per, 2, replace=False):
                l[t, g * per + e] = np.float32(offset) + np.float32(step * rng.integers(0, 17))
    check(torch.from_numpy(l).cuda(), 4, True, "softmax", None, groups, 1, 2)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups, top_groups", [(1, 1), (4, 2), (4, 4)])
def test_ties(scoring, groups, top_groups):
    """All alike, few distinct logits, with and without a bias of zeros or of a
    few values: ties to the lowest index."""
    rng = np.random.default_rng(groups)
    n, k = 48, 6
    few = torch.from_numpy(rng.integers(-1, 2, (200, n)).astype(np.float32)).cuda()
    for logits in (torch.zeros((200, n), device="cuda"), few, few.to(BF16)):
        for bias in (None, torch.zeros(n, device="cuda"),
                     torch.from_numpy(rng.integers(0, 2, n).astype(np.float32)).cuda()):
            for group_top in (1, 2):
                check(logits, k, True, scoring, bias, groups, top_groups, group_top)


def test_far_logits():
    """Scores that are all but 0 or 1 in fp32: the logits still decide without a
    bias, and renormalised weights do not vanish."""
    l = torch.tensor([[-100.0, -101.0, -99.0, -120.0], [30.0, 40.0, 35.0, 31.0],
                      [-60.0, 50.0, -70.0, 20.0], [-1e4, -2e4, -1e4, 0.0]], device="cuda")
    for renormalize in (False, True):
        check(l, 3, renormalize, "sigmoid", dweights=torch.ones((4, 3), device="cuda"))
    check(l, 2, True, "sigmoid", groups=2, top_groups=1)
    check(l, 3, True, "softmax", scale=3.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_masked_by_the_lowest_value(scoring, dtype):
    """Experts masked by the type's lowest number instead of -inf may be chosen where
    nothing else is left; a bias as low decides like one."""
    rng = np.random.default_rng(11)
    low = torch.finfo(dtype).min
    l = normal(rng, (40, 24), dtype)
    l[torch.from_numpy(rng.random((40, 24)) < 0.8).cuda()] = low
    l[3] = low
    bias = normal(rng, (24,), F32, 0.05)
    bias[5:9] = torch.finfo(F32).min
    for b in (None, bias):
        for groups, top, group_top in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
            check(l, 6, True, scoring, b, groups, top, group_top)
            check(l, 6, False, scoring, b, groups, top, group_top)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_barred(scoring):
    """-inf bars an expert, by its logit or its bias; tokens and groups may have
    none left."""
    rng = np.random.default_rng(5)
    n = 24
    l = normal(rng, (60, n))
    l[torch.from_numpy(rng.random((60, n)) < 0.6).cuda()] = float("-inf")
    l[7], l[8, 3:] = float("-inf"), float("-inf")
    bias = normal(rng, (n,), F32, 0.05)
    bias[4] = float("-inf")
    g = normal(rng, (60, 5))
    for b in (None, bias):
        check(l, 5, True, scoring, b, 1, 1, 1, 2.0, dweights=g)
        check(l, 5, False, scoring, b, 6, 3, 2, 2.0, dweights=g)
        check(l, 5, True, scoring, b, 6, 2, 1, 2.0, dweights=g)


def test_nan_and_infinities():
    """A NaN ranks first; only weights that it enters are NaN."""
    l = torch.zeros((4, 8), device="cuda")
    l[0, 5] = float("nan")
    l[1, 6] = float("inf")
    l[2, :] = torch.arange(8.0)
    for bias in (None, torch.zeros(8, device="cuda")):
        for groups, top in ((1, 1), (4, 2)):
            r = moe.route(l, 2, True, 0, "sigmoid", bias, groups, top, 1)
            ids, w = r.ids.tolist(), r.weights
            assert ids[0] == [5, 0] if groups == 1 else ids[0][0] == 5
            assert torch.isnan(w[0]).all() and torch.isfinite(w[1:]).all()
            assert ids[1][0] == 6 and ids[2] == [7, 6]
            r = moe.route(l, 2, True, 0, "softmax", bias, groups, top, 1, 2.0)
            assert torch.isnan(r.weights[0]).all() and torch.isnan(r.weights[1]).all()
            assert torch.isfinite(r.weights[2:]).all()
    # a bias that forces an expert
    bias = torch.zeros(8, device="cuda")
    bias[3] = float("inf")
    assert moe.route(l[2:], 2, True, 0, "sigmoid", bias).ids.tolist() == [[3, 7], [3, 0]]


def test_strided_and_repeated():
    rng = np.random.default_rng(6)
    wide = normal(rng, (100, 80), BF16)
    l, bias = wide[:, 3:63], normal(rng, (60,), F32, 0.05)
    a = check(l, 6, True, "sigmoid", bias, 6, 3, 2)
    for _ in range(3):
        b = moe.route(l, 6, True, 0, "sigmoid", bias, 6, 3, 2)
        assert all(torch.equal(p, q) for p, q in zip(vars(a).values(), vars(b).values()))


def test_no_tokens():
    l = torch.zeros((0, 8), device="cuda")
    r = check(l, 2, True, "sigmoid", torch.zeros(8, device="cuda"), 4, 2, 2)
    assert r.expert_rows.tolist() == [0] * 8
    assert moe.route_backward(l, r.ids, r.weights, r.weights, True, "sigmoid").shape == (0, 8)


def test_captured_beside_another():
    """A captured call has a workspace of its own: its replays run beside others."""
    rng = np.random.default_rng(7)
    l, other = normal(rng, (3000, 64)), normal(rng, (5000, 64))
    bias = normal(rng, (64,), F32, 0.05)
    args = (8, True, 0, "sigmoid", bias, 8, 4, 2, 2.5)
    want, want_other = moe.route(l, *args), moe.route(other, *args)
    torch.cuda.synchronize()
    live, graph = torch.zeros_like(l), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.route(live, *args)
    live.copy_(l)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            beside = moe.route(other, *args)
        torch.cuda.synchronize()
        for a, b in ((out, want), (beside, want_other)):
            assert all(torch.equal(p, q) for p, q in zip(vars(a).values(), vars(b).values()))


def test_defaults_are_the_plain_router():
    rng = np.random.default_rng(8)
    l, g = normal(rng, (50, 16)), normal(rng, (50, 4))
    a = moe.route(l, 4)
    b = moe.route(l, 4, True, 0, "softmax", None, 1, 1, 1, 1.0)
    assert all(torch.equal(p, q) for p, q in zip(vars(a).values(), vars(b).values()))
    assert torch.equal(moe.route_backward(l, a.ids, a.weights, g),
                       moe.route_backward(l, a.ids, a.weights, g, True, "softmax", 1.0))
    # the same choice by the balanced router, with a bias of zeros
    c = moe.route(l, 4, bias=torch.zeros(16, device="cuda"))
    assert torch.equal(a.ids, c.ids) and torch.equal(a.token_row, c.token_row)


def test_refusals():
    l = torch.zeros((2, 8), device="cuda")
    bad = [dict(scoring="tanh"), dict(groups=3), dict(groups=4, top_groups=5), dict(top_groups=2),
           dict(groups=4, group_top=3), dict(scale=0.0), dict(scale=float("inf")),
           dict(bias=torch.zeros(7, device="cuda")), dict(bias=torch.zeros(8, device="cuda").double()),
           dict(bias=torch.zeros(8)), dict(groups=8, top_groups=1, top_k=2)]
    for how in bad:
        with pytest.raises((ValueError, fo.FoError)):
            moe.route(l, **{"top_k": 2, **how})
    with pytest.raises(ValueError):
        moe.route(l.clone().requires_grad_(), 2, scoring="sigmoid")
    with pytest.raises(ValueError):
        moe.route_backward(l, torch.zeros((2, 2), dtype=torch.int32, device="cuda"),
                           torch.zeros((2, 2), device="cuda"), torch.zeros((2, 2), device="cuda"),
                           scoring="tanh")


def test_more_tokens_than_16_bits_count():
    """So many that a chunk's pairs per expert pass 16 bits (most go to one)."""
    T = 256 * 65536 + 77
    g = torch.Generator(device="cuda").manual_seed(9)
    l = torch.randn((T, 3), generator=g, device="cuda").to(BF16)
    l[:, 1] += 4
    r = moe.route(l, 1, True, 0, "sigmoid")
    ids = r.ids[:, 0].long()
    assert torch.equal(ids, l.float().argmax(1)) or (l.gather(1, ids[:, None]) == l.amax(1, True)).all()
    count = torch.bincount(ids, minlength=3)
    assert torch.equal(r.expert_rows.long(), count)
    span = (count + 127) // 128 * 128
    first = span.cumsum(0) - span
    assert torch.equal(r.expert_first.long(), first)
    for e in range(3):
        tokens = torch.nonzero(ids == e)[:, 0]
        rows = torch.arange(len(tokens), device="cuda") + first[e]
        assert torch.equal(r.token_row[tokens, 0].long(), rows)
        assert torch.equal(r.row_token[rows].long(), tokens)
    assert int((r.row_token >= 0).sum()) == T


def test_numbers_that_are_tensors():
    """They count by what they hold at the call; a scale that requires a gradient is refused."""
    rng = np.random.default_rng(12)
    l, bias = normal(rng, (40, 16)), normal(rng, (16,), F32, 0.05)
    one = lambda v: torch.tensor(v)
    k, groups, top, two, cap, scale = one(1), one(1), one(1), one(1), one(0), one(1.0)
    for v in ((2, 4, 3, 2, 0, 2.0), (3, 2, 1, 1, 8, 0.5), (5, 8, 4, 2, 128, 1.0)):
        for t, x in zip((k, groups, top, two, cap, scale), v):
            t.fill_(x)
        got = moe.route(l, k, True, cap, "sigmoid", bias, groups, top, two, scale)
        want = check(l, v[0], True, "sigmoid", bias, v[1], v[2], v[3], v[5], v[4])
        assert all(torch.equal(p, q) for p, q in zip(vars(got).values(), vars(want).values()))
        assert torch.equal(
            moe.route_backward(l, got.ids, got.weights, got.weights, False, "sigmoid", scale),
            moe.route_backward(l, got.ids, got.weights, got.weights, False, "sigmoid", v[5]))
    plain = [moe.route(l, k.fill_(n)) for n in (2, 6)]
    assert [r.ids.shape[1] for r in plain] == [2, 6]
    order = l.sort(dim=1, descending=True, stable=True).indices.int()
    assert all(torch.equal(r.ids, order[:, :r.ids.shape[1]]) for r in plain)
    for call in (lambda s: moe.route(l, 2, scoring="sigmoid", scale=s),
                 lambda s: moe.route_backward(l, got.ids, got.weights, got.weights, scale=s)):
        with pytest.raises(ValueError):
            call(torch.tensor(1.0, requires_grad=True))


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("how", [dict(top_groups=2), dict(top_groups=0), dict(group_top=3),
                                 dict(group_top=0), dict(groups=2, top_groups=3)])
def test_refusals_of_groups(how, biased):
    """The same with a bias and without, of the plain router's scores as of others."""
    l = torch.zeros((2, 8), device="cuda")
    bias = torch.zeros(8, device="cuda") if biased else None
    for scoring, scale in (("softmax", 1.0), ("softmax", 2.0), ("sigmoid", 1.0)):
        with pytest.raises((ValueError, fo.FoError)):
            moe.route(l, 2, scoring=scoring, scale=scale, bias=bias, **how)
    r = moe.route(l, 2, bias=bias, group_top=2)
    assert r.ids.tolist() == [[0, 1]] * 2

"""The block's operators on the GPU against the 64-bit oracle.

Tolerances, all derived before the first run (e = 2^-24; an output's own rounding
is at most half a step, eps / 2 of its type relative to the value):
 - the weighted sum: a rounding per slot, top_k e of the sum of magnitudes; its
   weights' gradients: a lane adds at most H / 32 + 1 products in a row, then 5 +
   8 sums, so (H / 32 + 16) e of the sum of magnitudes;
 - the activation: expf is within 2 ulp (4 e) and s = 1 / (1 + x) has two
   roundings more; h another two: 8 e relative.  With bf16 outputs the power of
   two's argument is rounded twice, (2 |g| log2(e) ln(2)) e, and it and the
   reciprocal are off by 2^-22 and 2^-23: (4 |g| + 16) e covers these and the
   products.  1 + g (1 - s) may cancel, so its gradient is off by twice that of
   dh v s (1 + |g|).  Products whose value lies
   below the normal numbers may be zeros: 2^-120 absolute;
 - checkpoint codes and scales are exact;
 - norms: a thread's squares are at most H / 256 + 8, then 5 + 32 sums: below 64 e
   for H below 4096 and 96 e here throughout; halved by the root, and with the
   products 64 e of the magnitudes each value is made of;
 - gradients of the norms: 256 e of the magnitudes (three sums, each as above, of
   magnitudes, and products of them); the parameters' (tokens + 256) e of theirs.
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo
from oracle import block as oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import block, moe

BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def normal(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).cuda()


def strided(t, pad, offset=0):
    """The same matrix with `pad` extra elements per row, starting `offset`
    elements into its memory."""
    R, C = t.shape
    buf = torch.full((R * (C + pad) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[offset:].view(R, C + pad)[:, :C]
    v.copy_(t)
    return v


def near(got, want, bound, dtype):
    """|got - want| within bound and the rounding of a value that far off."""
    got = host(got)
    bound = bound + half_step(dtype) * (np.abs(want) + bound) + 2.0 ** -120
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# ------------------------------------------------------------------ the weighted sum

def routing(rng, T, n, k, empty=0.1):
    """token_row and row_token: every row at most once, some slots without one."""
    rows = rng.permutation(n)[:T * k]
    rows = np.concatenate([rows, np.full(T * k - len(rows), -1)])
    token_row = np.where(rng.random((T, k)) < empty, -1, rng.permutation(rows).reshape(T, k))
    row_token = np.full(n, -1)
    for t, s in np.argwhere(token_row >= 0):
        row_token[token_row[t, s]] = t
    dev = lambda a: torch.from_numpy(a).int().cuda()
    return token_row, dev(token_row), dev(row_token)


COMBINE = [(1, 1, 1, 1), (3, 8, 8, 2), (5, 33, 40, 3), (7, 256, 7, 1), (40, 2048, 90, 2),
           (9, 2056, 80, 9), (6, 4101, 20, 3), (130, 64, 1100, 8), (4, 136, 200, 32), (3, 520, 0, 2)]


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("T, H, n, k", COMBINE)
def test_combine(T, H, n, k, types):
    rng = np.random.default_rng(T * H + k)
    t, o = types
    index, token_row, row_token = routing(rng, T, n, k)
    rows, w = normal(rng, (n, H), t), normal(rng, (T, k), F32)
    dy = normal(rng, (T, H), o)
    r64 = host(rows).reshape(n, H)
    rows[row_token < 0] = float("nan")          # nothing reads the rows without a token
    for weights in (w, None):
        w64 = host(weights)
        y = block.combine(rows, token_row, weights, out_dtype=o)
        mag = oracle.combine(np.abs(r64), index, None if w64 is None else np.abs(w64))
        near(y, oracle.combine(r64, index, w64), k * E * mag, o)
        drows, dw = block.combine_backward(dy, rows, token_row, row_token, weights)
        want, want_w = oracle.combine_backward(host(dy), r64, index, w64)
        near(drows, want, E * np.abs(want), t)
        if weights is None:
            assert dw is None
        else:
            _, mag = oracle.combine_backward(np.abs(host(dy)), np.abs(r64), index, w64)
            near(dw, want_w, (H / 32 + 16) * E * mag, F32)
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("pad, offset", [(8, 8), (1, 0), (3, 1), (2, 2), (4, 4)])
def test_combine_strides(pad, offset):
    rng = np.random.default_rng(pad)
    T, H, n, k = 9, 72, 30, 2
    index, token_row, row_token = routing(rng, T, n, k)
    rows, w, dy = normal(rng, (n, H), BF16), normal(rng, (T, k), F32), normal(rng, (T, H), BF16)
    y = block.combine(rows, token_row, w)
    drows, dw = block.combine_backward(dy, rows, token_row, row_token, w)
    out = torch.full((T, H + pad), 7.0, dtype=BF16, device="cuda")
    block.combine(strided(rows, pad, offset), token_row, w, out=out[:, :H])
    assert torch.equal(out[:, :H], y) and (out[:, H:] == 7).all()
    drows2, dw2 = block.combine_backward(strided(dy, pad, offset), strided(rows, pad, offset),
                                         token_row, row_token, w)
    assert torch.equal(drows2, drows)
    # (other threads, another order of the sum)
    near(dw2, host(dw), 2 * (H / 32 + 16) * E * (np.abs(host(dy)).max() * np.abs(host(rows)).max() * H),
         F32)


def test_combine_rows_out_of_range():
    """Their slots add nothing, and the status says so."""
    rows = torch.ones((4, 8), device="cuda")
    index = torch.tensor([[0, 4], [1 << 30, 2]], dtype=torch.int32, device="cuda")
    assert moe.device_status(clear=True) == fo.FO_OK
    y = block.combine(rows, index)
    assert torch.equal(y, torch.ones((2, 8), device="cuda"))
    assert moe.device_status(clear=True) == fo.FO_ERR_ARG
    # a row that holds another token is not written through this one's slot
    row_token = torch.tensor([0, 0, 1, -1], dtype=torch.int32, device="cuda")
    index = torch.tensor([[0, 1], [1, 2]], dtype=torch.int32, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    drows, dw = block.combine_backward(torch.full((2, 8), 3.0, device="cuda"), rows, index,
                                       row_token, w)
    assert torch.equal(drows[:3], torch.full((3, 8), 3.0, device="cuda"))
    assert not drows[3].any() and dw.tolist() == [[24, 24], [0, 24]]
    assert moe.device_status(clear=True) == fo.FO_ERR_ARG


def test_combine_infinite_weights_of_empty_slots():
    index = torch.tensor([[-1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("inf"), 2.0]], device="cuda")
    y = block.combine(torch.ones((1, 3), device="cuda"), index, w)
    assert y.tolist() == [[2, 2, 2]]


# ------------------------------------------------------------------ the activation

def check_act(u, dh, kind):
    I = u.shape[1] // 2
    g, v = np.split(host(u), 2, axis=1)
    h, kept = block.activate(u, kind, checkpoint=True)
    want = oracle.act(g, kind) * v
    off = 8 if u.dtype == F32 else 16 + 4 * np.abs(g)
    near(h, want, off * E * np.abs(want), u.dtype)
    assert torch.equal(block.activate(u, kind)[0], h)
    halves = [oracle.checkpoint(x) for x in (g, v)]
    codes = np.stack([c for c, _, _ in halves], 1)
    scales = np.stack([s for _, s, _ in halves], 1)
    assert np.array_equal(kept.scales.cpu().numpy(), scales.reshape(-1))
    assert np.array_equal(kept.codes.cpu().numpy(), codes.reshape(-1))
    values = np.concatenate([x for _, _, x in halves], 1)
    assert np.array_equal(host(kept.values()), values)
    g, v = np.split(values, 2, axis=1)
    du = block.activate_backward(dh, kept)
    d = host(dh)
    s = 1 / (1 + np.exp(-g)) if kind == "silu" else 1
    want = np.concatenate([d * v * oracle.act_slope(g, kind), d * oracle.act(g, kind)], 1)
    off = 8 if u.dtype == F32 else 16 + 4 * np.abs(g)
    bound = np.concatenate([np.abs(d * v) * s * (1 + np.abs(g)) * off, np.abs(want[:, I:]) * off], 1)
    near(du, want, 2 * E * bound, dh.dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, inter", [(1, 1), (2, 8), (3, 31), (5, 32), (4, 33), (7, 72),
                                         (3, 256), (2, 257), (33, 96), (3, 2056), (2, 4100), (300, 40)])
def test_act(rows, inter, dtype):
    rng = np.random.default_rng(rows * 1000 + inter)
    scale = 10.0 ** rng.uniform(-3, 1.5, (rows, 1))
    u = normal(rng, (rows, 2 * inter), dtype) * torch.from_numpy(scale).to(dtype).cuda()
    for kind in ("silu", "relu", "none"):
        check_act(u, normal(rng, (rows, inter), dtype), kind)


@pytest.mark.parametrize("pad, offset", [(8, 8), (1, 0), (3, 1), (2, 2)])
def test_act_strides(pad, offset):
    rng = np.random.default_rng(pad)
    u, dh = normal(rng, (5, 144), BF16), normal(rng, (5, 72), BF16)
    h, kept = block.activate(u, checkpoint=True)
    h2, kept2 = block.activate(strided(u, pad, offset), checkpoint=True)
    assert torch.equal(h, h2) and torch.equal(kept.codes, kept2.codes)
    assert torch.equal(kept.scales, kept2.scales)
    assert torch.equal(block.activate_backward(dh, kept),
                       block.activate_backward(strided(dh, pad, offset), kept2))


@pytest.mark.parametrize("inter", [64, 33])
def test_act_extremes(inter):
    """Zeros, the smallest and largest numbers, ties between codes, and blocks
    with an infinity or a NaN, which stand for NaNs and leave the others alone."""
    u = torch.zeros((8, 2 * inter), device="cuda")
    u[1, :3] = torch.tensor([1e-45, -3e-45, 2e-44], device="cuda")
    u[2, :4] = torch.tensor([3e38, -3.4e38, 1e38, 1.0], device="cuda")
    u[3, :4] = torch.tensor([64.0, 0.5, 1.5, -2.5], device="cuda")      # a step of 1
    u[4, :2] = torch.tensor([127.6, -127.9], device="cuda")
    u[5, inter:inter + 2] = torch.tensor([2.0 ** -126, 2.0 ** -121], device="cuda")
    u[6, 0] = float("inf")
    u[7, inter + 1] = float("nan")
    u[7, inter - 1] = 3.0
    _, kept = block.activate(u, checkpoint=True)
    halves = [oracle.checkpoint(x) for x in np.split(host(u), 2, axis=1)]
    assert np.array_equal(kept.scales.cpu().numpy(),
                          np.stack([s for _, s, _ in halves], 1).reshape(-1))
    assert np.array_equal(kept.codes.cpu().numpy(),
                          np.stack([c for c, _, _ in halves], 1).reshape(-1))
    values = np.concatenate([v for _, _, v in halves], 1)
    got = host(kept.values())
    assert np.array_equal(got, values, equal_nan=True)
    du = host(block.activate_backward(torch.ones((8, inter), device="cuda"), kept))
    bad = np.isnan(values)
    assert bad[6, :32].all() and bad[7, inter:inter + 32].all() and bad.sum() == 64
    assert np.isnan(du[6, :32]).all() and np.isnan(du[7, :32]).all()
    assert np.isfinite(du[:6]).all()


def test_act_far_gates():
    """silu of gates beyond expf's range: zeros and the gate itself."""
    g = torch.tensor([[-1e4, -200.0, -100.0, 100.0, 200.0, 1e4]], device="cuda")
    h, _ = block.activate(torch.cat((g, torch.full_like(g, 2.0)), 1))
    assert h.tolist() == [[0, 0, 0, 200, 400, 2e4]]
    for x in g[0].tolist():
        u = torch.tensor([[x, 2.0]], device="cuda")
        _, kept = block.activate(u, checkpoint=True)
        du = block.activate_backward(torch.ones((1, 1), device="cuda"), kept)
        v = host(kept.values())[0]
        assert du.tolist() == [[v[1], v[0]] if x > 0 else [0, 0]]


# ------------------------------------------------------------------ the norms

def check_norm(x, residual, post, gate, scale, pre, eps, dstream, dy):
    p = [host(t) for t in (x, residual, post, gate, pre)]
    x64, r64, post64, gate64, pre64 = p
    how = dict(post_gain=post, gate=gate, scale=scale, pre_gain=pre)
    scale = float(np.float32(scale))
    n = block.norm(x, residual, eps=eps, **how)
    f = oracle.norm(x64, r64, post64, gate64, scale, pre64, float(np.float32(eps)))
    T, H = x64.shape
    mag = np.abs(f["q"] * f["u"]) + (0 if r64 is None else np.abs(r64))
    if n.stream is x:
        assert residual is None and post is None and gate is None and scale == 1
    else:
        near(n.stream, f["sum"], 64 * E * mag, n.stream.dtype)
    # the second norm's inputs are off by 64 e of mag each
    sn_mag = mag * f["r2"]
    sn_mag = sn_mag + np.abs(f["sum"]) * f["r2"] * (sn_mag * np.abs(f["sum"]) * f["r2"]).mean(1, keepdims=True)
    if pre is None:
        assert n.y is None
    else:
        near(n.y, f["sum"] * f["r2"] * pre64, 128 * E * sn_mag * np.abs(pre64), x.dtype)
    d = block.norm_backward(x, residual, n, dstream=dstream, dy=dy, **how)
    d64 = np.zeros((T, H)) if dstream is None else host(dstream)
    want = oracle.norm_backward(x64, r64, post64, gate64, scale, pre64, float(np.float32(eps)),
                                None if dstream is None else d64, host(dy))
    big = np.abs(d64)
    if pre is not None:
        e = np.abs(host(dy) * pre64)
        big = big + f["r2"] * (e + sn_mag * (e * sn_mag).mean(1, keepdims=True))
    if residual is None:
        assert d.residual is None
    else:
        near(d.residual, want["residual"], 256 * E * big, residual.dtype)
    w = np.abs(f["q"]) * big
    if post is not None:
        xn = np.abs(f["xn"])
        near(d.post_gain, want["post_gain"], (T + 256) * E * (w * xn).sum(0), post.dtype)
        w = w * np.abs(post64)
        w = f["r1"] * (w + xn * (w * xn).mean(1, keepdims=True))
    else:
        assert d.post_gain is None
    near(d.x, want["x"], 256 * E * w, x.dtype)
    if gate is not None:
        mag = (scale * np.abs(f["u"]) * big).reshape(gate64.size // H, -1, H).sum(1)
        near(d.gate, want["gate"], (T + 256) * E * mag.reshape(gate64.shape), gate.dtype)
    else:
        assert d.gate is None
    if pre is not None:
        near(d.pre_gain, want["pre_gain"], (T + 256) * E * (np.abs(host(dy)) * sn_mag).sum(0),
             pre.dtype)
    return n, d


def norm_case(rng, T, H, x_type, s_type, p_type, post, gates, pre, residual):
    make = lambda there, shape, t: normal(rng, shape, t) if there else None
    x = normal(rng, (T, H), x_type, 2.0)
    s_type = s_type if residual else x_type
    gate = None if gates is None else normal(rng, (H,) if gates == 0 else (gates, H), p_type)
    return [x, make(residual, (T, H), s_type), make(post, (H,), p_type), gate, 0.75,
            make(pre, (H,), p_type), 1e-5, make(True, (T, H), s_type), make(pre, (T, H), x_type)]


NORM_SIZES = [(1, 1), (1, 8), (2, 33), (3, 64), (5, 264), (24, 72), (4, 1024), (6, 1032), (3, 1416),
              (12, 2752), (2, 4096), (3, 4104), (2, 8192), (1, 8200), (3, 1001), (2, 9001)]
TYPES = [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32), (BF16, BF16, F32),
         (F32, F32, BF16)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T, H", NORM_SIZES)
def test_norm(T, H, types):
    rng = np.random.default_rng(T * 10000 + H)
    gates = [None, 0, 1, T] + [g for g in (2, 3, 4) if g < T and T % g == 0]
    for i, (post, pre, residual) in enumerate(((True, True, True), (False, True, True),
                                               (True, False, True), (True, True, False))):
        check_norm(*norm_case(rng, T, H, *types, post, gates[(i + H) % len(gates)], pre, residual))


@pytest.mark.parametrize("H", [64, 2752, 8192, 333])
@pytest.mark.parametrize("T, gates", [(2500, 0), (2500, 4), (2500, 1250), (3000, 3000), (777, 7),
                                      (1217, 1), (5000, 100)])
def test_norm_many_tokens(T, gates, H):
    """More tokens than workers, gates' rows that end inside a worker's range."""
    if H > 3000 and T > 2500:
        T, gates = 1500, 1500 if gates == 3000 else 30
    rng = np.random.default_rng(T + gates)
    check_norm(*norm_case(rng, T, H, BF16, F32, F32, True, gates, True, True))


def test_norm_alone():
    """The norm before a block: the stream is x itself."""
    rng = np.random.default_rng(0)
    x, pre = normal(rng, (3, 64), BF16), normal(rng, (64,), BF16)
    n = block.norm(x, pre_gain=pre)
    assert n.stream is x
    check_norm(x, None, None, None, 1.0, pre, 1e-6, None, normal(rng, (3, 64), BF16))
    # and its gradient with one of the stream besides
    check_norm(x, None, None, None, 1.0, pre, 1e-6, normal(rng, (3, 64), BF16),
               normal(rng, (3, 64), BF16))


@pytest.mark.parametrize("H", [72, 9000])
def test_norm_without_a_gradient_of_the_stream(H):
    rng = np.random.default_rng(1)
    case = norm_case(rng, 5, H, BF16, BF16, F32, True, 0, True, True)
    case[7] = None
    check_norm(*case)
    # and of the stream alone
    case = norm_case(rng, 5, H, BF16, BF16, F32, False, 5, False, True)
    check_norm(*case)


@pytest.mark.parametrize("pad, offset", [(8, 8), (1, 0), (3, 1), (2, 2)])
def test_norm_strides(pad, offset):
    rng = np.random.default_rng(pad)
    x, res, post, gate, scale, pre, eps, ds, dy = norm_case(rng, 6, 72, BF16, BF16, BF16, True, 3,
                                                            True, True)
    wide = lambda t: strided(t, pad, offset)
    check_norm(wide(x), wide(res), post, wide(gate), scale, pre, eps, wide(ds), wide(dy))


def test_norm_rows_are_alone():
    """Zeros, infinities and NaN stay in their rows; a row of zeros without eps is
    0 / 0."""
    rng = np.random.default_rng(2)
    x, res, post, gate, scale, pre, _, ds, dy = norm_case(rng, 8, 136, F32, F32, F32, True, 0, True,
                                                          True)
    x[2], res[2] = 0, 0
    clean = block.norm(x, res, post, gate, scale, pre, eps=1e-6)
    assert not clean.y[2].any() and not clean.stream[2].any()
    assert torch.isfinite(clean.y).all()
    x[4, 3], x[5, 7], res[6, 1] = float("inf"), float("nan"), float("-inf")
    n = block.norm(x, res, post, gate, scale, pre, eps=1e-6)
    ok = [0, 1, 2, 3, 7]
    assert torch.equal(n.y[ok], clean.y[ok]) and torch.equal(n.stream[ok], clean.stream[ok])
    assert torch.isnan(n.y[5]).all() and torch.isnan(n.y[4]).any() and torch.isnan(n.y[6]).any()
    d0 = block.norm_backward(x, res, clean, ds, dy, post, gate, scale, pre)
    d = block.norm_backward(x, res, n, ds, dy, post, gate, scale, pre)
    assert torch.equal(d.x[ok], d0.x[ok]) and torch.equal(d.residual[ok], d0.residual[ok])
    assert torch.isnan(block.norm(torch.zeros((1, 8), device="cuda"), eps=0.0,
                                  pre_gain=torch.ones(8, device="cuda")).y).all()


def test_nothing():
    """No tokens, no columns, no rows."""
    z = lambda *s: torch.zeros(s, device="cuda")
    n = block.norm(z(0, 16), z(0, 16), post_gain=z(16), gate=z(16), pre_gain=z(16))
    assert n.y.shape == (0, 16)
    d = block.norm_backward(z(0, 16), z(0, 16), n, z(0, 16), z(0, 16), z(16), z(16), 1.0, z(16))
    assert not d.post_gain.any() and not d.gate.any() and not d.pre_gain.any()
    assert block.norm(z(3, 0), z(3, 0), pre_gain=z(0)).y.shape == (3, 0)
    h, kept = block.activate(z(0, 64), checkpoint=True)
    assert block.activate_backward(h, kept).shape == (0, 64)
    h, kept = block.activate(z(4, 0), checkpoint=True)
    assert block.activate_backward(h, kept).shape == (4, 0)
    none = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    assert block.combine(z(0, 8), none).tolist() == [[0] * 8] * 2
    drows, dw = block.combine_backward(z(2, 8), z(0, 8), none, none[:0, 0], z(2, 2))
    assert drows.shape == (0, 8) and not dw.any()
    empty = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    drows, dw = block.combine_backward(z(0, 8), z(3, 8) + 1, empty, none.view(-1)[:3].contiguous(),
                                       z(0, 2))
    assert not drows.any() and dw.shape == (0, 2)
    # rows without columns: products of nothing
    index = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    drows, dw = block.combine_backward(z(1, 0), z(3, 0), index,
                                       torch.tensor([0, 0, -1], dtype=torch.int32, device="cuda"),
                                       z(1, 2) + 5)
    assert drows.shape == (3, 0) and not dw.any() and block.combine(z(3, 0), index).shape == (1, 0)
    assert block.activate(z(0, 64), checkpoint=True)[1].values().shape == (0, 64)
    assert block.activate(z(4, 0), checkpoint=True)[1].values().shape == (4, 0)


# ------------------------------------------------------------------ how they are called

def all_calls(s):
    """One pass of each operator over s, a dict of tensors."""
    n = block.norm(s["x"], s["res"], s["post"], s["gate"], 0.5, s["pre"])
    d = block.norm_backward(s["x"], s["res"], n, s["ds"], s["dy"], s["post"], s["gate"], 0.5,
                            s["pre"])
    h, kept = block.activate(s["u"], checkpoint=True)
    du = block.activate_backward(s["dh"], kept)
    y = block.combine(s["rows"], s["token_row"], s["w"])
    drows, dw = block.combine_backward(s["dy2"], s["rows"], s["token_row"], s["row_token"], s["w"])
    return [n.stream, n.y, d.x, d.residual, d.post_gain, d.gate, d.pre_gain, h, du, y, drows, dw]


def some_inputs(seed, H=264, T=300):
    rng = np.random.default_rng(seed)
    x, res, post, gate, _, pre, _, ds, dy = norm_case(rng, T, H, BF16, BF16, BF16, True, 3, True, True)
    _, token_row, row_token = routing(rng, 50, 120, 2)
    return dict(x=x, res=res, post=post, gate=gate, pre=pre, ds=ds, dy=dy,
                u=normal(rng, (70, 2 * H), BF16), dh=normal(rng, (70, H), BF16),
                rows=normal(rng, (120, H), BF16), token_row=token_row, row_token=row_token,
                w=normal(rng, (50, 2), F32), dy2=normal(rng, (50, H), BF16))


@pytest.mark.parametrize("H", [264, 333, 4200])
def test_repeated_and_captured(H):
    """The same results in every run, from a graph, and on another stream beside
    the first; a graph's replay reads what its inputs hold by then."""
    a, b = some_inputs(0, H), some_inputs(1, H)
    want_a, want_b = all_calls(a), all_calls(b)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(all_calls(a), want_a))
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(one):
        got_a = all_calls(a)
    with torch.cuda.stream(two):
        got_b = all_calls(b)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got_a, want_a))
    assert all(torch.equal(p, q) for p, q in zip(got_b, want_b))
    live = {k: v.clone() for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(live)
    for src, want in ((a, want_a), (b, want_b), (a, want_a)):
        for k in live:
            live[k].copy_(src[k])
        graph.replay()
        beside = all_calls(b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
        assert all(torch.equal(p, q) for p, q in zip(beside, want_b))


def test_refusals():
    z = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")
    bad = [
        lambda: block.norm(z(2, 8), z(2, 8, t=BF16)),                   # fp32 into a bf16 stream
        lambda: block.norm(z(2, 8), z(3, 8)),
        lambda: block.norm(z(2, 8), post_gain=z(7)),
        lambda: block.norm(z(2, 8), post_gain=z(8), pre_gain=z(8, t=BF16)),
        lambda: block.norm(z(2, 8), gate=z(3, 8)),
        lambda: block.norm(z(2, 8), gate=z(0, 8)),
        lambda: block.norm(z(2, 8).half(), pre_gain=z(8)),
        lambda: block.norm(z(2, 8).t().contiguous().t(), pre_gain=z(8)),
        lambda: block.norm(z(1, 8).expand(2, 8), pre_gain=z(8)),
        lambda: block.norm(z(2, 8).requires_grad_(), pre_gain=z(8)),
        lambda: block.norm(z(2, 8), pre_gain=z(8).cpu()),
        lambda: block.norm(z(2, 8), pre_gain=z(8), scale=float("nan")),
        lambda: block.norm_backward(z(2, 8), None, block.norm(z(2, 8), pre_gain=z(8)), pre_gain=z(8)),
        lambda: block.norm_backward(z(2, 8), None, block.norm(z(2, 8)), dy=z(2, 8), pre_gain=z(8)),
        lambda: block.norm_backward(z(2, 8), None, block.norm(z(3, 8), pre_gain=z(8)), dy=z(2, 8),
                                    pre_gain=z(8)),
        lambda: block.activate(z(2, 7)),
        lambda: block.activate(z(2, 8), act="tanh"),
        lambda: block.activate(z(2, 8).double()),
        lambda: block.activate_backward(z(2, 5), block.activate(z(2, 8), checkpoint=True)[1]),
        lambda: block.combine(z(4, 8), z(2, 2)),
        lambda: block.combine(z(4, 8), z(2, 2).int(), z(2, 3)),
        lambda: block.combine(z(4, 8), z(2, 2).int(), out=z(2, 7)),
        lambda: block.combine_backward(z(2, 7), z(4, 8), z(2, 2).int(), z(4).int()),
        lambda: block.combine_backward(z(2, 8), z(4, 8), z(2, 2).int(), z(5).int()),
    ]
    for call in bad:
        with pytest.raises((ValueError, fo.FoError)):
            call()


@pytest.mark.parametrize("H", [72, 73, 4096])
@pytest.mark.parametrize("slots", [(0, 1), (1, 4), (2, 5), (0, 5)])
def test_combine_a_row_named_twice(H, slots):
    """Forward it counts twice; its gradient is that of the last slot.  A row that
    another token's slot names as well: left out there, and the status says so."""
    T, k = 37, 6
    rng = np.random.default_rng(H)
    token_row = np.arange(T * k, dtype=np.int32).reshape(T, k)
    row_token = np.repeat(np.arange(T, dtype=np.int32), k)
    lost = token_row[:, slots[1]].copy()
    token_row[:, slots[1]] = token_row[:, slots[0]]
    row_token[lost] = -1
    rows = rng.integers(-4, 5, (T * k, H)).astype(np.float32)
    w = rng.integers(1, 5, (T, k)).astype(np.float32)
    dy = rng.integers(-4, 5, (T, H)).astype(np.float32)
    put = lambda a: torch.from_numpy(a).cuda()
    y = block.combine(put(rows), put(token_row), put(w))
    assert np.array_equal(y.cpu().numpy(), np.einsum("tk,tkh->th", w, rows[token_row]))
    drows, dw = block.combine_backward(put(dy), put(rows), put(token_row), put(row_token), put(w))
    want = np.zeros_like(rows)
    for t in range(T):
        for s in range(k):
            want[token_row[t, s]] = w[t, s] * dy[t]
    assert np.array_equal(drows.cpu().numpy(), want)
    assert np.array_equal(dw.cpu().numpy(), np.einsum("th,tkh->tk", dy, rows[token_row]))
    assert moe.device_status() == fo.FO_OK
    token_row[1, slots[0]] = token_row[0, 3]
    drows, dw = block.combine_backward(put(dy), put(rows), put(token_row), put(row_token), put(w))
    assert np.array_equal(drows.cpu().numpy()[token_row[0, 3]], want[token_row[0, 3]])
    assert dw.cpu().numpy()[1, slots[0]] == 0
    assert moe.device_status(clear=True) == fo.FO_ERR_ARG


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("H", [8, 40, 64, 72, 136, 1000, 2040, 2056])
@pytest.mark.parametrize("T, k", [(1, 1), (9, 1), (9, 2), (14, 3)])
def test_combine_padded_rows(T, k, H, types):
    """Every row of 8 columns and padding on 16 bytes, an odd number of eights to a row or an
    even one: all of y, and nothing beside or behind it."""
    rng = np.random.default_rng(H + T)
    t, o = types
    n = 3 * T * k
    index, token_row, row_token = routing(rng, T, n, k)
    rows, w, dy = normal(rng, (n, H), t), normal(rng, (T, k), F32), normal(rng, (T, H), o)
    r64, w64 = host(rows), host(w)
    want = oracle.combine(r64, index, w64)
    bound = k * E * oracle.combine(np.abs(r64), index, np.abs(w64))
    drows, dw = block.combine_backward(dy, rows, token_row, row_token, w)
    for pad in (4, 8, 24, 3, 2):
        buf = torch.full(((T + 1) * (H + pad),), 7.0, dtype=o, device="cuda")
        out = buf[:T * (H + pad)].view(T, H + pad)
        block.combine(strided(rows, pad), token_row, w, out=out[:, :H])
        near(out[:, :H], want, bound, o)
        assert (out[:, H:] == 7).all() and (buf[T * (H + pad):] == 7).all()
        drows2, dw2 = block.combine_backward(strided(dy, pad), strided(rows, pad), token_row,
                                             row_token, w)
        assert torch.equal(drows2, drows)
        mag = np.abs(host(dy)).max() * np.abs(r64).max() * H
        near(dw2, host(dw), 2 * (H / 32 + 16) * E * mag, F32)
    assert moe.device_status() == fo.FO_OK


def test_norm_scale_of_a_tensor():
    """A scale or an eps that is a tensor counts by what it holds at the call, and one
    that requires a gradient is refused."""
    x, g = torch.ones((3, 8), device="cuda"), torch.ones(8, device="cuda")
    for device in ("cpu", "cuda"):
        scale, eps = torch.tensor(0.5, device=device), torch.tensor(0.0, device=device)
        for s, e in ((0.5, 0.0), (2.0, 3.0), (0.25, 15.0)):
            scale.fill_(s)
            eps.fill_(e)
            n = block.norm(x, scale=scale, pre_gain=g, eps=eps)
            assert (n.stream == s).all() and torch.equal(n.y, block.norm(x, scale=s, pre_gain=g, eps=e).y)
            assert (block.norm_backward(x, None, n, x, x - x, scale=scale, pre_gain=g).x == s).all()
    for how in (dict(scale=torch.tensor(1.0, requires_grad=True)),
                dict(eps=torch.tensor(1.0, requires_grad=True))):
        with pytest.raises(ValueError):
            block.norm(x, pre_gain=g, **how)
    with pytest.raises(ValueError):
        block.norm_backward(x, None, n, x, x, pre_gain=g, scale=torch.tensor(1.0, requires_grad=True))
    with torch.no_grad():
        assert (block.norm(x, scale=torch.tensor(2.0, requires_grad=True)).stream == 2).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("H, pad", [(264, 0), (264, 3), (264, 2), (4104, 0), (8200, 0), (9001, 0)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_gradient_does_not_see_the_stream(H, pad, types, residual):
    """Without a norm before the next block the gradients take no value of the stream: an
    infinity or a NaN there stays out of all of them, one of x where nothing norms it comes
    into the gate's gradient of its own column alone."""
    rng = np.random.default_rng(H + pad)
    wide = (lambda t: strided(t, pad)) if pad else (lambda t: t)
    bad = [(1, 3, float("inf")), (2, 5, float("nan")), (4, H - 1, float("-inf"))]
    for post in ((True, False) if residual else (False,)):
        x, res, p, gate, scale, _, eps, ds, _ = norm_case(rng, 6, H, *types, post, 3, False, residual)
        n = block.norm(x, res, p, gate, scale, eps=eps)
        want = block.norm_backward(x, res, n, ds, None, p, gate, scale)
        touched = res if residual else x
        for t, c, v in bad:
            touched[t, c] = v
        got = block.norm_backward(wide(x), None if res is None else wide(res), n, wide(ds), None, p,
                                  gate, scale)
        for name in ("x", "residual", "post_gain"):
            a, b = getattr(got, name), getattr(want, name)
            assert (a is None and b is None) or torch.isfinite(a).all(), name
        # (dx and the residual's gradient go by the same steps; sums may have another order)
        if not pad:
            assert torch.equal(got.x, want.x)
            assert not residual or torch.equal(got.residual, want.residual)
        alone = torch.isfinite(got.gate)
        assert alone.all() if residual else int((~alone).sum()) == len(bad)
        if not pad:
            assert torch.equal(got.gate[alone], want.gate[alone])
        if post:        # and where x is normed, its NaN stays out of the residual's gradient
            for t, c, v in bad:
                x[t, c] = v
            got = block.norm_backward(wide(x), wide(res), block.norm(x, res, p, gate, scale, eps=eps),
                                      wide(ds), None, p, gate, scale)
            assert torch.equal(got.residual, ds.to(res.dtype))


@pytest.mark.parametrize("rows", [0, 1, 3])
@pytest.mark.parametrize("H", [16, 33, 0])
def test_norm_of_no_tokens_with_a_gate(H, rows):
    """A gate per token has no rows either; rows that no token meets have zeros."""
    z = lambda *s: torch.zeros(s, device="cuda")
    n = block.norm(z(0, H), z(0, H), z(H), z(rows, H), 0.5, z(H))
    assert n.stream.shape == n.y.shape == (0, H)
    d = block.norm_backward(z(0, H), z(0, H), n, z(0, H), z(0, H), z(H), z(rows, H), 0.5, z(H))
    assert d.x.shape == d.residual.shape == (0, H) and d.gate.shape == (rows, H)
    assert not d.gate.any() and not d.post_gain.any() and not d.pre_gain.any()
    with pytest.raises(ValueError):
        block.norm(z(2, H), gate=z(0, H))


PADS = [(4, 0), (8, 8), (1, 0), (3, 1), (2, 2), (24, 0)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("pad, offset", PADS)
@pytest.mark.parametrize("T, H", [(1, 72), (7, 72), (6, 136), (4, 1000), (3, 4104)])
def test_norm_strides_of_all_types(T, H, pad, offset, types):
    rng = np.random.default_rng(pad + H)
    wide = lambda t: strided(t, pad, offset)
    for post, pre in ((True, True), (False, True), (True, False)):
        x, res, p, gate, scale, q, eps, ds, dy = norm_case(rng, T, H, *types, post, T, pre, True)
        check_norm(wide(x), wide(res), p, wide(gate), scale, q, eps, wide(ds),
                   None if dy is None else wide(dy))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad, offset", PADS)
@pytest.mark.parametrize("rows, inter", [(1, 72), (7, 72), (6, 136), (5, 33), (3, 2056)])
def test_act_strides_of_all_types(rows, inter, pad, offset, dtype):
    rng = np.random.default_rng(pad + inter)
    u, dh = normal(rng, (rows, 2 * inter), dtype), normal(rng, (rows, inter), dtype)
    for kind in ("silu", "relu"):
        check_act(strided(u, pad, offset), strided(dh, pad, offset), kind)
        h, kept = block.activate(u, kind, checkpoint=True)
        wide, same = block.activate(strided(u, pad, offset), kind, checkpoint=True)
        assert torch.equal(h, wide) and torch.equal(kept.codes, same.codes)


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("H", [8, 72, 136, 1000, 4104, 33, 4097])
def test_norm_writes_its_rows_alone(H, types):
    """By the library's calls, which take strides of the outputs too: nothing in the rows'
    padding, before the first row or behind the last."""
    rng = np.random.default_rng(H)
    x_type, s_type = types
    T, code = 5, {BF16: fo.FO_TYPE_BF16, F32: fo.FO_TYPE_F32}
    x, res = normal(rng, (T, H), x_type), normal(rng, (T, H), s_type)
    p, q = normal(rng, (H,), F32), normal(rng, (H,), F32)
    ds, dy = normal(rng, (T, H), s_type), normal(rng, (T, H), x_type)
    want = block.norm(x, res, p, None, 0.5, q)
    dwant = block.norm_backward(x, res, want, ds, dy, p, None, 0.5, q)
    desc = fo.make_norm_desc(T, H, code[x_type], code[s_type], fo.FO_TYPE_F32, 1, 0.5, 1e-6)
    ws = torch.empty(fo.fo_block_norm_workspace(desc), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for pad in (4, 8, 24, 1, 2):
        W = H + pad
        bufs = {}

        def out(name, dtype, rows=T, cols=H):
            bufs[name] = torch.full(((rows + 2) * W,), 7.0, dtype=dtype, device="cuda")
            return bufs[name].data_ptr() + W * bufs[name].element_size()

        rstd = torch.empty((2, T), device="cuda")
        at = rstd.data_ptr()
        fo.fo_block_norm(desc, x.data_ptr(), H, res.data_ptr(), H, p.data_ptr(), 0, 0, q.data_ptr(),
                         out("stream", s_type), W, out("y", x_type), W, at, at + 4 * T, stream)
        dp, dq = torch.empty_like(p), torch.empty_like(q)
        fo.fo_block_norm_backward(desc, x.data_ptr(), H, res.data_ptr(), H, p.data_ptr(), 0, 0,
                                  q.data_ptr(), at, at + 4 * T, ds.data_ptr(), H, dy.data_ptr(), H,
                                  out("x", x_type), W, out("residual", s_type), W, dp.data_ptr(), 0,
                                  dq.data_ptr(), ws.data_ptr(), stream)
        for name, w in (("stream", want.stream), ("y", want.y), ("x", dwant.x),
                        ("residual", dwant.residual)):
            m = bufs[name].view(T + 2, W)
            # (other kernels, other orders of a row's sums: within the norms' bound of it)
            off = (m[1:-1, :H].double() - w.double()).abs().amax()
            assert off <= 2 * (half_step(w.dtype) + 256 * E) * 16 * w.double().abs().amax(), name
            assert (m[0] == 7).all() and (m[-1] == 7).all() and (m[1:-1, H:] == 7).all(), name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [8, 72, 136, 1000, 33, 2056])
def test_act_and_combine_gradients_write_their_rows_alone(H, dtype):
    rng = np.random.default_rng(H)
    T, k, code = 7, 2, {BF16: fo.FO_TYPE_BF16, F32: fo.FO_TYPE_F32}[dtype]
    n = 3 * T * k
    _, token_row, row_token = routing(rng, T, n, k)
    rows, w, dy = normal(rng, (n, H), dtype), normal(rng, (T, k), F32), normal(rng, (T, H), dtype)
    drows, dw = block.combine_backward(dy, rows, token_row, row_token, w)
    u = normal(rng, (T, 2 * H), dtype)
    h, kept = block.activate(u, checkpoint=True)
    du = block.activate_backward(dy, kept)
    stream, status = torch.cuda.current_stream().cuda_stream, torch.zeros(1, dtype=torch.int32,
                                                                          device="cuda")
    for pad in (4, 8, 24, 1, 2):

        def check(want, call):
            R, C = want.shape
            buf = torch.full((R + 2, C + pad), 7.0, dtype=dtype, device="cuda")
            call(buf[1].data_ptr(), C + pad)
            assert torch.equal(buf[1:-1, :C], want)
            assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[1:-1, C:] == 7).all()

        got = torch.empty_like(dw)
        check(drows, lambda to, stride: fo.fo_moe_combine_backward(
            dy.data_ptr(), code, H, rows.data_ptr(), code, n, H, H, token_row.data_ptr(),
            row_token.data_ptr(), w.data_ptr(), T, k, to, stride, got.data_ptr(), status.data_ptr(),
            stream))
        check(h, lambda to, stride: fo.fo_gated_act(u.data_ptr(), code, T, H, 2 * H, fo.FO_ACT_SILU,
                                                    to, stride, 0, 0, stream))
        check(du, lambda to, stride: fo.fo_gated_act_backward(
            dy.data_ptr(), code, T, H, H, fo.FO_ACT_SILU, kept.codes.data_ptr(),
            kept.scales.data_ptr(), to, stride, stream))
    assert status.item() == fo.FO_OK


@pytest.mark.parametrize("H, pad", [(4096, 0), (4095, 1)])
def test_rows_past_32_bits(H, pad):
    """Offsets above 2^32 elements: the last rows as calls on those alone have them."""
    T, last, W = (1 << 32) // 4096 + 40, 24, H + pad
    g = torch.Generator(device="cuda").manual_seed(H)

    def draw(rows, cols=H, stride=W):
        t = torch.empty((rows, stride), dtype=BF16, device="cuda")[:, :cols]
        t[-last:] = torch.randn((last, cols), generator=g, device="cuda")
        t[:-last] = 1
        return t

    x, res, ds, dy = (draw(T) for _ in range(4))
    p, q = (torch.randn(H, generator=g, device="cuda") for _ in range(2))
    n = block.norm(x, res, p, None, 0.5, q)
    few = block.norm(x[-last:], res[-last:], p, None, 0.5, q)
    assert torch.equal(n.stream[-last:], few.stream) and torch.equal(n.y[-last:], few.y)
    d = block.norm_backward(x, res, n, ds, dy, p, None, 0.5, q)
    want = block.norm_backward(x[-last:], res[-last:], few, ds[-last:], dy[-last:], p, None, 0.5, q)
    assert torch.equal(d.x[-last:], want.x) and torch.equal(d.residual[-last:], want.residual)
    del d, n, ds
    # the same rows as a table, which two tokens name from both of its ends
    index = torch.tensor([[T - 1, 0], [T - 2, -1]], dtype=torch.int32, device="cuda")
    row_token = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    row_token[[T - 1, 0, T - 2]] = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, 0.5], [4.0, 8.0]], device="cuda")
    y = block.combine(x, index, w)
    assert torch.equal(y[0], (2 * x[-1].float() + 0.5 * x[0].float()).to(BF16))
    assert torch.equal(y[1], 4 * x[-2])
    drows, dw = block.combine_backward(y, x, index, row_token, w)
    assert torch.equal(drows[-1], 2 * y[0]) and torch.equal(drows[-2], 4 * y[1])
    assert torch.equal(drows[0], 0.5 * y[0])
    drows[[T - 1, T - 2, 0]] = 0
    assert not drows.any()
    del x, res, dy, drows
    # and the activation
    I = 14336 - pad
    R = (1 << 32) // (2 * 14336) + 40
    u, dh = draw(R, 2 * I, 2 * I), draw(R, I, I)
    h, kept = block.activate(u, checkpoint=True)
    few, fewer = block.activate(u[-last:], checkpoint=True)
    assert torch.equal(h[-last:], few) and torch.equal(kept.codes[-fewer.codes.numel():], fewer.codes)
    assert torch.equal(block.activate_backward(dh, kept)[-last:],
                       block.activate_backward(dh[-last:], fewer))
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [32, 33])
def test_act_gates_where_sigmoid_ends(inter, dtype):
    """silu of gates about -88, where 1 / (1 + e^-g) passes below the normal numbers: its
    product with a value that is not small is no zero.  s may be zero where e^-g passes
    fp32's largest number; else as above."""
    g = -torch.arange(127 - 63, 127, device="cuda", dtype=F32).repeat(inter)
    g = g[:g.numel() // inter * inter].view(-1, inter).to(dtype)      # (codes hold whole numbers)
    last = 2.0 ** -127.9
    rng = np.random.default_rng(inter)
    for size in (1.0, 40.0, 2.0 ** 40, 2.0 ** 100):
        v = torch.from_numpy(size * rng.choice([-1.0, 1.0], g.shape)).to(dtype).cuda()
        dh = normal(rng, tuple(g.shape), dtype)
        h, kept = block.activate(torch.cat((g, v), 1), checkpoint=True)
        assert torch.equal(kept.values(), torch.cat((g, v), 1).float())
        g64, v64, d64 = host(g), host(v), host(dh)
        off = 8 if dtype == F32 else 16 + 4 * np.abs(g64)
        want = oracle.act(g64, "silu") * v64
        near(h, want, off * E * np.abs(want) + last * np.abs(g64 * v64), dtype)
        assert size < 40 or bool((h[g >= -88] != 0).all())
        du = block.activate_backward(dh, kept)
        want = d64 * oracle.act(g64, "silu")
        near(du[:, inter:], want, 2 * off * E * np.abs(want) + last * np.abs(g64 * d64), dtype)
        s = 1 / (1 + np.exp(-g64))
        size_of = np.abs(d64 * v64) * (1 + np.abs(g64))
        near(du[:, :inter], d64 * v64 * oracle.act_slope(g64, "silu"),
             2 * off * E * s * size_of + last * size_of, dtype)


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, F32)])
@pytest.mark.parametrize("H", [64, 2752, 333, 4104])
@pytest.mark.parametrize("T, gates", [(2500, 0), (2500, None), (2500, 4), (2500, 1250), (3000, 3000),
                                      (1217, 1)])
def test_norm_of_many_tokens_without_the_second(T, gates, H, types):
    if H > 2000:
        T, gates = T // 5, 4 if gates == 4 else gates and min(gates, T // 5)
        gates = gates if gates in (0, 1, 4, None) else T
    rng = np.random.default_rng(T + H)
    for post, residual in ((True, True), (False, True), (True, False)):
        check_norm(*norm_case(rng, T, H, *types, post, gates, False, residual))

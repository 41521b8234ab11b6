"""The expert layer's operators on the GPU against the 64-bit oracle.

Tolerances, all derived before the first run:
 - 4-bit codes, scales, values and the router's integers are exact;
 - softmax weights: expf is within 2 ulp, the sums of up to 1024 terms are
   pairwise over 32 lanes (about 37 roundings at most) and one division, so
   64 * 2^-24 relative covers them;
 - the product: terms are exact in fp32 and their sum carries at most K
   roundings of 2^-24 (of the sum of magnitudes), doubled for accumulators
   that truncate, then one rounding of the output type;
 - the layer: hidden values carry one rounding to 8 bits (2^-9 of each term),
   fp32 sums another 2^-9 of it at these lengths, one rounding of y (2^-9).
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo
from oracle import moe as oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import moe

BF16, F32 = torch.bfloat16, torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


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


def check_packed(q, x64):
    codes, scales = oracle.mx_quantize(x64)
    want_c, want_s = oracle.mx_pack(codes, scales)
    got_s = q.scales.cpu().numpy()
    assert np.array_equal(got_s, want_s)
    got_c = q.codes.cpu().numpy()
    C = codes.shape[1]
    # the codes of a NaN block stand for nothing
    nan = np.repeat(scales == 255, 32, axis=1)
    got = np.stack([got_c & 15, got_c >> 4], 1).reshape(-1, C)
    want = np.stack([want_c & 15, want_c >> 4], 1).reshape(-1, C)
    assert np.array_equal(got[:len(codes)][~nan], want[:len(codes)][~nan])
    assert not got[len(codes):].any()
    return oracle.mx_values(codes, scales)[:, :x64.shape[1]]


# ------------------------------------------------------------------ 4-bit form

SIZES = [(1, 1), (1, 32), (1, 128), (3, 33), (127, 31), (128, 128), (129, 160), (200, 257),
         (5, 1000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, cols", SIZES)
def test_quantize_and_back(rows, cols, dtype):
    x = normal(np.random.default_rng(rows * 1000 + cols), (rows, cols), dtype, 3.0)
    q = moe.quantize(x)
    v = check_packed(q, host(x))
    for out in (BF16, F32):
        assert np.array_equal(host(moe.dequantize(q, out)), v)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, cols", SIZES)
def test_quantize_transposed(rows, cols, dtype):
    x = normal(np.random.default_rng(rows + 7 * cols), (cols, rows), dtype)
    check_packed(moe.quantize(x, transpose=True), host(x).T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("pad, offset", [(8, 0), (1, 0), (0, 1), (5, 3), (8, 4)])
def test_quantize_strides_and_alignment(pad, offset, transpose, dtype):
    x = normal(np.random.default_rng(pad + 10 * offset), (70, 136), dtype)
    v = strided(x, pad, offset)
    want = host(x).T if transpose else host(x)
    check_packed(moe.quantize(v, transpose=transpose), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_gathered_rows(dtype):
    rng = np.random.default_rng(1)
    x = normal(rng, (40, 96), dtype)
    idx = rng.integers(0, 40, 150)
    idx[[0, 7, 149]] = [-1, 40, 2 ** 31 - 1]     # rows that hold no token
    q = moe.quantize(x, row_index=torch.tensor(idx, dtype=torch.int32).cuda())
    want = np.where(((idx >= 0) & (idx < 40))[:, None], host(x)[np.clip(idx, 0, 39)], 0.0)
    check_packed(q, want)


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_batch(transpose):
    x = normal(np.random.default_rng(2), (3, 40, 100), BF16)
    q = moe.quantize(x, transpose=transpose)
    nc, ns = q.codes.numel() // 3, q.scales.numel() // 3
    for b in range(3):
        one = moe.MxTensor(q.codes[b * nc:(b + 1) * nc], q.scales[b * ns:(b + 1) * ns], 1,
                           q.rows, q.cols)
        check_packed(one, host(x[b]).T if transpose else host(x[b]))
    back = moe.dequantize(q, F32)
    assert back.shape == (3, q.rows, q.cols)
    assert torch.equal(back[1], moe.dequantize(one, F32)) == torch.equal(x[1], x[2])


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_special_values(transpose):
    big = float(torch.finfo(F32).max)
    x = torch.zeros((8, 64), dtype=F32)
    x[0, 1] = float("inf")
    x[1, 40] = float("nan")
    x[2, :3] = torch.tensor([big, -big, 1.0])
    x[3, :3] = torch.tensor([2.0 ** -149, -2.0 ** -140, 0.0])
    x[4, :2] = torch.tensor([-0.0, 2.0 ** -127])
    x[5, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])     # ties
    x[6, :8] = -x[5, :8]
    x[7, :4] = torch.tensor([6.0, 6.5, 7.99, -7.0])
    src = (x.t().contiguous() if transpose else x).cuda()
    q = moe.quantize(src, transpose=transpose)
    v = check_packed(q, host(x))
    assert np.array_equal(host(moe.dequantize(q, F32)), v, equal_nan=True)


def test_every_code_and_scale_comes_back():
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 8)          # 256 rows x 128
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)
    c, s = oracle.mx_pack(codes.numpy(), scales)
    q = moe.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), 1, 256, 128)
    want = oracle.mx_values(codes.numpy(), scales)
    with np.errstate(over="ignore"):
        assert np.array_equal(host(moe.dequantize(q, F32)), want.astype(np.float32), equal_nan=True)
    top = want.copy()
    top[np.abs(top) > 2.0 ** 128 * (1 - 2.0 ** -9)] *= np.inf
    assert np.array_equal(host(moe.dequantize(q, BF16)), top, equal_nan=True)


def test_empty_matrices():
    for shape in ((0, 64), (64, 0)):
        q = moe.quantize(torch.zeros(shape, device="cuda"))
        assert q.codes.numel() == 0
        assert moe.dequantize(q).shape == shape


# ------------------------------------------------------------------ the product

def product_case(M, N, K, out, seed, groups=None):
    rng = np.random.default_rng(seed)
    B = 1 if groups is None else len(groups)
    a, b = normal(rng, (M, K), F32), normal(rng, (B, N, K), F32, 0.5)
    qa, qb = moe.quantize(a), moe.quantize(b)
    av = host(moe.dequantize(qa, F32)).reshape(M, K)
    bv = host(moe.dequantize(qb, F32)).reshape(B, N, K)
    return qa, qb, av, bv


def product_close(got, av, bv, out):
    want = av @ bv.T
    K = av.shape[1]
    tol = 2 * K * 2.0 ** -24 * (np.abs(av) @ np.abs(bv).T) + 1e-30
    tol += np.abs(want) * (2.0 ** -8 if out == BF16 else 2.0 ** -23)
    assert (np.abs(host(got) - want) <= tol).all()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M, N, K", [
    (1, 1, 1), (1, 64, 128), (1, 1000, 96), (5, 200, 130), (16, 512, 256), (64, 256, 640),
    (127, 129, 1000), (128, 256, 384), (129, 257, 64), (256, 256, 512), (300, 520, 33),
    (513, 260, 1152), (1000, 96, 2752)])
def test_product(M, N, K, out):
    qa, qb, av, bv = product_case(M, N, K, out, M * 7 + N * 3 + K)
    got = moe.mx_gemm(qa, qb, out_dtype=out)
    product_close(got, av, bv[0], out)
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("M, N, K", [(2048, 4096, 1408), (4096, 1032, 512)])
def test_product_of_many_tiles(M, N, K):
    """More tiles than the GPU holds at once: every tile against the rows of
    the 64-bit product."""
    qa, qb, av, bv = product_case(M, N, K, BF16, 5)
    product_close(moe.mx_gemm(qa, qb), av, bv[0], BF16)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("pad, offset", [(8, 0), (3, 0), (0, 1), (5, 2)])
def test_product_writes_only_its_rows_and_columns(pad, offset, out):
    M, N, K = 70, 133, 160
    qa, qb, av, bv = product_case(M, N, K, out, 11)
    buf = torch.full((M * (N + pad) + offset + 64,), 7.0, dtype=out, device="cuda")
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    moe.mx_gemm(qa, qb, out=view)
    product_close(view, av, bv[0], out)
    view.fill_(7.0)
    assert bool((buf == 7.0).all())


GROUPS = [[5, 0, 128, 1, 129], [0, 0, 0], [300], [0, 0, 17], [1] * 20]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows", GROUPS)
def test_product_per_expert(rows, out):
    first, at = [], 0
    for r in rows:
        first.append(at)
        at += -(-r // 128) * 128 + (128 if r == 17 else 0)   # and a gap between ranges
    M, N, K = max(at, 1), 200, 224
    qa, qb, av, bv = product_case(M, N, K, out, sum(rows), rows)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    d = torch.full((M, N), 7.0, dtype=out, device="cuda")
    if len(rows) == 1:
        qb = moe.MxTensor(qb.codes, qb.scales, 1, N, K)
    moe.mx_gemm(qa, qb, out=d, group_first=dev(first), group_rows=dev(rows))
    used = np.zeros(M, dtype=bool)
    for g, (f, r) in enumerate(zip(first, rows)):
        used[f:f + r] = True
        if r:
            product_close(d[f:f + r], av[f:f + r], bv[g], out)
    assert (host(d)[~used] == 7.0).all()
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows", [[300, 0, 257, 1, 1200, 128], [2000], [513] * 4])
def test_product_per_expert_of_many_tiles(rows, out):
    """More tiles than the GPU has SMs, with ragged ends in both directions."""
    first = [sum(-(-r // 128) * 128 for r in rows[:g]) for g in range(len(rows))]
    M, N, K = first[-1] + -(-rows[-1] // 128) * 128, 1301, 333
    qa, qb, av, bv = product_case(M, N, K, out, sum(rows) + 1, rows)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    d = torch.full((M, N), 7.0, dtype=out, device="cuda")
    if len(rows) == 1:
        qb = moe.MxTensor(qb.codes, qb.scales, 1, N, K)
    moe.mx_gemm(qa, qb, out=d, group_first=dev(first), group_rows=dev(rows))
    used = np.zeros(M, dtype=bool)
    for g, (f, r) in enumerate(zip(first, rows)):
        used[f:f + r] = True
        if r:
            product_close(d[f:f + r], av[f:f + r], bv[g], out)
    assert (host(d)[~used] == 7.0).all()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("pad, offset", [(0, 0), (3, 1), (8, 4)])
def test_product_of_many_ragged_tiles(pad, offset, out):
    M, N, K = 1930, 1301, 333
    qa, qb, av, bv = product_case(M, N, K, out, 12)
    buf = torch.full((M * (N + pad) + offset + 64,), 7.0, dtype=out, device="cuda")
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    moe.mx_gemm(qa, qb, out=view)
    product_close(view, av, bv[0], out)
    view.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("first, rows", [
    ([0, 64], [64, 64]), ([0, -128], [64, 64]), ([0, 128], [64, -1]), ([0, 256], [64, 1]),
    ([0, 128], [64, 2 ** 31 - 1])])
def test_product_leaves_out_bad_groups(first, rows):
    """The first group is in order, the second is not: the first is computed,
    the second left out and reported."""
    M, N, K = 256, 96, 64
    qa, qb, av, bv = product_case(M, N, K, BF16, 1, rows)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    d = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    moe.device_status(clear=True)
    moe.mx_gemm(qa, qb, out=d, group_first=dev(first), group_rows=dev(rows))
    assert moe.device_status(clear=True) == fo.FO_ERR_ARG
    product_close(d[:64], av[:64], bv[0], BF16)
    assert (host(d)[64:] == 7.0).all()


def test_product_without_columns_is_zero():
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    for out in (BF16, F32):
        d = moe.mx_gemm(moe.MxTensor(empty, empty, 1, 5, 0), moe.MxTensor(empty, empty, 1, 9, 0),
                        out_dtype=out)
        assert d.shape == (5, 9) and not d.any()


def test_product_keeps_nan_and_infinity_in_their_row_and_column():
    rng = np.random.default_rng(4)
    a, b = normal(rng, (140, 256), F32), normal(rng, (150, 256), F32)
    a[130, 255] = float("nan")
    b[3, 0] = float("inf")
    d = host(moe.mx_gemm(moe.quantize(a), moe.quantize(b)))
    bad = ~np.isfinite(d)
    want = np.zeros_like(bad)
    want[130, :] = want[:, 3] = True
    assert np.array_equal(bad, want)


def test_product_gradients():
    """dA = dD . B and dB = dD^T . A from transposed conversions, against the
    products of the values those conversions stand for."""
    rng = np.random.default_rng(6)
    M, N, K = 96, 160, 224
    a, b, g = normal(rng, (M, K), BF16), normal(rng, (N, K), BF16), normal(rng, (M, N), BF16)
    values = lambda q: host(moe.dequantize(q, F32))
    ga, bt = moe.quantize(g), moe.quantize(b, transpose=True)
    product_close(moe.mx_gemm(ga, bt), values(ga), values(bt), BF16)
    gt, at = moe.quantize(g, transpose=True), moe.quantize(a, transpose=True)
    product_close(moe.mx_gemm(gt, at), values(gt), values(at), BF16)


def test_product_on_another_stream_and_twice():
    qa, qb, av, bv = product_case(200, 300, 256, F32, 9)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d1 = moe.mx_gemm(qa, qb, out_dtype=F32)
        d2 = moe.mx_gemm(qa, qb, out_dtype=F32)
    s.synchronize()
    product_close(d1, av, bv[0], F32)
    assert torch.equal(d1, d2)


# ------------------------------------------------------------------ the router

def check_route(logits, k, renormalize, capacity=0):
    r = moe.route(logits, k, renormalize, capacity)
    want = oracle.route(host(logits), k, renormalize, capacity)
    for n in ("ids", "row_token", "row_slot", "token_row", "expert_first", "expert_rows"):
        assert np.array_equal(host(getattr(r, n)), want[n]), n
    got = host(r.weights)
    assert np.array_equal(np.isnan(got), np.isnan(want["weights"]))
    ok = ~np.isnan(got)
    assert (np.abs(got - want["weights"])[ok] <= 64 * 2.0 ** -24 * want["weights"][ok]
            + 1e-38).all()
    assert moe.device_status() == fo.FO_OK
    return r, want


ROUTES = [(1, 1, 1), (1, 8, 2), (1, 256, 8), (15, 8, 8), (16, 33, 3), (17, 64, 6), (300, 8, 2),
          (301, 128, 8), (1000, 7, 1), (40, 1024, 32), (2500, 60, 4)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T, E, k", ROUTES)
def test_route(T, E, k, renormalize, dtype):
    x = normal(np.random.default_rng(T + E + k), (T, E), dtype, 2.0)
    check_route(x, k, renormalize)      # (bf16 logits repeat: ties are met)


@pytest.mark.parametrize("capacity", [1, 100, 128, 256])
def test_route_capacity(capacity):
    x = normal(np.random.default_rng(capacity), (900, 8), F32)
    x[:, 2] += 2.0                      # one expert far above its share
    check_route(x, 2, True, capacity)


def test_route_masks_ties_and_not_numbers():
    low, inf, nan = torch.finfo(F32).min, float("inf"), float("nan")
    x = normal(np.random.default_rng(8), (12, 40), F32)
    x[0] = -inf                         # every expert barred
    x[1] = -inf
    x[1, 33] = 0.5                      # fewer left than slots
    x[2] = low                          # the type's lowest value is a logit
    x[3, :39] = low
    x[4] = 0.0                          # all equal
    x[5, 10] = nan
    x[6, 10] = inf
    x[7, [3, 4]] = nan
    x[8] = nan
    x[9, ::2] = -0.0
    x[9, 1::2] = 0.0
    x[10] = -inf
    x[10, 0] = low
    for renormalize in (True, False):
        r, want = check_route(x, 5, renormalize)
    # and a gradient that stays finite where the weights do
    g = torch.ones((12, 5), device="cuda")
    d = host(moe.route_backward(x, r.ids, r.weights, g, renormalize=False))
    for t in (0, 1, 2, 3, 4, 9, 10, 11):
        assert np.isfinite(d[t]).all()
    assert not d[0].any()


def test_route_strides_and_no_tokens():
    x = normal(np.random.default_rng(10), (50, 24), BF16)
    a, _ = check_route(x, 4, True)
    b = moe.route(strided(x, 3, 1), 4, True)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)
    for capacity in (0, 128):
        r = moe.route(x[:0], 4, True, capacity)
        assert not r.expert_rows.any() and bool((r.row_token == -1).all())


def test_route_is_the_same_in_every_run():
    x = normal(np.random.default_rng(12), (5000, 16), BF16)
    a = moe.route(x, 4)
    for _ in range(5):
        b = moe.route(x, 4)
        for n in ("ids", "weights", "row_token", "row_slot", "token_row", "expert_first"):
            assert torch.equal(getattr(a, n), getattr(b, n))


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T, E, k", [(1, 8, 2), (33, 20, 20), (70, 128, 8), (5, 1024, 32)])
def test_route_backward(T, E, k, renormalize):
    rng = np.random.default_rng(T * E)
    x, g = normal(rng, (T, E), F32), normal(rng, (T, k), F32)
    x[0, 1] = float("-inf")
    r = moe.route(x, k, renormalize)
    got = host(moe.route_backward(x, r.ids, r.weights, g, renormalize))
    x64, ids, g64 = host(x), host(r.ids).astype(int), host(g)
    want = oracle.route_backward(x64, ids, g64, renormalize)
    # terms of size |g| * weight, each with the weights' 64 ulp
    tol = 128 * 2.0 ** -24 * np.abs(g64).sum(1, keepdims=True) + 1e-30
    assert (np.abs(got - want) <= tol).all()
    # and against central differences of the weights in 64 bits (h^2 and
    # 1e-16 / h of values around 1)
    f = lambda z: (g64 * oracle.route_weights(z, ids, renormalize)).sum()
    for t, e in [(0, int(ids[0, 0])), (T - 1, E - 1), (T - 1, int(ids[T - 1, 0]))]:
        h = np.zeros_like(x64)
        h[t, e] = 1e-5
        assert abs((f(x64 + h) - f(x64 - h)) / 2e-5 - got[t, e]) <= tol[t] + 1e-7


def test_route_backward_types_and_strides():
    rng = np.random.default_rng(14)
    x, g = normal(rng, (20, 24), BF16), normal(rng, (20, 3), F32)
    r = moe.route(x, 3, False)
    got = host(moe.route_backward(strided(x, 3, 1), r.ids, r.weights, g, False))
    want = oracle.route_backward(host(x), host(r.ids).astype(int), host(g), False)
    tol = np.abs(want) * 2.0 ** -8 + 128 * 2.0 ** -24 * np.abs(host(g)).sum(1, keepdims=True)
    assert (np.abs(got - want) <= tol).all()


def test_route_feeds_the_routing_tables():
    """A routing with a capacity is what fo_plan_route takes: the plan's
    destination counts are those of the oracle's routing."""
    rng = np.random.default_rng(15)
    x = normal(rng, (200, 4), F32)
    r, want = check_route(x, 2, True, 128)
    M, R = 4 * 128, 4
    d = fo.make_desc(M=M, N=256, K=64, swizzle=2, wave_width=4, group_waves=(1,),
                     layout=fo.FO_LAYOUT_A2A_SUBTOKEN, n_dest=R, expert_rows=[128] * 4)
    plan = fo.fo_plan_groups(d)
    try:
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        fo.fo_plan_route(plan, r.row_token.data_ptr(), r.row_slot.data_ptr(), 200, 2,
                         st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        tok = want["row_token"]
        assert fo.fo_plan_table(plan, fo.FO_TAB_DEST_UNITS) == [
            int(((tok >= 0) & (tok % R == k)).sum()) for k in range(R)]
    finally:
        fo.fo_plan_destroy(plan)


# ------------------------------------------------------------------ few tokens

def layer_case(T, H, I, E, seed, weights):
    rng = np.random.default_rng(seed)
    x = normal(rng, (T, H), BF16)
    router = normal(rng, (E, H), BF16, 2 / np.sqrt(H))
    w1, w2 = normal(rng, (E, 2 * I, H), BF16, H ** -0.5), normal(rng, (E, H, I), BF16, I ** -0.5)
    if weights == "bf16":
        return x, router, w1, w2, host(w1), host(w2)
    q1, q2 = moe.quantize(w1), moe.quantize(w2)
    back = lambda q: host(moe.dequantize(q, F32)).reshape(q.batch, q.rows, q.cols)
    return x, router, q1, q2, back(q1), back(q2)


def layer_close(y, want, spread):
    tol = np.abs(want) * 2.0 ** -8 + spread * 2.0 ** -8 + 1e-30
    assert (np.abs(host(y) - want) <= tol).all()
    # and far closer than the bound on the whole: roundings do not line up
    assert np.linalg.norm(host(y) - want) <= 2.0 ** -7 * np.linalg.norm(want) + 1e-30


FEW = [(1, 64, 64, 4, 2), (1, 128, 256, 8, 1), (2, 136, 72, 5, 3), (3, 256, 128, 16, 4),
       (7, 264, 200, 60, 4), (16, 128, 136, 3, 3), (17, 512, 384, 8, 2), (33, 256, 64, 128, 8),
       (64, 384, 192, 4, 2), (64, 136, 520, 2, 2), (5, 2048, 1416, 6, 2), (2, 8, 8, 2, 1)]


@pytest.mark.parametrize("weights", ["bf16", "mx"])
@pytest.mark.parametrize("T, H, I, E, k", FEW)
def test_few(T, H, I, E, k, weights):
    x, router, w1, w2, v1, v2 = layer_case(T, H, I, E, T + H + I, weights)
    for renormalize in (True, False):
        layer = moe.FewTokenLayer(router, w1, w2, k, renormalize=renormalize)
        y = layer(x)
        want, spread = oracle.few(host(x), host(router), v1, v2, k, renormalize)
        layer_close(y, want, spread)
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("weights", ["bf16", "mx"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_few_activations(act, weights):
    x, router, w1, w2, v1, v2 = layer_case(5, 128, 96, 4, 3, weights)
    y = moe.FewTokenLayer(router, w1, w2, 2, act=act)(x)
    layer_close(y, *oracle.few(host(x), host(router), v1, v2, 2, True, act))


@pytest.mark.parametrize("weights", ["bf16", "mx"])
def test_few_one_expert_takes_every_token(weights):
    x, router, w1, w2, v1, v2 = layer_case(64, 128, 128, 8, 4, weights)
    x[:, 0] = 8.0
    router[3, 0] = 8.0                  # a logit far above the others
    layer = moe.FewTokenLayer(router, w1, w2, 1)
    layer_close(layer(x), *oracle.few(host(x), host(router), v1, v2, 1, True))


@pytest.mark.parametrize("weights", ["bf16", "mx"])
def test_few_strides_streams_and_repeats(weights):
    x, router, w1, w2, v1, v2 = layer_case(9, 256, 128, 8, 5, weights)
    layer = moe.FewTokenLayer(router, w1, w2, 2)
    y = layer(x)
    layer_close(y, *oracle.few(host(x), host(router), v1, v2, 2, True))
    wide = strided(x, 8)
    out = torch.full((9, 256 + 3), 7.0, dtype=BF16, device="cuda")
    layer(wide, out=out[:, :256])
    assert torch.equal(out[:, :256], y) and bool((out[:, 256:] == 7.0).all())
    # the same bits in every run, at every token count before it, on a stream
    for n in (1, 9, 4, 9):
        z = layer(x[:n])
    assert torch.equal(z, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = layer(x)
    s.synchronize()
    assert torch.equal(z, y)
    assert layer(x[:0]).shape == (0, 256)


@pytest.mark.parametrize("weights", ["bf16", "mx"])
def test_few_not_numbers_stay_in_their_token(weights):
    x, router, w1, w2, v1, v2 = layer_case(6, 128, 128, 4, 6, weights)
    layer = moe.FewTokenLayer(router, w1, w2, 2)
    clean = layer(x)
    x[2, 5] = float("nan")
    y = layer(x)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[2]).any())


def test_few_barred_experts():
    """A router row of -inf bars its expert; all barred: zeros."""
    x, router, w1, w2, v1, v2 = layer_case(4, 64, 64, 3, 7, "bf16")
    x = x.abs()
    router[0] = float("-inf")
    y = moe.FewTokenLayer(router, w1, w2, 3)(x)
    layer_close(y, *oracle.few(host(x), host(router), v1, v2, 3, True))
    router[:] = float("-inf")
    assert not moe.FewTokenLayer(router, w1, w2, 3)(x).any()


@pytest.mark.parametrize("weights", ["bf16", "mx"])
def test_few_in_a_graph(weights):
    x, router, w1, w2, v1, v2 = layer_case(4, 256, 128, 8, 8, weights)
    layer = moe.FewTokenLayer(router, w1, w2, 2)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x, out=out)               # the workspace exists before the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer(x, out=out)
    x2 = layer_case(4, 256, 128, 8, 9, weights)[0]
    x.copy_(x2)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    layer_close(out, *oracle.few(host(x2), host(router), v1, v2, 2, True))


def test_refusals_of_the_tensor_calls():
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    q = moe.quantize(x)
    bad = [lambda: moe.quantize(x.half()), lambda: moe.quantize(x[0]),
           lambda: moe.quantize(x.t()), lambda: moe.quantize(x.cpu()),
           lambda: moe.quantize(x, row_index=torch.zeros(4, device="cuda")),
           lambda: moe.quantize(x, True, torch.zeros(4, dtype=torch.int32, device="cuda")),
           lambda: moe.dequantize(q, torch.float16),
           lambda: moe.mx_gemm(q, moe.quantize(x[:, :32])),
           lambda: moe.mx_gemm(q, q, out=torch.zeros((4, 5), device="cuda")),
           lambda: moe.mx_gemm(q, q, group_first=torch.zeros(1, dtype=torch.int32,
                                                             device="cuda")),
           lambda: moe.mx_gemm(q, moe.quantize(x.view(2, 2, 64))),
           lambda: moe.MxTensor(q.codes[1:], q.scales, 1, 4, 64),
           lambda: moe.route(x.view(-1), 2), lambda: moe.route(x.half(), 2),
           lambda: moe.route_backward(x, torch.zeros((4, 2), device="cuda"), x, x),
           lambda: moe.FewTokenLayer(x, x, x, 2),
           lambda: moe.FewTokenLayer(x, torch.zeros((4, 16, 64), device="cuda"),
                                     torch.zeros((4, 64, 8), device="cuda"), 2)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fo.FoError):
        moe.route(x, 65)

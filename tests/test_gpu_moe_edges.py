"""The expert layer's operators at the edges of what include/fo.h promises:
sizes between the tested ones, calls that share a device's memory, tokens and
experts that are missing, values at the ends of their types.

Tolerances, derived before the first run:
 - softmax weights: as for the router's other tests, 64 * 2^-24 of the weight;
 - the layer of few tokens: 2^-8 of the value and of the terms' magnitudes (a
   rounding of each hidden value and one of the output, 2^-9 each, doubled);
 - logits of a bf16 product with fp32 sums: H roundings of 2^-24 of the sum of
   magnitudes, doubled;
 - a token of the prompt path: see test_prompt_token_by_token.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo
from oracle import moe as oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import expert_layer, moe

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def host(t):
    return t.detach().double().cpu().numpy()


def normal(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).cuda()


# ------------------------------------------------------------------ workspaces

def few_layer(T, H, I, E, k, seed):
    rng = np.random.default_rng(seed)
    w1, w2 = normal(rng, (E, 2 * I, H), BF16, H ** -0.5), normal(rng, (E, H, I), BF16, I ** -0.5)
    layer = moe.FewTokenLayer(normal(rng, (E, H), BF16, 2 * H ** -0.5), w1, w2, k)
    return layer, normal(rng, (T, H), BF16)


def captured(stream, call):
    """call(), warmed up and captured on the same stream."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
    return g


def test_graphs_outlive_a_larger_call():
    """A larger call on the capture's stream gives that stream's workspaces back;
    what takes their memory neither disturbs a replay nor is disturbed."""
    layer, x = few_layer(4, 256, 128, 8, 2, 31)
    logits = normal(np.random.default_rng(32), (300, 8), F32)
    y, ids = layer(x), moe.route(logits, 2).ids
    s, out, got = torch.cuda.Stream(), torch.empty_like(x), []
    g1 = captured(s, lambda: layer(x, out=out))
    g2 = captured(s, lambda: got.append(moe.route(logits, 2)))
    large, x2 = few_layer(64, 1024, 2048, 8, 4, 33)
    with torch.cuda.stream(s):
        large(x2)
        moe.route(normal(np.random.default_rng(34), (300, 1024), F32), 2)
        taken = [torch.full((1 << n,), 255, dtype=torch.uint8, device="cuda")
                 for n in range(12, 23) for _ in range(4)]
    s.synchronize()
    for _ in range(3):
        out.zero_()
        got[-1].ids.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y) and torch.equal(got[-1].ids, ids)
    assert all(bool((t == 255).all()) for t in taken)
    assert moe.device_status() == fo.FO_OK


def test_a_replay_beside_eager_calls():
    """A graph replayed on one stream while the stream that it was captured on
    goes on with calls of its own."""
    layer, x = few_layer(5, 512, 256, 8, 2, 35)
    y = layer(x)
    s, r, out = torch.cuda.Stream(), torch.cuda.Stream(), torch.empty_like(x)
    g = captured(s, lambda: layer(x, out=out))
    torch.cuda.synchronize()
    wrong = torch.zeros(2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(r):
            g.replay()
            wrong[0] += (out != y).sum()
        with torch.cuda.stream(s):
            wrong[1] += (layer(x) != y).sum()
    torch.cuda.synchronize()
    assert wrong.tolist() == [0, 0]
    assert moe.device_status() == fo.FO_OK


def test_a_workspace_is_fresh_after_an_error_is_cleared():
    """Counters of joined output rows as a wait that ran out may leave them, and
    its status, set from here: the next call has a workspace without them."""
    layer, x = few_layer(9, 512, 640, 8, 2, 36)
    y = layer(x)
    dev = x.device
    key = ("few", dev, torch.cuda.current_stream().cuda_stream)
    moe._workspaces[key][256:512] = 1
    moe._status[dev].fill_(fo.FO_ERR_TIMEOUT)
    assert moe.device_status(clear=True) == fo.FO_ERR_TIMEOUT
    assert torch.equal(layer(x), y)
    assert moe.device_status() == fo.FO_OK


# ------------------------------------------------------------------ the router's sizes

def routed(logits, k):
    """The router's outputs for finite logits (float64), all tokens at once."""
    T, E = logits.shape
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(logits, 1).gather(1, ids)
    flat = ids.reshape(-1)
    i = torch.arange(T * k, device=flat.device)
    order = torch.sort(flat, stable=True).indices
    rows = torch.bincount(flat, minlength=E)
    span = (rows + 127) // 128 * 128
    first = span.cumsum(0) - span
    at = torch.empty_like(i)
    at[order] = first[flat[order]] + i - (rows.cumsum(0) - rows)[flat[order]]
    M = (T * k + E * 127) // 128 * 128
    row_token, row_slot = at.new_full((M,), -1), at.new_zeros(M)
    row_token[at], row_slot[at] = i // k, i % k
    return dict(ids=ids, weights=w / w.sum(1, keepdim=True), row_token=row_token,
                row_slot=row_slot, token_row=at.view(T, k), expert_first=first,
                expert_rows=rows)


def check_routed(T, E, k, dtype=F32):
    x = normal(np.random.default_rng(T + E + k), (T, E), dtype, 2.0)
    r, want = moe.route(x, k), routed(x.double(), k)
    for n in ("ids", "row_token", "row_slot", "token_row", "expert_first", "expert_rows"):
        assert torch.equal(getattr(r, n).long(), want[n]), n
    off = (r.weights.double() - want["weights"]).abs()
    assert bool((off <= 64 * 2.0 ** -24 * want["weights"] + 1e-38).all())
    assert moe.device_status() == fo.FO_OK


# per expert and token of a block the kernel takes shared memory: sizes whose
# part that the launch asks for is below 48 KB, and the sum above
BETWEEN = [(5, 600, 8), (3, 715, 8), (24000, 512, 10), (90000, 384, 8), (120000, 256, 8)]


@pytest.mark.parametrize("T, E, k", BETWEEN)
def test_route_as_a_process_first_call(T, E, k):
    """(An earlier, larger call would leave the kernel with more shared memory.)"""
    code = f"import test_gpu_moe_edges as t; t.check_routed({T}, {E}, {k})"
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_route_from_two_threads():
    """Calls of different sizes of one kernel, each from a thread and on a stream
    of its own."""
    failed = []

    def calls(T, E, k):
        try:
            x = normal(np.random.default_rng(E), (T, E), F32)
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.cuda.synchronize()
                for _ in range(300):
                    moe.route(x, k)
                torch.cuda.synchronize()
        except Exception as e:      # noqa: BLE001 (reported by the test)
            failed.append(e)

    threads = [threading.Thread(target=calls, args=a) for a in ((20, 1024, 32), (20, 730, 8))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, E, k", [(200, 300, 10), (33, 600, 8), (500, 512, 10), (100, 1000, 32),
                                     (300, 40, 32), (1, 1024, 1)])
def test_route_of_many_experts(T, E, k, dtype):
    check_routed(T, E, k, dtype)


@pytest.mark.parametrize("T, E, k", [(250000, 32, 32), (170000, 1024, 32)])
def test_route_of_more_tokens_than_shared_memory_holds(T, E, k):
    check_routed(T, E, k)


# ------------------------------------------------------------------ the layer

def layer_of(router, H, I, E, k, rng):
    w1, w2 = normal(rng, (E, 2 * I, H), BF16, H ** -0.5), normal(rng, (E, H, I), BF16, I ** -0.5)
    return expert_layer.ExpertLayer(router, moe.quantize(w1), moe.quantize(w2), k,
                                    w1_t=moe.quantize(w1, transpose=True))


def test_prompt_and_generation_choose_the_same_experts():
    """Experts 2j and 2j + 1 have logits 2^-8 apart, less than a bf16 step of
    most: all tokens choose the odd one, in a prompt and one at a time."""
    rng = np.random.default_rng(21)
    T, H, I, E = 70, 256, 64, 8
    x = normal(rng, (T, H), BF16)
    x[:, 0] = 1.0
    router = normal(rng, (E, H), BF16, 4 / np.sqrt(H))
    router[1::2] = router[::2]
    router[::2, 0], router[1::2, 0] = 0.0, 2.0 ** -8
    layer = layer_of(router, H, I, E, 1, rng)
    y, step = layer.forward(x)
    logits = host(x) @ host(router).T
    size = np.abs(host(x)) @ np.abs(host(router)).T
    assert (np.abs(host(step.logits) - logits) <= 2 * H * 2.0 ** -24 * size).all()
    want = oracle.route(logits, 1, True)["ids"]
    assert (want % 2 == 1).all() and np.array_equal(host(step.routing.ids), want)
    # two experts' outputs are as far apart as they are large; one's in 4 bits
    # (a prompt's activations) and in 16 about a fifth of that
    few = host(torch.cat([layer(x[t:t + 1]) for t in range(T)]))
    off = np.linalg.norm(host(y) - few, axis=1)
    assert (off <= np.linalg.norm(few, axis=1) / 2).all()


@pytest.mark.parametrize("T, H, I, E, k", [(70, 256, 192, 4, 2), (130, 136, 264, 6, 3)])
def test_prompt_token_by_token(T, H, I, E, k):
    """A prompt against the definition with its 4-bit roundings, each token by
    itself, the experts chosen from 64-bit logits.  A hidden value carries bf16
    roundings (2^-7 of it in all) that the oracle's does not, so one in twenty
    takes the neighbouring code and moves by half its size at most.  Of a token's
    I >= 192 values under each expert that is up to 1/20 + 5 sqrt(1/20 / I) = 0.13
    of them: sqrt(0.13) / 2 = 0.18 of the norm; 1/4 covers it with the sum over
    experts.  (A wrong weight or row moves a token by its own norm.)"""
    layer = expert_layer.ExpertLayer.random(H, I, E, k, seed=T)
    x = normal(np.random.default_rng(T), (T, H), BF16)
    y = host(layer.forward(x)[0])
    values = lambda q: host(moe.dequantize(q, F32)).reshape(q.batch, q.rows, q.cols)
    rounded = lambda v: oracle.mx_values(*oracle.mx_quantize(v))[:, :v.shape[1]]
    w1, w2, xq = values(layer.w1), values(layer.w2), rounded(host(x))
    r = oracle.route(host(x) @ host(layer.router).T, k, True)
    for t in range(T):
        exact = np.zeros(H)
        for e, w in zip(r["ids"][t], r["weights"][t]):
            g, u = np.split(w1[e] @ xq[t], 2)
            exact += w * (w2[e] @ rounded((g / (1 + np.exp(-g)) * u)[None])[0])
        assert np.linalg.norm(y[t] - exact) <= np.linalg.norm(exact) / 4, t


def test_slots_without_a_row_read_none():
    """One expert is barred, and a NaN stands in the first row of the tables:
    nothing of it reaches the slots that have no row."""
    rng = np.random.default_rng(22)
    T, H, I, E = 70, 64, 64, 3
    x = normal(rng, (T, H), BF16).abs()
    router = normal(rng, (E, H), BF16, H ** -0.5)
    router[1] = float("-inf")
    layer = layer_of(router, H, I, E, 3, rng)
    clean, step = layer.forward(x)
    assert bool((step.routing.token_row == -1).any(1).all())
    rows = step.routing.row_token.numel()
    dup = normal(rng, (rows, 2 * I), BF16)
    g = normal(rng, (T, 3), F32)
    _, dx = layer.backward(step, g, dup)
    first = int(step.routing.row_token[0])
    others = [t for t in range(T) if t != first]
    bad = x.clone()
    bad[first] = float("nan")
    y, _ = layer.forward(bad)
    assert bool(y[others].isfinite().all()) and torch.equal(y[others], clean[others])
    dup[0] = float("nan")
    _, dx_bad = layer.backward(step, g, dup)
    assert torch.equal(dx_bad[others], dx[others])
    assert bool(torch.isnan(dx_bad[first]).all())


def test_prompt_of_barred_tokens_is_zero():
    rng = np.random.default_rng(23)
    router = torch.full((3, 64), float("-inf"), dtype=BF16, device="cuda")
    layer = layer_of(router, 64, 64, 3, 2, rng)
    y, _ = layer.forward(normal(rng, (70, 64), BF16).abs())
    assert not y.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gathered_rows_of_a_matrix_without_rows(dtype):
    idx = torch.tensor([-1, 0, 5], dtype=torch.int32, device="cuda")
    q = moe.quantize(torch.empty((0, 96), dtype=dtype, device="cuda"), row_index=idx)
    assert (q.rows, q.cols) == (3, 96) and not moe.dequantize(q).any()


@pytest.mark.parametrize("E", [1, 4])
def test_prompt_without_tokens(E):
    layer = expert_layer.ExpertLayer.random(64, 64, E, 1)
    y, step = layer.forward(torch.empty((0, 64), dtype=BF16, device="cuda"))
    assert y.shape == (0, 64)
    rows = step.routing.row_token.numel()
    dlogits, dx = layer.backward(step, torch.empty((0, 1), device="cuda"),
                                 torch.empty((rows, 128), dtype=BF16, device="cuda"))
    assert dlogits.shape == (0, E) and dx.shape == (0, 64)


@pytest.mark.parametrize("K", [0, 64])
def test_product_over_no_experts(K):
    """A product per expert with no expert at all: every row keeps what it holds."""
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    bytes_ = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    a = moe.MxTensor(*map(bytes_, fo.fo_mx_sizes(1, 5, K)), 1, 5, K)
    b = moe.MxTensor(bytes_(0), bytes_(0), 0, 9, K)
    d = torch.full((5, 9), 7.0, dtype=F32, device="cuda")
    assert moe.mx_gemm(a, b, out=d, group_first=none, group_rows=none) is d
    assert bool((d == 7.0).all())


def test_backward_refuses_gradients_of_other_tables():
    """(The routing's rows index the product of `dup`.)"""
    layer = expert_layer.ExpertLayer.random(64, 64, 3, 2)
    _, step = layer.forward(normal(np.random.default_rng(24), (70, 64), BF16))
    rows, g = step.routing.row_token.numel(), torch.zeros((70, 2), device="cuda")
    for n in (0, rows - 128, rows + 128):
        with pytest.raises(ValueError):
            layer.backward(step, g, torch.zeros((n, 128), dtype=BF16, device="cuda"))
    layer.backward(step, g, torch.zeros((rows, 128), dtype=BF16, device="cuda"))


@pytest.mark.parametrize("form", ["bf16", "mx"])
@pytest.mark.parametrize("gate", [-88.0, -87.5, -60.0, -0.0078125, 30.0])
def test_silu_far_from_zero(gate, form):
    """silu(g) = g e^g is small but not zero at -88, where 1 + e^-g nears the
    largest fp32 value; a large second factor brings it back."""
    H, E = 64, 1
    x = torch.zeros((1, H), dtype=BF16, device="cuda")
    x[0, 0] = abs(gate) / 64
    w1 = torch.zeros((E, 2 * H, H), dtype=BF16, device="cuda")
    w1[:, :H, 0] = 64.0 * np.sign(gate)
    w1[:, H:, 0] = 2.0 ** 100
    w2 = torch.eye(H, dtype=BF16, device="cuda")[None]
    router = torch.zeros((E, H), dtype=BF16, device="cuda")
    args = (host(x), host(router), host(w1), host(w2))
    if form == "mx":
        w1, w2 = moe.quantize(w1), moe.quantize(w2)
    y = host(moe.FewTokenLayer(router, w1, w2, 1)(x))
    want, spread = oracle.few(*args, 1, True)
    assert (np.abs(y - want) <= (np.abs(want) + spread) * 2.0 ** -8).all() and want.all()


@pytest.mark.parametrize("which", ["x", "router", "w1", "w2"])
def test_few_refuses_tensors_that_require_a_gradient(which):
    rng = np.random.default_rng(37)
    t = dict(x=normal(rng, (3, 64), BF16), router=normal(rng, (4, 64), BF16, 0.1),
             w1=normal(rng, (4, 64, 64), BF16, 0.1), w2=normal(rng, (4, 64, 32), BF16, 0.1))
    y = moe.FewTokenLayer(t["router"], t["w1"], t["w2"], 2)(t["x"])
    t[which].requires_grad_()
    layer = moe.FewTokenLayer(t["router"], t["w1"], t["w2"], 2)
    with pytest.raises(ValueError, match="gradient"):
        layer(t["x"])
    with torch.no_grad():
        assert torch.equal(layer(t["x"]), y)


def test_prompt_refuses_tensors_that_require_a_gradient():
    layer = expert_layer.ExpertLayer.random(64, 64, 3, 2)
    x = normal(np.random.default_rng(38), (70, 64), BF16)
    y = layer(x)
    layer.router.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        layer(x)
    with torch.no_grad():
        assert torch.equal(layer(x), y)


def test_an_error_on_another_stream_is_kept(monkeypatch):
    """The device's first call runs behind other work on its stream, an erring call
    at once on a second: the first's zeroing of the status does not undo it."""
    monkeypatch.setattr(moe, "_status", {})
    q = moe.quantize(torch.ones((128, 64), dtype=BF16, device="cuda"))
    first, rows = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (64, 1))
    d = torch.zeros((128, 128), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
        moe.mx_gemm(q, q)
    with torch.cuda.stream(r):
        moe.mx_gemm(q, q, out=d, group_first=first, group_rows=rows)
    assert moe.device_status(clear=True) == fo.FO_ERR_ARG
    assert moe.device_status() == fo.FO_OK

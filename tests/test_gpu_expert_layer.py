"""The expert layer's operators together, as ExpertLayer runs them, and their
offsets past 32 bits.

Tolerances, derived before the first run:
 - the prompt path quantizes the hidden values, which carry roundings of 2^-9
   in the gate, in the other factor and in the activation's argument (under
   2^-7 of the value together).  The oracle's chain has none of them, so a value
   that lies that near to a boundary between two codes may take the other: the
   boundaries are at least a third of a value apart, hence about one value in
   twenty, and each moves by half its size at most.  sqrt(1/20) / 2 is 0.11 of
   the norm; 1/8 covers it with the other roundings.  (A row at a wrong place
   or a wrong weight moves a token by its own norm.)
 - the logits' gradient: one rounding to their bf16 (2^-9 of it, doubled) and
   2^-18 of the weighted sum of magnitudes for fp32 weights and sums.
 - the gradient's product: as for the product alone, 2 K 2^-24 of the sum of
   magnitudes, and top_k roundings of the sum over a token's rows.
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo
from oracle import moe as oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import expert_layer, moe

BF16, F32 = torch.bfloat16, torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


def values(q):
    return host(moe.dequantize(q, F32)).reshape(q.batch, q.rows, q.cols)


def rounded(x64):
    return oracle.mx_values(*oracle.mx_quantize(x64))[:, :x64.shape[1]]


@pytest.mark.parametrize("T, H, I, E, k", [(70, 256, 192, 4, 2), (130, 136, 72, 6, 3)])
def test_prompt(T, H, I, E, k):
    layer = expert_layer.ExpertLayer.random(H, I, E, k, seed=T)
    x = torch.from_numpy(np.random.default_rng(T).standard_normal((T, H))).to(BF16).cuda()
    y, step = layer.forward(x)
    assert torch.equal(layer(x), y)
    w1, w2, xq = values(layer.w1), values(layer.w2), rounded(host(x))
    ids = step.routing.ids.cpu().numpy()
    want = oracle.route(host(step.logits), k, True)
    assert np.array_equal(ids, want["ids"])
    exact = np.zeros((T, H))
    for t in range(T):
        for s in range(k):
            e = ids[t, s]
            g, u = np.split(w1[e] @ xq[t], 2)
            h = rounded((g / (1 + np.exp(-g)) * u)[None])[0]
            exact[t] += want["weights"][t, s] * (w2[e] @ h)
    off = np.linalg.norm(host(y) - exact, axis=1)
    assert np.linalg.norm(off) <= np.linalg.norm(exact) / 8
    assert moe.device_status() == fo.FO_OK


@pytest.mark.parametrize("T, H, I, E, k", [(70, 256, 192, 4, 2), (130, 136, 72, 6, 3)])
def test_backward(T, H, I, E, k):
    layer = expert_layer.ExpertLayer.random(H, I, E, k, seed=T)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    _, step = layer.forward(x)
    r = step.routing
    g = torch.from_numpy(rng.standard_normal((T, k))).to(F32).cuda()
    rows = r.row_token.numel()
    dup = torch.from_numpy(rng.standard_normal((rows, 2 * I))).to(BF16).cuda()
    dlogits, dx = layer.backward(step, g, dup)
    want = oracle.route_backward(host(step.logits), r.ids.cpu().numpy(), host(g), True)
    mag = (host(r.weights) * np.abs(host(g))).sum(1, keepdims=True)
    assert (np.abs(host(dlogits) - want) <= np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -18).all()
    w1t, d = values(layer.w1_t), rounded(host(dup))
    ids, at = r.ids.cpu().numpy(), r.token_row.cpu().numpy()
    for t in range(T):
        exact, size = np.zeros(H), np.zeros(H)
        for s in range(k):
            m = w1t[ids[t, s]]
            exact += m @ d[at[t, s]]
            size += np.abs(m) @ np.abs(d[at[t, s]])
        tol = size * (2 * 2 * I + k) * 2.0 ** -24
        assert (np.abs(host(dx[t]) - exact) <= tol).all()


def test_generation_is_the_layer_of_few_tokens():
    layer = expert_layer.ExpertLayer.random(256, 192, 4, 2, seed=3)
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((5, 256))).to(BF16).cuda()
    want, spread = oracle.few(host(x), host(layer.router), values(layer.w1), values(layer.w2), 2,
                              True)
    assert (np.abs(host(layer(x)) - want) <= (np.abs(want) + spread) * 2.0 ** -8 + 1e-30).all()


def test_command(capsys):
    expert_layer.main("--hidden 256 --inter 384 --experts 4 --top_k 2 --tokens 300".split())
    out = capsys.readouterr().out
    assert "prompt of 300 tokens" in out and "from a graph" in out
    with pytest.raises(ValueError):
        layer = expert_layer.ExpertLayer.random(64, 64, 2, 1)
        layer.w1_t = None
        layer.backward(None, None, None)


# ------------------------------------------------------------------ long strides

FAR = 2 ** 31 + 24      # elements from row to row


def far(rows, cols, dtype):
    buf = torch.empty((rows - 1) * FAR + cols, dtype=dtype, device="cuda")
    return buf.as_strided((rows, cols), (FAR, 1))


def test_rows_past_32_bits():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((4, 200))).to(BF16).cuda()
    v = far(4, 200, BF16)
    v.copy_(x)
    a, b = moe.quantize(x), moe.quantize(v)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    idx = torch.tensor([3, 1, -1], dtype=torch.int32, device="cuda")
    a, b = moe.quantize(x, row_index=idx), moe.quantize(v, row_index=idx)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    a, b = moe.quantize(x, True), moe.quantize(v, True)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    q = moe.quantize(x)
    v.fill_(0)
    moe.mx_gemm(q, moe.quantize(torch.eye(200, device="cuda")), out=v)
    assert torch.equal(v, moe.dequantize(q, BF16))
    logits = far(3, 16, F32)
    logits.copy_(x[:3, :16])
    assert torch.equal(moe.route(logits, 2).ids, moe.route(x[:3, :16].float(), 2).ids)


@pytest.mark.parametrize("form", ["bf16", "mx"])
def test_few_tokens_past_32_bits(form):
    rng = np.random.default_rng(2)
    put = lambda *s: torch.from_numpy(rng.standard_normal(s) / 8).to(BF16).cuda()
    router, w1, w2, x = put(4, 64), put(4, 64, 64), put(4, 64, 32), put(3, 64)
    if form == "mx":
        w1, w2 = moe.quantize(w1), moe.quantize(w2)
    layer = moe.FewTokenLayer(router, w1, w2, 2)
    v, y = far(3, 64, BF16), far(3, 64, BF16)
    v.copy_(x)
    layer(v, out=y)
    assert torch.equal(y, layer(x))

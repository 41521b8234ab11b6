"""A model's block with an expert layer: its operators in a run, forward and back.

Tolerances, derived before the first run:
 - what passes no 4-bit conversion between the inputs given here and the result is
   off by roundings of bf16 alone: the norms' inputs, outputs and gradients (2^-9
   each, at most eight of them in a row) stay within 2^-6 of their norm;
 - a conversion to 4 bits moves normal data by 0.11 of its norm (the oracle's, on
   10^5 draws).  From the block's input to its expert rows there are two, from the
   rows' gradient to the norm's output two more, and the activations that the
   gradient is taken at carry those of the first: five in the longest chain, which
   add up as squares: 0.11 sqrt(5) is 0.25.  2/5 leaves room for sizes this small.
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import block as ops
    from communication_overlap_gb300 import expert_layer, moe

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

ROUTINGS = [
    dict(),
    dict(scoring="sigmoid", scale=2.5),
    dict(scoring="sigmoid", groups=2, top_groups=1, group_top=2, scale=1.5),
    dict(scoring="softmax", groups=3, top_groups=2),
]


def near(got, want, part):
    off = (got.double() - want).norm() / want.norm()
    assert off <= part, off


def exact(block, stream, ids, dstream):
    """The block in 64 bits with the values of its 4-bit weights and the experts that
    it chose, and its gradients by autograd."""
    layer = block.layer
    values = lambda q: moe.dequantize(q, F32).double()
    w1, w2 = values(layer.w1), values(layer.w2)
    leaf = lambda t: None if t is None else t.double().requires_grad_()
    p = dict(stream=leaf(stream), router=leaf(layer.router), pre_gain=leaf(block.pre_gain),
             post_gain=leaf(block.post_gain), gate=leaf(block.gate))
    norm = lambda v, g: v / torch.sqrt((v ** 2).mean(1, keepdim=True) + block.eps) * g
    n = norm(p["stream"], p["pre_gain"])
    logits = n @ p["router"].t()
    how = block.routing
    s = torch.sigmoid(logits) if how.get("scoring") == "sigmoid" else torch.softmax(logits, 1)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * how.get("scale", 1.0)
    z = []
    for t in range(len(n)):
        y = 0
        for k, e in enumerate(ids[t].tolist()):
            gate, up = (w1[e] @ n[t]).chunk(2)
            y = y + w[t, k] * (w2[e] @ (torch.nn.functional.silu(gate) * up))
        z.append(y)
    z = torch.stack(z)
    u = z if p["post_gain"] is None else norm(z, p["post_gain"])
    out = p["stream"] + block.scale * (u if p["gate"] is None else p["gate"] * u)
    names = [k for k, v in p.items() if v is not None]
    grads = torch.autograd.grad(out, [p[k] for k in names], dstream.double())
    return out.detach(), dict(zip(names, grads))


@pytest.mark.parametrize("routing", ROUTINGS)
@pytest.mark.parametrize("T, H, I, E, k", [(70, 256, 192, 6, 2), (130, 136, 72, 12, 3)])
def test_block(T, H, I, E, k, routing):
    if "groups" in routing:
        routing = dict(routing, bias=torch.linspace(-0.01, 0.01, E, device="cuda"))
    block = expert_layer.ExpertBlock.random(H, I, E, k, seed=T, scale=0.75, routing=routing)
    rng = np.random.default_rng(T)
    draw = lambda: torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    stream, dstream = draw(), draw()
    out, step = block.forward(stream)
    assert torch.equal(block(stream), out)
    grads = block.backward(step, dstream)
    ids = step.routing.ids.long()
    assert (ids >= 0).all()
    want, dwant = exact(block, stream, ids, dstream)
    near(out, want, 0.4 * float((want - stream.double()).norm() / want.norm()) + 2.0 ** -6)
    assert grads.router.dtype == F32 and grads.stream.dtype == BF16
    for name in ("stream", "router", "pre_gain", "post_gain", "gate"):
        near(getattr(grads, name), dwant[name], 0.4)
    # the norms' own parts, from the block's own values
    u = step.mixed.double()
    u = u / torch.sqrt((u ** 2).mean(1, keepdim=True) + block.eps)
    u = u * block.scale
    near(grads.gate, (dstream.double() * u * block.post_gain.double()).sum(0), 2.0 ** -6)
    near(grads.post_gain, (dstream.double() * u * block.gate.double()).sum(0), 2.0 ** -6)
    near(out, stream.double() + block.gate.double() * block.post_gain.double() * u, 2.0 ** -6)
    assert moe.device_status() == fo.FO_OK


def test_block_of_few_tokens():
    """The one-kernel layer between the norms, and the same tokens in a prompt."""
    block = expert_layer.ExpertBlock.random(256, 192, 6, 2, seed=3)
    rng = np.random.default_rng(3)
    stream = torch.from_numpy(rng.standard_normal((80, 256))).to(BF16).cuda()
    few, many = block(stream[:7]), block(stream)[:7]
    moved = (many.double() - stream[:7].double()).norm()
    assert (few.double() - many.double()).norm() <= 0.4 * moved
    plain = expert_layer.ExpertBlock(block.layer, block.pre_gain)
    n = ops.norm(stream[:7], pre_gain=block.pre_gain, eps=plain.eps)
    want = stream[:7].double() + block.layer.few(n.y).double()
    near(plain(stream[:7]), want, 2.0 ** -8)
    with pytest.raises(ValueError, match="w2_t"):
        plain.backward(plain.forward(stream)[1], stream)


def test_gradient_captured():
    """A whole forward and backward pass from a graph, on what its inputs hold then."""
    block = expert_layer.ExpertBlock.random(
        136, 72, 12, 3, seed=5, routing=dict(scoring="sigmoid", groups=3, top_groups=2, group_top=2))
    rng = np.random.default_rng(5)
    draw = lambda: torch.from_numpy(rng.standard_normal((90, 136))).to(BF16).cuda()
    inputs = [(draw(), draw()) for _ in range(2)]

    def run(stream, dstream):
        out, step = block.forward(stream)
        g = block.backward(step, dstream)
        return [out, g.stream, g.router, g.pre_gain, g.post_gain, g.gate]

    want = [run(*i) for i in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    live = [t.clone() for t in inputs[0]]
    with torch.cuda.stream(side):
        run(*live)              # (the products' library warms up outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*live)
    for i in (1, 0, 1):
        for to, of in zip(live, inputs[i]):
            to.copy_(of)
        graph.replay()
        beside = run(*inputs[0])
        torch.cuda.synchronize()
        # (rows of no expert hold anything: the results that do not see them are equal)
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(beside, want[0]))


EXACT = [
    (True, dict(scoring="sigmoid", scale=2.0)),
    (False, dict(scoring="sigmoid", scale=2.0)),
    (True, dict(scale=2.0)),
    (False, dict(scale=2.0)),
    (True, dict(scoring="sigmoid", scale=2.0, groups=4, top_groups=1, group_top=2)),
    (False, dict(scoring="softmax", scale=2.0, groups=4, top_groups=1, group_top=1)),
]


@pytest.mark.parametrize("renormalize, routing", EXACT)
@pytest.mark.parametrize("T", [65, 300])
def test_block_of_values_that_4_bits_hold(T, renormalize, routing):
    """The whole chain without a rounding to 4 bits, so that each result is off by bf16's
    roundings alone, element by element.

    The stream is -1 and 1 (1 in its first 32 columns), so are its norm and its product with
    pre_gain; a row of w1 has one value, 16 in a column of ones for a gate (silu is the gate
    itself there, to 2^-23) and 1 or 2 for the others; w2 is a permutation with signs for
    each expert; both chosen experts have the logit 0, and weights of 2 / 2; the gradient of
    the stream is 1, 1.5, 2 or 3.  So every block of 32 that is converted holds multiples by
    a power of two of 0.5, 1, 1.5, 2, 3, 4 and 6, the values of 4 bits, and 8-bit codes
    hold them too.  Roundings to bf16, 2^-9 each: of the product with w1_t, of its rows'
    sum, of the logits' gradient, of their sum, and of the result: five, below 2^-6
    of the magnitudes that were added.  The gradients of router and gate see one and two."""
    H, I, E, k = 64, 64, 8, 2
    rng = np.random.default_rng(T)
    sign = lambda *shape: rng.choice([-1.0, 1.0], shape)
    stream, pre = sign(T, H), sign(H)
    stream[:, :32], pre[:42] = 1, 1
    w1, w2 = np.zeros((E, 2 * I, H)), np.zeros((E, H, I))
    for e in range(E):
        w1[e, np.arange(I), np.arange(I) % 32] = 16
        w1[e, I + np.arange(I), rng.integers(0, H, I)] = sign(I) * rng.choice([1, 2], I)
        w2[e, rng.permutation(H), np.arange(I)] = sign(I) / 16
    # two experts per pair of signs of columns 40 and 41: theirs have the logit 0
    router = np.zeros((E, H))
    for e in range(E):
        router[e, 0], router[e, 40], router[e, 41] = -64, 32 * (-1) ** (e // 2), 32 * (-1) ** (e // 4)
    gate, scale = sign(H), 0.5
    dstream = sign(T, H) * rng.choice([1, 1.5, 2, 3], (T, H))
    put = lambda a: torch.from_numpy(a).to(BF16).cuda()
    kept = [(moe.quantize(put(w)), moe.quantize(put(w), transpose=True)) for w in (w1, w2)]
    for w, (q, _) in zip((w1, w2), kept):
        assert torch.equal(moe.dequantize(q), put(w))
    layer = expert_layer.ExpertLayer(put(router), kept[0][0], kept[1][0], k, renormalize,
                                     w1_t=kept[0][1])
    block = expert_layer.ExpertBlock(layer, put(pre), None, put(gate), scale, w2_t=kept[1][1],
                                     routing=routing)
    out, step = block.forward(put(stream))
    grads = block.backward(step, put(dstream))
    # the definitions in 64 bits
    n = stream * pre / np.sqrt(1 + block.eps)
    logits = n @ router.T
    ids = step.routing.ids.cpu().numpy()
    pair = 2 * (stream[:, 41] < 0) + (stream[:, 40] < 0)
    assert np.array_equal(np.sort(ids, 1), np.stack([2 * pair, 2 * pair + 1], 1))
    every = np.arange(T)[:, None]
    if routing.get("scoring") == "sigmoid":
        s = 1 / (1 + np.exp(-logits))
        slope = lambda ds: ds * s * (1 - s)
    else:
        s = np.exp(logits) / np.exp(logits).sum(1, keepdims=True)
        slope = lambda ds: s * (ds - (s * ds).sum(1, keepdims=True))
    chosen = s[every, ids]
    total = chosen.sum(1, keepdims=True)
    w = 2 * chosen / (total if renormalize else 1)
    up = np.einsum("tsih,th->tsi", w1[ids], n)
    g, v = up[..., :I], up[..., I:]
    act = g / (1 + np.exp(-g))
    rows = np.einsum("tshi,tsi->tsh", w2[ids], act * v)
    z = (w[..., None] * rows).sum(1)
    host = lambda t: t.double().cpu().numpy()

    def near(got, want, part, size):
        off = np.abs(host(got) - want)
        assert (off <= part * size).all(), (off / size).max()

    near(step.mixed, z, 2.0 ** -8, np.abs(z))
    near(out, stream + scale * gate * z, 2.0 ** -8, np.abs(stream) + np.abs(scale * z))
    values = host(step.kept.values()).reshape(-1, 2 * I)
    held = step.routing.token_row.long().cpu().numpy()
    assert np.array_equal(values[held], np.einsum("tsih,th->tsi", w1[ids], stream * pre))
    dz = scale * gate * dstream
    dw = (dz[:, None] * rows).sum(2)
    dh = np.einsum("tshi,tsh->tsi", w2[ids], w[..., None] * dz[:, None])
    sg = 1 / (1 + np.exp(-g))
    dup = np.concatenate([dh * v * sg * (1 + g * (1 - sg)), dh * act], 2)
    dn = np.einsum("tsih,tsi->tsh", w1[ids], dup)
    ds = np.zeros((T, E))
    ds[every, ids] = 2 * (dw / total - (dw * chosen).sum(1, keepdims=True) / total ** 2
                          if renormalize else dw)
    dl = slope(ds)
    near(grads.router, dl.T @ n, 2.0 ** -8, np.abs(dl).T @ np.abs(n) + 2.0 ** -20 * np.abs(dw).max())
    sn = stream / np.sqrt(1 + block.eps)
    sum_n = dn.sum(1) + dl @ router
    size = np.abs(dn).sum(1) + np.abs(dl) @ np.abs(router)
    near(grads.pre_gain, (sum_n * sn).sum(0), 2.0 ** -6, size.sum(0))
    near(grads.gate, (scale * z * dstream).sum(0), 2.0 ** -8, np.abs(scale * z * dstream).sum(0))
    e = sum_n * pre
    want = dstream + (e - sn * (e * sn).mean(1, keepdims=True)) / np.sqrt(1 + block.eps)
    bound = np.abs(dstream) + size + size.mean(1, keepdims=True)
    near(grads.stream, want, 2.0 ** -6, bound)
    # a third of the experts' part would not pass, in most of the elements that have one
    part = np.abs(dn.sum(1))
    assert (part / 3 > 2.0 ** -6 * bound)[part > 0].mean() > 0.5
    assert moe.device_status() == fo.FO_OK

"""The expert layer's operators at the edges of what include/fo.h promises:
sizes between the tested ones, calls that share a device's memory, tokens and
experts that are missing, values at the ends of their types.
"""
import numpy as np
import pytest
import torch

from communication_overlap_gb300 import fo

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from communication_overlap_gb300 import moe

BF16, F32 = torch.bfloat16, torch.float32


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

"""An expert layer made of the operators of ``moe.py``, as a model runs it.

  layer = ExpertLayer.random(hidden, inter, experts, top_k)
  y = layer(x)                       # many tokens: a prompt; few: a generation step
  y, step = layer.forward(x)         # the same, and what a backward pass needs
  dlogits, dx = layer.backward(step, dweights, dup)

Weights are kept once, in the 4-bit form.  Up to fo.FO_MOE_FEW_TOKENS tokens
go through the one-kernel layer, which reads only the experts that are chosen.
More go through the router, the gathering quantizer and one product per
projection over all experts; the router's logits, the activation between the
projections and the weighted sum of a token's rows are plain torch operations.
Neither way is part of autograd: backward is called with gradients, and tensors
that require one are refused.

``python -m communication_overlap_gb300.expert_layer`` runs a prompt, a
gradient and some generation steps (the last ones replayed from a CUDA graph)
and prints what they took.
"""
import argparse
from dataclasses import dataclass

import torch

from . import fo, moe


@dataclass
class Step:
    """What forward leaves for backward."""
    logits: torch.Tensor
    routing: moe.Routing


class ExpertLayer:
    """router: bf16 [experts, hidden]; w1: [experts, 2 inter, hidden] and w2:
    [experts, hidden, inter] as moe.MxTensor batches.  w1_t, for backward: the
    transpose of w1, quantized along its own rows."""

    def __init__(self, router, w1, w2, top_k, renormalize=True, w1_t=None):
        self.router, self.w1, self.w2, self.w1_t = router, w1, w2, w1_t
        self.top_k, self.renormalize = top_k, renormalize
        self.few = moe.FewTokenLayer(router, w1, w2, top_k, renormalize, "silu")

    @classmethod
    def random(cls, hidden, inter, experts, top_k, seed=0, device="cuda"):
        """Seeded weights, N(0, 1) / sqrt(columns)."""
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape):
            w = torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5
            return w.to(torch.bfloat16)

        router = draw(experts, hidden)
        w1, w2 = draw(experts, 2 * inter, hidden), draw(experts, hidden, inter)
        return cls(router, moe.quantize(w1), moe.quantize(w2), top_k,
                   w1_t=moe.quantize(w1, transpose=True))

    def __call__(self, x):
        return self.few(x) if x.shape[0] <= fo.FO_MOE_FEW_TOKENS else self.forward(x)[0]

    def forward(self, x):
        # fp32, as the one-kernel layer has them: in bf16 close logits would tie, and
        # a token might choose other experts in a prompt than in a generation step
        logits = torch.mm(x, self.router.t(), out_dtype=torch.float32)
        r = moe.route(logits, self.top_k, self.renormalize)
        groups = dict(group_first=r.expert_first, group_rows=r.expert_rows)
        # (rows of no expert are left as they are, and nothing reads them)
        up = torch.empty((r.row_token.numel(), self.w1.rows), dtype=torch.bfloat16,
                         device=x.device)
        moe.mx_gemm(moe.quantize(x, row_index=r.row_token), self.w1, out=up, **groups)
        gate, up = up.chunk(2, dim=1)
        # (the gate, up and silu rounded to bf16, 2^-9 each: the conversion that
        # follows rounds to two significant bits)
        h = torch.nn.functional.silu(gate).mul_(up)
        rows = self._rows(moe.quantize(h), self.w2, groups)
        y = torch.bmm(r.weights.unsqueeze(1), rows[r.token_row.long()]).squeeze(1)
        return y.to(x.dtype), Step(logits, r)

    @staticmethod
    def _rows(a, w, groups):
        """The product per expert in fp32, and after it a row of zeros: the row of
        index -1, which slots without one read."""
        rows = torch.empty((a.rows + 1, w.rows), device=a.codes.device)
        rows[-1] = 0
        moe.mx_gemm(a, w, out=rows[:-1], **groups)
        return rows

    def backward(self, step, dweights, dup):
        """The logits' (fp32) gradient from that of the routing weights (fp32 [tokens,
        top_k]), and the first projection's input's from that of its output
        (`dup`, a row per row of the routing's tables)."""
        if self.w1_t is None:
            raise ValueError("backward needs w1_t")
        r = step.routing
        if dup.dim() != 2 or dup.shape[0] != r.row_token.numel():
            raise ValueError(f"dup: {r.row_token.numel()} rows expected, not {tuple(dup.shape)}")
        dlogits = moe.route_backward(step.logits, r.ids, r.weights, dweights, self.renormalize)
        drows = self._rows(moe.quantize(dup), self.w1_t,
                           dict(group_first=r.expert_first, group_rows=r.expert_rows))
        dx = drows[r.token_row.long()].sum(1)
        return dlogits, dx


def _timed(what, call, n=5):
    call()
    s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    s.record()
    for _ in range(n):
        out = call()
    e.record()
    torch.cuda.synchronize()
    print(f"{what:<44}{s.elapsed_time(e) / n * 1e3:10.1f} us")
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description="an expert layer: prompt, gradient, generation")
    for name, value in (("hidden", 4096), ("inter", 14336), ("experts", 8), ("top_k", 2),
                        ("tokens", 16384)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    layer = ExpertLayer.random(a.hidden, a.inter, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    y, step = _timed(f"prompt of {a.tokens} tokens", lambda: layer.forward(x))
    r = step.routing
    dweights = torch.randn_like(r.weights)
    dup = torch.randn((r.row_token.numel(), 2 * a.inter), device="cuda").to(torch.bfloat16)
    _timed("its gradient (router, first projection)", lambda: layer.backward(step, dweights, dup))
    for n in (1, 8, 48):
        _timed(f"generation step of {n} token{'s' * (n > 1)}", lambda: layer(x[:n]))
    graph, token = torch.cuda.CUDAGraph(), x[:1].clone()
    with torch.cuda.graph(graph):
        out = layer(token)
    _timed("the same of 1 token, from a graph", graph.replay)
    few = y[:1].float()
    off = ((out.float() - few).norm() / few.norm()).item()
    print(f"the prompt's first token against generation's: {off:.3f} apart (the prompt's "
          "activations are 4-bit)")
    if moe.device_status() != fo.FO_OK:
        raise SystemExit(fo.fo_status_string(moe.device_status()))


if __name__ == "__main__":
    main()

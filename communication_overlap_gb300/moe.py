"""The expert layer's operators on torch tensors.

Plumbing only, as ``pipeline.py`` is for the signaled GEMM: torch provides
device memory and the current stream, every step is a libfo.so call (see
``fo.py`` and ``include/fo.h``, which states what each computes).

  route, route_backward   the router: top-k experts, weights, row tables
  quantize, dequantize    to and from the microscaled 4-bit form (MxTensor)
  mx_gemm                 the product of two 4-bit matrices, or one per expert
  FewTokenLayer           a whole expert layer for a generation step's tokens

Calls run on the current stream of the tensors' device and, but for a device's
first, do not synchronise.  Workspaces are kept per device and stream, so calls
on different streams do not share one; a call that is captured into a CUDA graph
takes one of its own from the graph's memory.  ``device_status`` reads (and
synchronises) the sticky status of the calls' bounded waits.  No call is part of
autograd: where it would lose a gradient (not where its result is in 4 bits,
which carry none) it refuses tensors that require one.

A generation step makes small calls, so the time here counts: the device is
switched only where another is current, sizes are computed once per shape.
"""
import functools
import operator
from dataclasses import dataclass

import torch

from . import fo

_TYPES = {torch.bfloat16: fo.FO_TYPE_BF16, torch.float32: fo.FO_TYPE_F32}
_ACTS = {"none": fo.FO_ACT_NONE, "relu": fo.FO_ACT_RELU, "silu": fo.FO_ACT_SILU}
_status, _workspaces = {}, {}


def _type(dtype):
    type_ = _TYPES.get(dtype)
    if type_ is None:
        raise ValueError(f"bf16 or fp32 expected, not {dtype}")
    return type_


def _on_gpu(first, *others):
    """The common CUDA device of the tensors (None entries are skipped)."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")
    if index < 0 or not first.is_cuda:
        raise ValueError("tensors must be on one CUDA device")
    return first.device


def _untracked(*tensors):
    """Refuses tensors whose gradient a call would lose without a word (None entries
    are skipped)."""
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            raise ValueError("no gradient flows through this call: detach its tensors, or call it "
                             "under torch.no_grad() (route_backward is the router's gradient)")


def _number(x):
    """x as a float: what is kept per argument is kept by its value, not by a tensor's
    identity.  A tensor that requires a gradient is refused."""
    if type(x) is float:
        return x
    if isinstance(x, torch.Tensor):
        _untracked(x)
    return float(x)


def _int32(t, n, what):
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what}: contiguous int32[{n}] expected")


def _inner(t, what):
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")


def _row_stride(t, what):
    """Row stride of a matrix (of its length where it has one row)."""
    rows, cols = t.shape[-2:]
    if t.is_contiguous():
        return cols
    _inner(t, what)
    stride = t.stride(-2)
    if rows <= 1:
        return max(cols, stride if t.numel() else 0)
    if stride < cols:
        raise ValueError(f"{what}: rows overlap")
    return stride


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _run(dev, call, *args):
    """call(*args) with dev current."""
    if torch._C._cuda_getDevice() == dev.index:
        call(*args)
    else:
        with torch.cuda.device(dev):
            call(*args)


def _capturing(dev):
    """Whether dev's current stream is being captured into a CUDA graph."""
    if torch._C._cuda_getDevice() == dev.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(dev):
        return torch.cuda.is_current_stream_capturing()


def _status_word(dev):
    st = _status.get(dev)
    if st is None:
        if _capturing(dev):
            raise RuntimeError("call once on this device before capturing into a CUDA graph")
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        torch.cuda.current_stream(dev).synchronize()    # (other streams' calls write it, too)
        _status[dev] = st
    return st.data_ptr()


def _workspace(kind, dev, nbytes, captured=None):
    """A zeroed workspace of at least nbytes for this device and stream.  A call
    under capture gets one of its own (of captured() bytes, where that is less),
    also on a stream that has one: the graph keeps the address, the stream's goes
    back to the allocator when a larger call comes, and a replay may run on
    another stream beside it.  Its memory is the graph's, zeroed by each replay."""
    if _capturing(dev):
        return torch.zeros(captured() if captured else nbytes, dtype=torch.uint8, device=dev)
    key = (kind, dev, _stream(dev))
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _workspaces[key] = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    return ws


def device_status(device="cuda", clear=False):
    """The device's sticky status (FO_OK, FO_ERR_ARG for a product's group out
    of range, FO_ERR_TIMEOUT).  Synchronises.  Clearing an error also gives up the
    device's workspaces: a call whose wait ran out leaves its counters anywhere."""
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if dev not in _status:
        return fo.FO_OK
    torch.cuda.synchronize(dev)
    st = int(_status[dev].item())
    if clear and st != fo.FO_OK:
        _status[dev].zero_()
        torch.cuda.synchronize(dev)     # (before another stream's next error)
        for key in [k for k in _workspaces if k[1] == dev]:
            del _workspaces[key]
    return st


# ------------------------------------------------------------------ 4-bit form

_mx_sizes = functools.lru_cache(256)(fo.fo_mx_sizes)
_route_sizes = functools.lru_cache(256)(fo.fo_moe_route_sizes)


@dataclass
class MxTensor:
    """`batch` matrices rows x cols in the 4-bit form (uint8 tensors)."""
    codes: torch.Tensor
    scales: torch.Tensor
    batch: int
    rows: int
    cols: int

    def __post_init__(self):
        want = _mx_sizes(self.batch, self.rows, self.cols)
        have = (self.codes.numel(), self.scales.numel())
        if have != want or self.codes.dtype != torch.uint8 or self.scales.dtype != torch.uint8:
            raise ValueError(f"uint8 codes and scales of {want} bytes expected, not {have}")
        if not (self.codes.is_contiguous() and self.scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        if self.codes.get_device() != self.scales.get_device():
            raise ValueError("codes and scales must be on one device")


def quantize(x, transpose=False, row_index=None):
    """x: bf16 or fp32, [rows, cols] or [batch, rows, cols] (any row stride).
    transpose: of each matrix's transpose, blocks along its rows.  row_index:
    int32 rows of x to take (an index outside x: a row of zeros)."""
    if x.dim() not in (2, 3):
        raise ValueError("a matrix or a batch of matrices expected")
    dev, type_ = _on_gpu(x, row_index), _type(x.dtype)
    *batch, src_rows, src_cols = x.shape
    batch, batch_stride = (batch[0], x.stride(0)) if batch else (1, 0)
    stride = _row_stride(x, "x")
    rows, cols = (src_cols, src_rows) if transpose else (src_rows, src_cols)
    if row_index is not None:
        if transpose or batch != 1:
            raise ValueError("row_index goes with one matrix, not transposed")
        _int32(row_index, row_index.numel(), "row_index")
        rows = row_index.numel()
    nc, ns = _mx_sizes(batch, rows, cols)
    codes = torch.empty(nc, dtype=torch.uint8, device=dev)
    scales = torch.empty(ns, dtype=torch.uint8, device=dev)
    _run(dev, fo.fo_mx_quantize, x.data_ptr(), type_, batch, batch_stride, rows, cols, stride,
         transpose, 0 if row_index is None else row_index.data_ptr(), src_rows, codes.data_ptr(),
         scales.data_ptr(), _stream(dev))
    return MxTensor(codes, scales, batch, rows, cols)


def dequantize(q, dtype=torch.bfloat16):
    """The values q stands for: [rows, cols], or [batch, rows, cols]."""
    dev, type_ = _on_gpu(q.codes, q.scales), _type(dtype)
    batch, rows, cols = q.batch, q.rows, q.cols
    out = torch.empty((rows, cols) if batch == 1 else (batch, rows, cols), dtype=dtype, device=dev)
    _run(dev, fo.fo_mx_dequantize, q.codes.data_ptr(), q.scales.data_ptr(), batch, rows, cols,
         out.data_ptr(), type_, rows * cols, cols, _stream(dev))
    return out


def mx_gemm(a, b, out=None, out_dtype=torch.bfloat16, group_first=None, group_rows=None):
    """a (M x K) times the transpose of b (N x K).  With group_first and
    group_rows (int32, one entry per matrix of b) a product per expert; rows
    in no group keep what `out` holds."""
    dev = _on_gpu(a.codes, b.codes, out, group_first, group_rows)
    if a.batch != 1 or a.cols != b.cols:
        raise ValueError("a: one matrix with as many columns as b")
    groups = 0
    if (group_first is None) != (group_rows is None):
        raise ValueError("group_first and group_rows go together")
    if group_first is not None:
        groups = b.batch
        _int32(group_first, groups, "group_first")
        _int32(group_rows, groups, "group_rows")
    elif b.batch != 1:
        raise ValueError("a batch of b needs group_first and group_rows")
    if out is None:
        make = torch.zeros if groups else torch.empty
        out = make((a.rows, b.rows), dtype=out_dtype, device=dev)
    if tuple(out.shape) != (a.rows, b.rows):
        raise ValueError(f"out: {(a.rows, b.rows)} expected, not {tuple(out.shape)}")
    if group_first is not None and groups == 0:
        return out          # no row is in a group (to the library, 0: one product of all rows)
    _run(dev, fo.fo_mx_gemm, a.rows, b.rows, a.cols, a.codes.data_ptr(), a.scales.data_ptr(),
         b.codes.data_ptr(), b.scales.data_ptr(), groups,
         0 if group_first is None else group_first.data_ptr(),
         0 if group_rows is None else group_rows.data_ptr(), out.data_ptr(), _type(out.dtype),
         _row_stride(out, "out"), _status_word(dev), _stream(dev))
    return out


# ------------------------------------------------------------------ the router

@dataclass
class Routing:
    ids: torch.Tensor           # int32 [tokens, top_k], -1: no expert
    weights: torch.Tensor       # fp32 [tokens, top_k]
    row_token: torch.Tensor     # int32 [table rows], -1: no token
    row_slot: torch.Tensor      # int32 [table rows]
    token_row: torch.Tensor     # int32 [tokens, top_k], -1: dropped
    expert_first: torch.Tensor  # int32 [experts]
    expert_rows: torch.Tensor   # int32 [experts]


_SCORES = {"softmax": fo.FO_SCORE_SOFTMAX, "sigmoid": fo.FO_SCORE_SIGMOID}


@functools.lru_cache(256)
def _route_desc(experts, top_k, renormalize, capacity, scoring, groups, top_groups, group_top,
                scale):
    """The balanced router's description, None where the call is the plain router's."""
    if scoring not in _SCORES:
        raise ValueError(f"scoring: one of {sorted(_SCORES)} expected, not {scoring!r}")
    if scoring == "softmax" and groups == 1 and scale == 1.0:
        return None
    return fo.make_route_desc(experts, top_k, renormalize, capacity, _SCORES[scoring], groups,
                              top_groups, group_top, scale)


def route(logits, top_k, renormalize=True, capacity=0, scoring="softmax", bias=None, groups=1,
          top_groups=1, group_top=1, scale=1.0):
    """The top-k choice of logits [tokens, experts] (bf16 or fp32).

    The balanced router's options: scoring "softmax" or "sigmoid"; bias (fp32
    [experts]) is added to the scores for the choice, not for the weights;
    with groups, only the experts of the top_groups groups whose group_top (1
    or 2) largest sum to the most may be chosen; scale multiplies the weights."""
    _untracked(logits)
    if logits.dim() != 2:
        raise ValueError("logits: [tokens, experts] expected")
    dev, type_ = _on_gpu(logits, bias), _type(logits.dtype)
    T, E = logits.shape
    index = operator.index      # (as _number: integers, not tensors that may change)
    top_k, capacity, groups = index(top_k), index(capacity), index(groups)
    top_groups, group_top, scale = index(top_groups), index(group_top), _number(scale)
    M, nbytes = _route_sizes(T, E, top_k, capacity)
    desc = _route_desc(E, top_k, bool(renormalize), capacity, scoring, groups, top_groups,
                       group_top, scale)
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_contiguous() or tuple(bias.shape) != (E,):
            raise ValueError(f"bias: contiguous fp32[{E}] expected")
    if desc is None and (bias is not None or (top_groups, group_top) != (1, 1)):
        # (of one group there is one to choose: as the balanced router refuses others)
        desc = fo.make_route_desc(E, top_k, renormalize, capacity, top_groups=top_groups,
                                  group_top=group_top)
    # (seven allocations are cheaper than one and seven views of it)
    empty, i32 = torch.empty, torch.int32
    ids = empty((T, top_k), dtype=i32, device=dev)
    token_row = empty((T, top_k), dtype=i32, device=dev)
    row_token = empty(M, dtype=i32, device=dev)
    row_slot = empty(M, dtype=i32, device=dev)
    first, rows = empty(E, dtype=i32, device=dev), empty(E, dtype=i32, device=dev)
    weights = empty((T, top_k), dtype=torch.float32, device=dev)
    ws = _workspace("route", dev, nbytes)
    to = (ids.data_ptr(), weights.data_ptr(), row_token.data_ptr(), row_slot.data_ptr(),
          token_row.data_ptr(), first.data_ptr(), rows.data_ptr(), ws.data_ptr(),
          _status_word(dev), _stream(dev))
    if desc is None:
        _run(dev, fo.fo_moe_route, logits.data_ptr(), type_, T, E, _row_stride(logits, "logits"),
             top_k, renormalize, capacity, *to)
    else:
        _run(dev, fo.fo_moe_route_scored, desc, logits.data_ptr(), type_, T,
             _row_stride(logits, "logits"), 0 if bias is None else bias.data_ptr(), *to)
    return Routing(ids, weights, row_token, row_slot, token_row, first, rows)


def route_backward(logits, ids, weights, dweights, renormalize=True, scoring="softmax",
                   scale=1.0):
    """The gradient of the logits from that of the weights (fp32).  The bias and
    the groups have had their say in ids and enter no further."""
    _untracked(logits, weights, dweights)
    if logits.dim() != 2:
        raise ValueError("logits: [tokens, experts] expected")
    dev, type_ = _on_gpu(logits, ids, weights, dweights), _type(logits.dtype)
    T, E = logits.shape
    k = ids.shape[-1]
    _int32(ids, T * k, "ids")
    for t, what in ((weights, "weights"), (dweights, "dweights")):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != T * k:
            raise ValueError(f"{what}: contiguous fp32[{T}, {k}] expected")
    desc = _route_desc(E, k, bool(renormalize), 0, scoring, 1, 1, 1, _number(scale))
    out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    if desc is None:
        _run(dev, fo.fo_moe_route_backward, logits.data_ptr(), type_, T, E,
             _row_stride(logits, "logits"), k, renormalize, ids.data_ptr(), weights.data_ptr(),
             dweights.data_ptr(), out.data_ptr(), E, _stream(dev))
    else:
        _run(dev, fo.fo_moe_route_scored_backward, desc, logits.data_ptr(), type_, T,
             _row_stride(logits, "logits"), ids.data_ptr(), weights.data_ptr(),
             dweights.data_ptr(), out.data_ptr(), E, _stream(dev))
    return out


# ------------------------------------------------------------------ few tokens

class FewTokenLayer:
    """An expert layer for up to fo.FO_MOE_FEW_TOKENS tokens at a time.

    router: bf16 [experts, hidden].  w1: bf16 [experts, 2 * inter, hidden],
    the gate's rows first, and w2: bf16 [experts, hidden, inter]; or both as
    MxTensor batches of those shapes.  x's rows and all of these start on 16
    bytes."""

    def __init__(self, router, w1, w2, top_k, renormalize=True, act="silu"):
        mx = isinstance(w1, MxTensor)
        if mx != isinstance(w2, MxTensor):
            raise ValueError("w1 and w2 take the same form")
        E, H = router.shape
        s1 = (w1.batch, w1.rows, w1.cols) if mx else tuple(w1.shape)
        s2 = (w2.batch, w2.rows, w2.cols) if mx else tuple(w2.shape)
        I = s2[-1]
        if s1 != (E, 2 * I, H) or s2 != (E, H, I):
            raise ValueError(f"w1 {s1} and w2 {s2} do not fit a router of {E} x {H}")
        parts = (w1.codes, w1.scales, w2.codes, w2.scales) if mx else (w1, None, w2, None)
        for t in (router,) + (() if mx else (w1, w2)):
            if t.dtype != torch.bfloat16 or not t.is_contiguous():
                raise ValueError("contiguous bf16 weights expected")
        self.device = _on_gpu(router, *parts)
        self.router, self._keep = router, parts
        self._float = (router,) if mx else (router, w1, w2)
        self.hidden, self.top_k = H, top_k
        self._w = [0 if t is None else t.data_ptr() for t in parts]
        self._desc = functools.lru_cache(fo.FO_MOE_FEW_TOKENS)(lambda tokens: fo.make_few_desc(
            tokens, H, I, E, top_k, renormalize, _ACTS[act],
            fo.FO_TYPE_MX4 if mx else fo.FO_TYPE_BF16))
        self._bytes = fo.fo_moe_few_workspace(self._desc(fo.FO_MOE_FEW_TOKENS))   # any call's

    def __call__(self, x, out=None):
        """x: bf16 [tokens, hidden] -> y of the same shape."""
        _untracked(x, *self._float)
        if x.dim() != 2 or x.shape[1] != self.hidden or x.dtype != torch.bfloat16:
            raise ValueError(f"x: bf16 [tokens, {self.hidden}] expected")
        dev = _on_gpu(x, self.router, out)
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        if out.shape != x.shape or out.dtype != torch.bfloat16:
            raise ValueError("out: bf16 of x's shape expected")
        w1, s1, w2, s2 = self._w
        desc = self._desc(x.shape[0])
        ws = _workspace("few", dev, self._bytes, lambda: fo.fo_moe_few_workspace(desc))
        _run(dev, fo.fo_moe_few, desc, x.data_ptr(), _row_stride(x, "x"),
             self.router.data_ptr(), w1, s1, w2, s2, out.data_ptr(), _row_stride(out, "out"),
             ws.data_ptr(), _status_word(dev), _stream(dev))
        return out

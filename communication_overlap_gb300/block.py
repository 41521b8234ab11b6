"""What stands around the expert layer's products in a model's block, on torch
tensors.

Plumbing only, as ``moe.py``: torch provides device memory and the current
stream, every step is a libfo.so call (``include/fo.h`` states what each
computes).

  norm, norm_backward           RMS norm of a block's output, its gate and scale
                                into the residual stream, RMS norm of the stream
                                for the next block, in one pass
  activate, activate_backward   the gated activation between the projections,
                                with a checkpoint of 8 bits for the backward pass
  combine, combine_backward     the weighted sum of a token's rows of the experts'
                                outputs

Calls run on the current stream of the tensors' device and do not synchronise.
None is part of autograd: tensors that require a gradient are refused (detach
them, or call under ``torch.no_grad()``).  ``moe.device_status`` tells of a row
index that was out of range.
"""
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import fo
from .moe import (_ACTS, _int32, _number, _on_gpu, _row_stride, _run, _status_word, _stream,
                  _type, _untracked)

_checkpoint_sizes = functools.lru_cache(256)(fo.fo_checkpoint_sizes)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stride(t, what):
    """Row stride of a matrix, 0 of none."""
    return 0 if t is None else _row_stride(t, what)


def _matrix(t, shape, dtype, what):
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} {shape} expected, not {t.dtype} {tuple(t.shape)}")


# ------------------------------------------------------------------ the norms

@dataclass
class Normed:
    stream: torch.Tensor                # the residual stream after the block
    y: Optional[torch.Tensor]           # the next block's input, where pre_gain was given
    rstd: Optional[torch.Tensor]        # fp32 [2, tokens], of the two norms: norm_backward
                                        #   reads the rows whose gains were given

    @property
    def post_rstd(self):
        return self.rstd[0]

    @property
    def pre_rstd(self):
        return self.rstd[1]


@dataclass
class NormGrads:
    x: torch.Tensor
    residual: Optional[torch.Tensor]
    post_gain: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    pre_gain: Optional[torch.Tensor]


@functools.lru_cache(256)
def _norm_desc(T, H, dtype, stream_dtype, param_dtype, gates, scale, eps):
    if dtype == torch.float32 and stream_dtype != torch.float32:
        raise ValueError("a bf16 residual stream takes bf16 blocks")
    if gates < 1 or T % gates:
        raise ValueError(f"gate: {gates} rows do not divide {T} tokens")
    desc = fo.make_norm_desc(T, H, _type(dtype), _type(stream_dtype), _type(param_dtype), gates,
                             scale, eps)
    return desc, fo.fo_block_norm_workspace(desc)


def _norm_args(x, residual, post_gain, gate, pre_gain, scale, eps):
    """(device, tokens, hidden, (description, workspace bytes), the gate's row stride)"""
    dev = _on_gpu(x, residual, post_gain, gate, pre_gain)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: [tokens, hidden] expected")
    T, H = shape
    stream_dtype = x.dtype
    if residual is not None:
        stream_dtype = residual.dtype
        if residual.shape != shape:
            raise ValueError(f"residual: {tuple(shape)} expected, not {tuple(residual.shape)}")
    param_dtype, gates, gate_stride = None, 1, 0
    for p, what in ((post_gain, "post_gain"), (pre_gain, "pre_gain")):
        if p is None:
            continue
        if p.shape != (H,) or not p.is_contiguous():
            raise ValueError(f"{what}: contiguous [{H}] expected, not {tuple(p.shape)}")
        if param_dtype is not None and p.dtype != param_dtype:
            raise ValueError("the gains and the gate have one type")
        param_dtype = p.dtype
    if gate is not None:
        if gate.dim() == 2 and gate.shape[1] == H:
            # (of no tokens, no rows are a row for each, too)
            gates, gate_stride = gate.shape[0] or int(T == 0), _row_stride(gate, "gate")
        elif gate.shape == (H,) and gate.is_contiguous():
            gate_stride = H
        else:
            raise ValueError(f"gate: [{H}] or [rows, {H}] expected, not {tuple(gate.shape)}")
        if param_dtype is not None and gate.dtype != param_dtype:
            raise ValueError("the gains and the gate have one type")
        param_dtype = gate.dtype
    return dev, T, H, _norm_desc(T, H, x.dtype, stream_dtype, param_dtype or torch.float32, gates,
                                 scale, eps), gate_stride


def norm(x, residual=None, post_gain=None, gate=None, scale=1.0, pre_gain=None, eps=1e-6):
    """stream = residual + scale * gate * (RMS norm of x times post_gain), y = RMS
    norm of the stream times pre_gain; without post_gain x as it is, without
    residual or gate as if they were zeros or ones.

    x: [tokens, hidden], bf16 or fp32 (any row stride); y has its type.
    residual and stream: bf16 or fp32, fp32 for fp32 x.  gains: [hidden]; gate:
    [hidden], or [rows, hidden] where rows divides tokens (a row for each run of
    tokens / rows tokens); all of one type.  Where nothing but pre_gain is
    given, the stream is x itself."""
    _untracked(x, residual, post_gain, gate, pre_gain)
    scale, eps = _number(scale), _number(eps)
    dev, T, H, (desc, _), gate_stride = _norm_args(x, residual, post_gain, gate, pre_gain, scale,
                                                   eps)
    stream, y, rstd, at = x, None, None, 0
    summed = residual is not None or post_gain is not None or gate is not None or scale != 1.0
    if summed:
        stream = torch.empty((T, H), dtype=x.dtype if residual is None else residual.dtype,
                             device=dev)
    if pre_gain is not None:
        y = torch.empty((T, H), dtype=x.dtype, device=dev)
    if pre_gain is not None or post_gain is not None:
        rstd = torch.empty((2, T), dtype=torch.float32, device=dev)
        at = rstd.data_ptr()
    _run(dev, fo.fo_block_norm, desc, x.data_ptr(), _row_stride(x, "x"), _ptr(residual),
         _stride(residual, "residual"), _ptr(post_gain), _ptr(gate), gate_stride, _ptr(pre_gain),
         stream.data_ptr() if summed else 0, H, _ptr(y), H, at, at + 4 * T if at else 0,
         _stream(dev))
    return Normed(stream, y, rstd)


def norm_backward(x, residual, normed, dstream=None, dy=None, post_gain=None, gate=None,
                  scale=1.0, pre_gain=None):
    """The gradients of norm's inputs and parameters, from those of its stream
    (None: zeros) and of its y (None where there was none).  x, residual and the
    parameters: the forward call's; normed: what it returned."""
    _untracked(x, residual, post_gain, gate, pre_gain, dstream, dy)
    dev, T, H, (desc, nbytes), gate_stride = _norm_args(x, residual, post_gain, gate, pre_gain,
                                                        _number(scale), 0.0)
    rstd = normed.rstd
    _on_gpu(x, dstream, dy, rstd)
    if (dy is None) != (pre_gain is None):
        raise ValueError("dy and pre_gain go together")
    if dy is not None:
        _matrix(dy, (T, H), x.dtype, "dy")
    if dstream is not None:
        _matrix(dstream, (T, H), x.dtype if residual is None else residual.dtype, "dstream")
    at = 0
    if post_gain is not None or pre_gain is not None:
        if (rstd is None or rstd.shape != (2, T) or rstd.dtype != torch.float32
                or not rstd.is_contiguous()):
            raise ValueError(f"normed holds no norms of {T} tokens")
        at = rstd.data_ptr()
    empty, like = torch.empty, torch.empty_like
    dx = empty((T, H), dtype=x.dtype, device=dev)
    dresidual = None if residual is None else empty((T, H), dtype=residual.dtype, device=dev)
    dpost = None if post_gain is None else like(post_gain)
    dpre = None if pre_gain is None else like(pre_gain)
    dgate = None if gate is None else empty(gate.shape, dtype=gate.dtype, device=dev)
    ws = empty(nbytes, dtype=torch.uint8, device=dev)
    _run(dev, fo.fo_block_norm_backward, desc, x.data_ptr(), _row_stride(x, "x"), _ptr(residual),
         _stride(residual, "residual"), _ptr(post_gain), _ptr(gate), gate_stride, _ptr(pre_gain),
         at, at + 4 * T if at else 0, _ptr(dstream), _stride(dstream, "dstream"), _ptr(dy),
         _stride(dy, "dy"), dx.data_ptr(), H, _ptr(dresidual), H, _ptr(dpost), _ptr(dgate),
         _ptr(dpre), ws.data_ptr(), _stream(dev))
    return NormGrads(dx, dresidual, dpost, dgate, dpre)


# ------------------------------------------------------------------ the activation

@dataclass
class Checkpoint:
    """[gate | up] rows in 8 bits: int8 codes [rows, 2, padded], a scale byte per
    32 values (include/fo.h states the form)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    inter: int
    act: str

    def __post_init__(self):
        want = _checkpoint_sizes(self.rows, self.inter)
        have = (self.codes.numel(), self.scales.numel())
        if have != want or self.codes.dtype != torch.int8 or self.scales.dtype != torch.uint8:
            raise ValueError(f"int8 codes and uint8 scales of {want} bytes expected, not {have}")
        if not (self.codes.is_contiguous() and self.scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        if self.codes.get_device() != self.scales.get_device():
            raise ValueError("codes and scales must be on one device")
        if self.act not in _ACTS:
            raise ValueError(f"act: one of {sorted(_ACTS)} expected, not {self.act!r}")

    def values(self, dtype=torch.float32):
        """The values it stands for, [rows, 2 * inter]."""
        if self.rows == 0 or self.inter == 0:
            return torch.empty((self.rows, 2 * self.inter), dtype=dtype, device=self.codes.device)
        s = self.scales.view(self.rows, 2, -1, 1).to(torch.int32)
        step = torch.where(s == 0, torch.full_like(s, 1 << 22), s << 23).view(torch.float32)
        step = torch.where(s == 255, torch.full_like(step, float("nan")), step)
        v = self.codes.view(self.rows, 2, s.shape[2], 32).to(torch.float32) * step
        return v.view(self.rows, 2, -1)[..., :self.inter].reshape(self.rows, -1).to(dtype)


def activate(u, act="silu", checkpoint=False):
    """h = act(gate) * up for rows u = [gate | up] (bf16 or fp32, any row stride),
    and with checkpoint what activate_backward needs of u, in 8 bits: (h, kept),
    kept None without."""
    _untracked(u)
    if u.dim() != 2 or u.shape[1] % 2:
        raise ValueError("u: [rows, 2 * inter] expected")
    dev, type_ = _on_gpu(u), _type(u.dtype)
    if act not in _ACTS:
        raise ValueError(f"act: one of {sorted(_ACTS)} expected, not {act!r}")
    R, I = u.shape[0], u.shape[1] // 2
    h = torch.empty((R, I), dtype=u.dtype, device=dev)
    kept = None
    if checkpoint:
        nc, ns = _checkpoint_sizes(R, I)
        kept = Checkpoint(torch.empty(nc, dtype=torch.int8, device=dev),
                          torch.empty(ns, dtype=torch.uint8, device=dev), R, I, act)
    _run(dev, fo.fo_gated_act, u.data_ptr(), type_, R, I, _row_stride(u, "u"), _ACTS[act],
         h.data_ptr(), I, kept.codes.data_ptr() if kept else 0,
         kept.scales.data_ptr() if kept else 0, _stream(dev))
    return h, kept


def activate_backward(dh, kept):
    """The gradient of u (in dh's type) from that of h, with the values that the
    checkpoint stands for."""
    _untracked(dh)
    if tuple(dh.shape) != (kept.rows, kept.inter):
        raise ValueError(f"dh: {(kept.rows, kept.inter)} expected, not {tuple(dh.shape)}")
    dev, type_ = _on_gpu(dh, kept.codes, kept.scales), _type(dh.dtype)
    du = torch.empty((kept.rows, 2 * kept.inter), dtype=dh.dtype, device=dev)
    _run(dev, fo.fo_gated_act_backward, dh.data_ptr(), type_, kept.rows, kept.inter,
         _row_stride(dh, "dh"), _ACTS[kept.act], kept.codes.data_ptr(), kept.scales.data_ptr(),
         du.data_ptr(), 2 * kept.inter, _stream(dev))
    return du


# ------------------------------------------------------------------ the weighted sum

def _slots(token_row, weights):
    if token_row.dim() != 2:
        raise ValueError("token_row: int32 [tokens, top_k] expected")
    _int32(token_row, token_row.numel(), "token_row")
    if weights is not None and (weights.dtype != torch.float32 or not weights.is_contiguous()
                                or weights.shape != token_row.shape):
        raise ValueError(f"weights: contiguous fp32 {tuple(token_row.shape)} expected")
    return token_row.shape


def combine(rows, token_row, weights=None, out=None, out_dtype=None):
    """y[t] = sum over slots s of weights[t, s] * rows[token_row[t, s]] (-1: no
    row; no weights: ones).  rows: [table rows, hidden], bf16 or fp32, any row
    stride; token_row and weights as a Routing holds them; out must not overlap
    rows."""
    _untracked(rows, weights, out)
    if rows.dim() != 2:
        raise ValueError("rows: [table rows, hidden] expected")
    T, k = _slots(token_row, weights)
    dev, type_ = _on_gpu(rows, token_row, weights, out), _type(rows.dtype)
    M, H = rows.shape
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype or rows.dtype, device=dev)
    if tuple(out.shape) != (T, H):
        raise ValueError(f"out: {(T, H)} expected, not {tuple(out.shape)}")
    _run(dev, fo.fo_moe_combine, _ptr(rows), type_, M, H, _row_stride(rows, "rows"),
         token_row.data_ptr(), _ptr(weights), T, k, out.data_ptr(), _type(out.dtype),
         _row_stride(out, "out"), _status_word(dev), _stream(dev))
    return out


def combine_backward(dy, rows, token_row, row_token, weights=None):
    """(drows, dweights): drows has rows' type, with zeros where a row holds no
    token; dweights (fp32) is None without weights.  token_row and row_token: of
    one Routing."""
    _untracked(dy, rows, weights)
    if rows.dim() != 2:
        raise ValueError("rows: [table rows, hidden] expected")
    T, k = _slots(token_row, weights)
    M, H = rows.shape
    if tuple(dy.shape) != (T, H):
        raise ValueError(f"dy: {(T, H)} expected, not {tuple(dy.shape)}")
    _int32(row_token, M, "row_token")
    dev = _on_gpu(dy, rows, token_row, row_token, weights)
    drows = torch.empty((M, H), dtype=rows.dtype, device=dev)
    dweights = None if weights is None else torch.empty_like(weights)
    _run(dev, fo.fo_moe_combine_backward, dy.data_ptr(), _type(dy.dtype), _row_stride(dy, "dy"),
         rows.data_ptr(), _type(rows.dtype), M, H, _row_stride(rows, "rows"),
         token_row.data_ptr(), row_token.data_ptr(), _ptr(weights), T, k, drows.data_ptr(), H,
         _ptr(dweights), _status_word(dev), _stream(dev))
    return drows, dweights

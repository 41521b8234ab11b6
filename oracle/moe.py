"""The expert layer's operators in plain numpy, in 64 bits.

Written from the definitions alone (include/fo.h states them); shares no code
with the library.  Matrices in the microscaled 4-bit form are handled as
(codes, scales): codes 0..15 per value and scale bytes per 32 values, both
unpadded in rows and padded with zeros to whole blocks of 128 columns.
"""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------ 4-bit form

def mx_quantize(x):
    """x: float64 [rows, cols] -> (codes [rows, C], scales [rows, C / 32])."""
    rows, cols = x.shape
    full = np.zeros((rows, _up(cols, 128)))
    full[:, :cols] = x
    b = full.reshape(rows, -1, 32)
    codes = np.zeros(b.shape, dtype=np.uint8)
    scales = np.zeros(b.shape[:2], dtype=np.uint8)
    for r in range(rows):
        for j in range(b.shape[1]):
            v = b[r, j]
            if not np.isfinite(v).all():
                scales[r, j] = 255
                continue
            a = np.abs(v).max()
            e = max(int(np.floor(np.log2(a))) - 2, -127) if a > 0 else -127
            if a > 0 and 2.0 ** (e + 3) <= a and e > -127:   # log2 rounded down
                e += 1
            scales[r, j] = e + 127
            u = np.abs(v) / 2.0 ** e
            dist = np.abs(u[:, None] - E2M1[None])
            near = dist == dist.min(1, keepdims=True)
            for i in range(32):
                c = np.flatnonzero(near[i])
                # a tie lies between neighbours: the even code
                codes[r, j, i] = c[0] if len(c) == 1 or c[0] % 2 == 0 else c[1]
            codes[r, j] += np.where(np.signbit(v), 8, 0).astype(np.uint8)
    return codes.reshape(rows, -1), scales


def mx_values(codes, scales):
    sign = np.where(codes >= 8, -1.0, 1.0)
    v = sign * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(len(codes), -1, 32) * s[..., None]).reshape(codes.shape)


def mx_pack(codes, scales):
    """The library's bytes: rows padded to 128, scales in blocks of 512."""
    rows, C = codes.shape
    R = _up(rows, 128)
    full = np.zeros((R, C), dtype=np.uint8)
    full[:rows] = codes
    s = np.zeros((R, C // 32), dtype=np.uint8)
    s[:rows] = scales
    out = np.zeros((R // 128, C // 128, 512), dtype=np.uint8)
    for r in range(R):
        for j in range(C // 32):
            q = r % 128
            out[r // 128, j // 4, (q % 32) * 16 + (q // 32) * 4 + j % 4] = s[r, j]
    return (full[:, 0::2] | (full[:, 1::2] << 4)).reshape(-1), out.reshape(-1)


# ------------------------------------------------------------------ the router

def route(logits, top_k, renormalize, capacity=0):
    """logits: float64 [tokens, experts].  A dict of the router's outputs."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int64)
    w = np.zeros((T, top_k))
    for t in range(T):
        l = logits[t]
        order = sorted(range(E), key=lambda e: (not np.isnan(l[e]),
                                                -l[e] if not np.isnan(l[e]) else 0.0, e))
        chosen = [e for e in order if l[e] != -np.inf][:top_k]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if not l[chosen[0]] < np.inf:      # NaN or +inf
            w[t, :len(chosen)] = np.nan
            continue
        p = np.exp(l - l[chosen[0]])
        w[t, :len(chosen)] = p[chosen] / (p[chosen].sum() if renormalize else p.sum())
    M = E * capacity if capacity else (T * top_k + E * 127) // 128 * 128
    row_token, row_slot = np.full(M, -1), np.zeros(M, dtype=np.int64)
    token_row = np.full((T, top_k), -1)
    first, rows, at = [], [], 0
    for e in range(E):
        if capacity:
            at = e * capacity
        pairs = [(t, s) for t, s in zip(*np.nonzero(ids == e))]
        if capacity:
            pairs = pairs[:capacity]
        for i, (t, s) in enumerate(pairs):
            row_token[at + i], row_slot[at + i], token_row[t, s] = t, s, at + i
        first.append(at)
        rows.append(len(pairs))
        at += _up(len(pairs), 128)
    return dict(ids=ids, weights=w, row_token=row_token, row_slot=row_slot,
                token_row=token_row, expert_first=np.array(first), expert_rows=np.array(rows))


def route_weights(logits, ids, renormalize):
    """The weights of a given choice: what the gradient differentiates."""
    w = np.zeros(ids.shape)
    for t in range(len(logits)):
        live = ids[t] >= 0
        if live.any():
            p = np.exp(logits[t] - logits[t].max())
            c = p[ids[t][live]]
            w[t, live] = c / (c.sum() if renormalize else p.sum())
    return w


def route_backward(logits, ids, g, renormalize):
    """The gradient of sum(g * weights) by the softmax's Jacobian."""
    d = np.zeros_like(logits)
    w = route_weights(logits, ids, renormalize)
    for t in range(len(logits)):
        live = ids[t] >= 0
        if not live.any():
            continue
        i, wt, gt = ids[t][live], w[t][live], g[t][live]
        if renormalize:
            d[t, i] = (np.diag(wt) - np.outer(wt, wt)) @ gt
        else:
            p = np.exp(logits[t] - logits[t].max())
            p /= p.sum()
            full = np.zeros(len(p))
            full[i] = gt
            d[t] = (np.diag(p) - np.outer(p, p)) @ full
    return d


# ------------------------------------------------------------------ few tokens

def activation(g, act):
    if act == "relu":
        return np.where(g > 0, g, 0.0)
    return g / (1.0 + np.exp(-g)) if act == "silu" else g


def few(x, router, w1, w2, top_k, renormalize, act="silu"):
    """(y, spread): the layer's outputs, and sum_s w_s |W2| |h|, the size of
    the terms that are added up."""
    I = w2.shape[2]
    r = route(x @ router.T, top_k, renormalize)
    y, spread = np.zeros_like(x), np.zeros_like(x)
    for t in range(len(x)):
        for s in range(top_k):
            e = r["ids"][t, s]
            if e < 0:
                continue
            a = w1[e] @ x[t]
            h = activation(a[:I], act) * a[I:]
            y[t] += r["weights"][t, s] * (w2[e] @ h)
            spread[t] += r["weights"][t, s] * (np.abs(w2[e]) @ np.abs(h))
    return y, spread

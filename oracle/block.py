"""The operators around the expert layer's products in plain numpy, in 64 bits.

Written from the definitions alone (include/fo.h states them); shares no code
with the library.
"""
import numpy as np


# ------------------------------------------------------------------ the router

def scores(l, sigmoid):
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1 / (1 + np.exp(-l))
        e = np.exp(l - l.max())
        return e / e.sum()


def _ranked(c):
    """Indices by descending value, NaN above everything, ties to the lowest."""
    key = np.where(np.isnan(c), np.inf, c)
    return np.lexsort((np.arange(len(c)), -key, ~np.isnan(c)))


def choose(l, sigmoid, bias, groups, top_groups, group_top, top_k):
    """The experts of one token, fewer than top_k where fewer are left."""
    c = scores(l, sigmoid)
    by = l.copy() if bias is None else c + bias     # without a bias the order is the logits'
    c = c if bias is None else by
    barred = (l == -np.inf) | (by == -np.inf)
    per = len(l) // groups
    total = np.full(groups, -np.inf)
    for g in range(groups):
        mine = np.array([i for i in range(g * per, (g + 1) * per) if not barred[i]], dtype=int)
        if not len(mine):
            continue
        v = c[mine] if group_top == 2 or bias is not None else by[mine]
        total[g] = v[_ranked(v)[:group_top]].sum()
    keep = [g for g in _ranked(total)[:top_groups] if total[g] != -np.inf]
    open_ = [i for i in range(len(l)) if i // per in keep and not barred[i]]
    order = _ranked(by[open_])
    return [open_[i] for i in order[:top_k]]


def route_scored(logits, top_k, renormalize, sigmoid, bias=None, groups=1, top_groups=1,
                 group_top=1, scale=1.0):
    T = len(logits)
    ids, w = np.full((T, top_k), -1), np.zeros((T, top_k))
    for t in range(T):
        mine = choose(logits[t], sigmoid, bias, groups, top_groups, group_top, top_k)
        s = scores(logits[t], sigmoid)[mine]
        if renormalize and len(mine):
            if sigmoid:     # (scaled, so that small ones do not vanish)
                l = logits[t][mine]
                with np.errstate(all="ignore"):
                    log_s = -np.logaddexp(0, -l)
                s = np.exp(log_s - log_s.max())
            else:
                s = np.exp(logits[t][mine] - logits[t][mine].max())
            s = s / s.sum()
        ids[t, :len(mine)] = mine
        w[t, :len(mine)] = scale * s
    return ids, w


def route_scored_backward(logits, ids, dweights, renormalize, sigmoid, scale=1.0):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        slots = np.flatnonzero(ids[t] >= 0)
        if not len(slots):
            continue
        mine = ids[t][slots]
        g = dweights[t][slots]
        s = scores(logits[t], sigmoid)
        chosen = s[mine]
        if renormalize:
            total = chosen.sum()
            ds = scale * (g / total - (g * chosen).sum() / total ** 2)
        else:
            ds = scale * g
        if sigmoid:
            out[t, mine] = ds * chosen * (1 - chosen)
        else:
            full = np.zeros(E)
            full[mine] = ds
            out[t] = s * (full - (s * full).sum())
    return out


# ------------------------------------------------------------------ the norms

def _gate_rows(gate, T, H):
    if gate is None:
        return np.ones((T, H))
    gate = gate.reshape(-1, H)
    return np.repeat(gate, T // len(gate), axis=0)


def norm(x, residual, post, gate, scale, pre, eps):
    """(sum, y, and the values in between)"""
    T, H = x.shape
    r1 = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    xn = x * r1 if post is not None else x
    u = xn * post if post is not None else x
    q = scale * _gate_rows(gate, T, H)
    s = q * u + (0 if residual is None else residual)
    r2 = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    y = s * r2 * pre if pre is not None else None
    return dict(sum=s, y=y, xn=xn, u=u, q=q, r1=r1, r2=r2)


def norm_backward(x, residual, post, gate, scale, pre, eps, dsum, dy):
    T, H = x.shape
    f = norm(x, residual, post, gate, scale, pre, eps)
    d = np.zeros((T, H)) if dsum is None else dsum.copy()
    out = {}
    if pre is not None:
        sn = f["sum"] * f["r2"]
        out["pre_gain"] = (dy * sn).sum(0)
        e = dy * pre
        d += f["r2"] * (e - sn * (e * sn).mean(1, keepdims=True))
    out["residual"] = d
    if gate is not None:
        part = scale * f["u"] * d
        out["gate"] = part.reshape(gate.size // H, -1, H).sum(1).reshape(gate.shape)
    e = f["q"] * d
    if post is not None:
        out["post_gain"] = (e * f["xn"]).sum(0)
        e = e * post
        e = f["r1"] * (e - f["xn"] * (e * f["xn"]).mean(1, keepdims=True))
    out["x"] = e
    return out


# ------------------------------------------------------------------ the activation

def act(g, kind):
    with np.errstate(all="ignore"):
        if kind == "silu":
            return g / (1 + np.exp(-g))
    return np.where(g > 0, g, 0) if kind == "relu" else g


def act_slope(g, kind):
    if kind == "silu":
        with np.errstate(all="ignore"):
            s = 1 / (1 + np.exp(-g))
        return s * (1 + g * (1 - s))
    return np.where(g > 0, 1.0, 0.0) if kind == "relu" else np.ones_like(g)


def checkpoint(half):
    """(codes [rows, padded], scale bytes, values [rows, cols]) of one half."""
    R, C = half.shape
    P = -(-C // 32) * 32
    full = np.zeros((R, P))
    full[:, :C] = half
    b = full.reshape(R, -1, 32)
    codes, scales = np.zeros(b.shape, dtype=np.int64), np.zeros(b.shape[:2], dtype=np.int64)
    values = np.zeros(b.shape)
    for r in range(R):
        for j in range(b.shape[1]):
            v = b[r, j]
            if not np.isfinite(v).all():
                scales[r, j] = 255
                values[r, j] = np.nan
                continue
            a = np.abs(v).max()
            e = max(int(np.frexp(a)[1]) - 1 - 6, -127) if a > 0 else -127
            scales[r, j] = e + 127
            codes[r, j] = np.clip(np.rint(v / 2.0 ** e), -127, 127)
            values[r, j] = codes[r, j] * 2.0 ** e
    return codes.reshape(R, P), scales, values.reshape(R, P)[:, :C]


# ------------------------------------------------------------------ the weighted sum

def combine(rows, token_row, weights):
    T, k = token_row.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for s in range(k):
            if 0 <= token_row[t, s] < len(rows):
                y[t] += (1.0 if weights is None else weights[t, s]) * rows[token_row[t, s]]
    return y


def combine_backward(dy, rows, token_row, weights):
    drows = np.zeros(rows.shape)
    dw = np.zeros(token_row.shape)
    for t, s in np.argwhere(token_row >= 0):
        r = token_row[t, s]
        drows[r] = (1.0 if weights is None else weights[t, s]) * dy[t]
        dw[t, s] = dy[t] @ rows[r]
    return drows, dw

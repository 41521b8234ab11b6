"""The operators around the expert layer's products: what is measured of them.

Four operators, as a program that trains or serves a block of a model with an
expert layer meets them:

  route    the balanced router: sigmoid or softmax scores, a bias that decides
           the choice but not the weights, groups of experts of which a token
           may use some, top-k, renormalised and scaled weights, the row tables
           of the grouped products, and the gradient of the weights
  norm     RMS norm of a block's output, gate and scale into the residual
           stream, and RMS norm of the stream for the next block, in one pass,
           with the gradients of all of them
  act      the gated activation between an expert's projections, which keeps
           its input in 8 bits for the backward pass (a power-of-two scale per
           32 values), and its gradient from there
  combine  the weighted sum of a token's rows of the experts' outputs, and the
           gradients of the rows and of the weights

``own = False`` computes each in its plain form (elementary torch operations
in 32 bits, rounded once at the end; the router's choice in 64 bits, because
two sums of a score and a bias may be nearer to each other than 32 bits tell),
``own = True`` by the calls of ``communication_overlap_gb300``.
"""
import math

import torch

own = False

BLOCK = 32          # values of a checkpoint that share a scale
ROWS = 128          # an expert's row alignment
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token over many small experts in groups: pure latency
        dict(name="route_one_token", op="route", tokens=1, experts=128, top_k=8, groups=8,
             top_groups=4, group_top=2, scoring="sigmoid", bias=True, scale=2.5, dtype="f32",
             renormalize=True, capacity=0, backward=False),
        # a training batch over 256 experts in 8 groups, with the gradient
        dict(name="route_train_256", op="route", tokens=16384, experts=256, top_k=8, groups=8,
             top_groups=4, group_top=2, scoring="sigmoid", bias=True, scale=2.5, dtype="f32",
             renormalize=True, capacity=0, backward=True),
        # softmax scores over 60 experts in groups of 10, an odd batch, experts of
        # limited capacity, weights as they are
        dict(name="route_softmax_60", op="route", tokens=4095, experts=60, top_k=6, groups=6,
             top_groups=3, group_top=1, scoring="softmax", bias=False, scale=16.0,
             dtype="bf16", renormalize=False, capacity=640, backward=True),
        # one generated token between two blocks: latency
        dict(name="norm_one_token", op="norm", tokens=1, hidden=4096, dtype="bf16",
             stream="bf16", params="bf16", post=True, gate="channel", gates=1, scale=1.0,
             pre=True, backward=False),
        # a training batch: both norms, a gate per channel, forward and backward
        dict(name="norm_train", op="norm", tokens=16384, hidden=4096, dtype="bf16",
             stream="bf16", params="bf16", post=True, gate="channel", gates=1, scale=0.5,
             pre=True, backward=True),
        # five sequences with a gate each, the stream kept in fp32, an odd length
        # of a hidden size that is no power of two
        dict(name="norm_gated_sequences", op="norm", tokens=5 * 819, hidden=2752, dtype="bf16",
             stream="f32", params="f32", post=True, gate="sequence", gates=5, scale=1.0,
             pre=True, backward=True),
        # the two rows of one generated token; nothing is kept for a gradient
        dict(name="act_two_rows", op="act", rows=2, inter=14336, dtype="bf16", act="silu",
             backward=False),
        # the All-to-All expert layer's routed rows, forward and backward
        dict(name="act_train", op="act", rows=32768, inter=14336, dtype="bf16", act="silu",
             backward=True),
        # an odd number of rows of a width whose last scale covers 8 values, fp32
        dict(name="act_odd", op="act", rows=999, inter=1416, dtype="f32", act="silu",
             backward=True),
        # a generation step of a few tokens
        dict(name="combine_seven_tokens", op="combine", tokens=7, hidden=4096, experts=8,
             top_k=2, capacity=0, dtype="bf16", out="bf16", backward=False),
        # the All-to-All expert layer, forward and backward
        dict(name="combine_train", op="combine", tokens=16384, hidden=4096, experts=8, top_k=2,
             capacity=0, dtype="bf16", out="bf16", backward=True),
        # many small experts whose capacity drops some pairs, fp32 rows
        dict(name="combine_dropped", op="combine", tokens=5001, hidden=2048, experts=60,
             top_k=6, capacity=512, dtype="f32", out="bf16", backward=True),
    ]


def _log_int(rng, lo, hi):
    """An integer in [lo, hi], uniform in its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["route", "norm", "act", "combine"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 6, 8])
        experts = groups * _log_int(rng, 4, 256 // groups)
        tokens = _log_int(rng, 1, min(32768, 16384 * 256 // experts))
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, top_groups * (experts // groups)))
        # (softmax without groups is the other router)
        scoring = "sigmoid" if groups == 1 else rng.choice(["sigmoid", "softmax"])
        cap = rng.random() < 0.3
        capacity = -(-int(1.25 * tokens * top_k / experts + 1) // ROWS) * ROWS if cap else 0
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), scoring=scoring,
                    bias=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["bf16", "f32"]),
                    # (of one weight, renormalised, the gradient is zero)
                    renormalize=top_k > 1 and rng.random() < 0.5,
                    capacity=capacity, backward=rng.random() < 0.5)
    if op == "norm":
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            hidden = -(-hidden // 8) * 8
        post = rng.random() < 0.6
        pre = not post or rng.random() < 0.5
        gate = rng.choice(["none", "channel", "sequence", "token"])
        gates = _log_int(rng, 2, 16) if gate == "sequence" else 1
        tokens = gates * _log_int(rng, 1, min(32768, 16384 * 4096 // hidden) // gates)
        if gate == "token":
            tokens = max(1, tokens // 2)
            gates = tokens
        dtype = rng.choice(["bf16", "f32"])
        stream = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        if stream == "f32":
            tokens = gates * max(1, tokens // gates // 2)
        return dict(op=op, tokens=tokens, hidden=hidden, dtype=dtype, stream=stream,
                    params=rng.choice(["bf16", "f32"]), post=post, gate=gate, gates=gates,
                    scale=rng.choice([1.0, 0.5, 0.22]), pre=pre, backward=rng.random() < 0.6)
    if op == "act":
        inter = _log_int(rng, 32, 14336)
        if rng.random() < 0.6:
            inter = -(-inter // 8) * 8
        dtype = rng.choice(["bf16", "f32"])
        most = 32768 * 14336 // (inter * (2 if dtype == "f32" else 1))
        return dict(op=op, rows=_log_int(rng, 1, min(65536, most)), inter=inter, dtype=dtype,
                    act=rng.choice(["silu", "silu", "relu"]), backward=rng.random() < 0.6)
    hidden = _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        hidden = -(-hidden // 8) * 8
    experts = _log_int(rng, 4, 128)
    top_k = rng.randint(1, min(8, experts))
    dtype = rng.choice(["bf16", "f32"])
    most = 16384 * 4096 * 2 // (hidden * top_k * (2 if dtype == "f32" else 1))
    tokens = _log_int(rng, 1, min(32768, most))
    cap = rng.random() < 0.3
    capacity = -(-int(1.1 * tokens * top_k / experts + 1) // ROWS) * ROWS if cap else 0
    return dict(op=op, tokens=tokens, hidden=hidden, experts=experts, top_k=top_k,
                capacity=capacity, dtype=dtype, out=rng.choice(["bf16", "f32"]),
                backward=rng.random() < 0.6)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    """Bytes and operations.  Where a case has a backward pass it is a call of
    its own, long after the forward pass in a program: it reads what it needs
    once more."""
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        es = _size(case["dtype"])
        # logits, bias; ids, weights and token rows; row tables; experts' ranges
        b = T * E * es + 4 * E * case["bias"] + 12 * T * k + 8 * _table_rows(case) + 8 * E
        f = T * E * (k + 8)
        if case["backward"]:
            # ids, weights and their gradients in, logit gradients out; softmax
            # without renormalisation needs all logits, else the chosen ones do
            dense = case["scoring"] == "softmax" and not case["renormalize"]
            b += 12 * T * k + T * E * es + (T * E if dense else T * k) * es
            f += 4 * T * (E if dense else k)
        return {"bytes": b, "flops": f}
    if op == "norm":
        T, H = case["tokens"], case["hidden"]
        a, s, p = (_size(case[n]) for n in ("dtype", "stream", "params"))
        params = H * p * (case["post"] + case["pre"] + (case["gates"] if case["gate"] != "none"
                                                        else 0))
        # x and the residual in, the stream out, the next block's input out
        b = T * H * (a + 2 * s + a * case["pre"]) + params
        f = T * H * 8
        if case["backward"]:
            # x, the residual, both gradients in; their gradients out
            b += T * H * (a + s + s + a * case["pre"] + a + s) + 2 * params
            f += T * H * 24
        return {"bytes": b, "flops": f}
    if op == "act":
        n = case["rows"] * case["inter"]
        a = _size(case["dtype"])
        b, f = n * 3 * a, n * 6
        if case["backward"]:
            # the checkpoint out and in again, h's gradient in, the input's out
            b += 2 * (2 * n * 33 / 32) + n * 3 * a
            f += n * 22
        return {"bytes": b, "flops": f}
    T, H, k = case["tokens"], case["hidden"], case["top_k"]
    a, o = _size(case["dtype"]), _size(case["out"])
    pairs = T * k
    if case["capacity"]:
        pairs = min(pairs, case["experts"] * case["capacity"])
    b, f = pairs * H * a + T * H * o + 8 * T * k, 2 * pairs * H
    if case["backward"]:
        # y's gradient and the rows in, the rows' gradient out
        b += T * H * o + pairs * H * a + _table_rows(case) * (H * a + 4) + 12 * T * k
        f += 3 * pairs * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(g, rows, cols, dtype):
    """Rows with a few strong channels, as a model's hidden states have."""
    chan = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    out = torch.empty((rows, cols), dtype=dtype, device="cuda")
    for r in range(0, rows, 4096):      # (in pieces: the fp32 draws of a large one are large)
        n = min(4096, rows - r)
        out[r:r + n] = torch.randn((n, cols), generator=g, device="cuda") * chan
    return out


def _up(n, m):
    return -(-n // m) * m


def _table_rows(case):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    return E * case["capacity"] if case["capacity"] else (T * k + E * (ROWS - 1)) // ROWS * ROWS


def _tables(ids, E, cap, M):
    """The experts' ranges and which pair sits in which row, for ids [T, k]."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    hot = (torch.arange(E, device=ids.device)[:, None] == flat).to(torch.int32)
    before = hot.cumsum(1)
    pos = before.gather(0, flat[None])[0] - 1
    count = hot.sum(1)
    if cap:
        first = torch.arange(E, device=ids.device) * cap
        kept, count = pos < cap, count.clamp_max(cap)
    else:
        span = (count + ROWS - 1) // ROWS * ROWS
        first, kept = span.cumsum(0) - span, pos >= 0
    row = torch.where(kept, first[flat] + pos, -1)
    i = torch.arange(T * k, device=ids.device)
    at = torch.where(kept, row, M)     # dropped pairs land in a spare last entry
    row_token = torch.full((M + 1,), -1, dtype=torch.int64, device=ids.device)
    row_slot = torch.zeros((M + 1,), dtype=torch.int64, device=ids.device)
    row_token[at] = i // k
    row_slot[at] = i % k
    return dict(row_token=row_token[:M].int(), row_slot=row_slot[:M].int(),
                token_row=row.reshape(T, k).int(), expert_first=first.int(),
                expert_rows=count.int())


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        st["logits"] = _randn(g, (T, E), 1.5, DTYPES[case["dtype"]])
        # as large as balancing makes it: a fraction of the scores' own spread
        spread = 0.05 if case["scoring"] == "sigmoid" else 0.5 / E
        st["bias"] = _randn(g, (E,), spread) if case["bias"] else None
        if case["backward"]:
            st["dweights"] = _randn(g, (T, k))
    elif op == "norm":
        T, H = case["tokens"], case["hidden"]
        dt, sd, pd = (DTYPES[case[n]] for n in ("dtype", "stream", "params"))
        st["x"] = _activations(g, T, H, dt)
        st["residual"] = _activations(g, T, H, sd)
        st["post"] = (1 + _randn(g, (H,), 0.1)).to(pd) if case["post"] else None
        st["pre"] = (1 + _randn(g, (H,), 0.1)).to(pd) if case["pre"] else None
        st["gate"] = None
        if case["gate"] == "channel":
            st["gate"] = _randn(g, (H,), 0.5, pd)
        elif case["gate"] != "none":
            st["gate"] = _randn(g, (case["gates"], H), 0.5, pd)
        if case["backward"]:
            st["dstream"] = _randn(g, (T, H), 1.0, sd)
            st["dy"] = _randn(g, (T, H), 1.0, dt) if case["pre"] else None
    elif op == "act":
        R, I, dt = case["rows"], case["inter"], DTYPES[case["dtype"]]
        st["u"] = _activations(g, R, 2 * I, dt)
        if case["backward"]:
            st["dh"] = _activations(g, R, I, dt)
    else:
        T, H, E, k = (case[n] for n in ("tokens", "hidden", "experts", "top_k"))
        M, dt = _table_rows(case), DTYPES[case["dtype"]]
        ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k]
        st.update(_tables(ids, E, case["capacity"], M))
        w = torch.rand((T, k), generator=g, device="cuda") + 0.1
        st["weights"] = w / w.sum(1, keepdim=True)
        st["rows"] = _activations(g, M, H, dt)
        # (nothing wrote the rows that hold no token)
        st["rows"][st["row_token"] < 0] = float("nan")
        if case["backward"]:
            st["dy"] = _randn(g, (T, H), 1.0, DTYPES[case["out"]])
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "norm": _plain_norm, "act": _plain_act,
            "combine": _plain_combine}[state["case"]["op"]](state)


def _run_own(st):
    from communication_overlap_gb300 import block, moe
    case = st["case"]
    op = case["op"]
    if op == "route":
        r = moe.route(st["logits"], case["top_k"], renormalize=case["renormalize"],
                      capacity=case["capacity"], scoring=case["scoring"], bias=st["bias"],
                      groups=case["groups"], top_groups=case["top_groups"],
                      group_top=case["group_top"], scale=case["scale"])
        out = dict(ids=r.ids, weights=r.weights, row_token=r.row_token, row_slot=r.row_slot,
                   token_row=r.token_row, expert_first=r.expert_first,
                   expert_rows=r.expert_rows)
        if case["backward"]:
            out["dlogits"] = moe.route_backward(
                st["logits"], r.ids, r.weights, st["dweights"],
                renormalize=case["renormalize"], scoring=case["scoring"], scale=case["scale"])
        return out
    if op == "norm":
        how = dict(post_gain=st["post"], gate=st["gate"], scale=case["scale"],
                   pre_gain=st["pre"])
        n = block.norm(st["x"], st["residual"], eps=EPS, **how)
        out = dict(stream=n.stream, y=n.y)
        if case["backward"]:
            d = block.norm_backward(st["x"], st["residual"], n, dstream=st["dstream"],
                                    dy=st["dy"], **how)
            out.update(dx=d.x, dresidual=d.residual, dpost=d.post_gain, dgate=d.gate,
                       dpre=d.pre_gain)
        return {name: t for name, t in out.items() if t is not None}
    if op == "act":
        h, kept = block.activate(st["u"], act=case["act"], checkpoint=case["backward"])
        if not case["backward"]:
            return dict(h=h)
        return dict(h=h, du=block.activate_backward(st["dh"], kept))
    y = block.combine(st["rows"], st["token_row"], st["weights"],
                      out_dtype=DTYPES[case["out"]])
    if not case["backward"]:
        return dict(y=y)
    drows, dweights = block.combine_backward(st["dy"], st["rows"], st["token_row"],
                                             st["row_token"], st["weights"])
    return dict(y=y, drows=drows, dweights=dweights)


def _choose(x, k):
    """The k largest of each row, ties to the lowest index (elementary ops)."""
    n = x.shape[1]
    iota = torch.arange(n, device=x.device)
    left, ids = x.clone(), []
    for _ in range(k):
        m = left.amax(1, keepdim=True)
        i = torch.where(left == m, iota, n).amin(1)
        ids.append(i)
        left.scatter_(1, i[:, None], float("-inf"))
    return torch.stack(ids, 1)


def _plain_route(st):
    case = st["case"]
    T, E, k, G = (case[n] for n in ("tokens", "experts", "top_k", "groups"))
    sigmoid = case["scoring"] == "sigmoid"
    # the choice: a score and a bias nearly tie often enough to need 64 bits
    x = st["logits"].double()
    if sigmoid:
        c = 1 / (1 + torch.exp(-x))
    else:
        c = torch.exp(x - x.amax(1, keepdim=True))
        c = c / c.sum(1, keepdim=True)
    if st["bias"] is not None:
        c = c + st["bias"].double()
    if G > 1:
        by_group = c.view(T, G, E // G)
        n = min(case["group_top"], E // G)
        top = _choose(by_group.reshape(T * G, E // G), n)
        score = by_group.reshape(T * G, E // G).gather(1, top).sum(1).view(T, G)
        keep = torch.zeros((T, G), dtype=torch.bool, device=c.device)
        keep.scatter_(1, _choose(score, case["top_groups"]), True)
        c = torch.where(keep[:, :, None], by_group, float("-inf")).reshape(T, E)
    ids = _choose(c, k)
    # the weights, in 32 bits
    x = st["logits"].float()
    if sigmoid:
        s = 1 / (1 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    chosen = s.gather(1, ids)
    share = chosen / chosen.sum(1, keepdim=True) if case["renormalize"] else chosen
    out = dict(ids=ids.int(), weights=share * case["scale"],
               **_tables(ids, E, case["capacity"], _table_rows(case)))
    if case["backward"]:
        g = st["dweights"] * case["scale"]
        d = torch.zeros_like(x)
        if case["renormalize"]:
            ds = (g - (share * g).sum(1, keepdim=True)) * share
            d.scatter_(1, ids, ds * (1 - chosen) if sigmoid else ds)
        elif sigmoid:
            d.scatter_(1, ids, g * chosen * (1 - chosen))
        else:
            d = s * (d.scatter_(1, ids, g) - (chosen * g).sum(1, keepdim=True))
        out["dlogits"] = d.to(st["logits"].dtype)
    return out


def _plain_norm(st):
    case = st["case"]
    dt, sd, pd = (DTYPES[case[n]] for n in ("dtype", "stream", "params"))
    B, scale = case["gates"], case["scale"]
    x, res = st["x"].float(), st["residual"].float()
    T, H = x.shape
    post = None if st["post"] is None else st["post"].float()
    pre = None if st["pre"] is None else st["pre"].float()
    gate = scale
    if st["gate"] is not None:
        gate = st["gate"].float().view(B, 1, H).expand(B, T // B, H).reshape(T, H) * scale
    u = x
    if post is not None:
        r1 = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        xn = x * r1
        u = xn * post
    s = res + gate * u
    out = dict(stream=s.to(sd))
    if pre is not None:
        r2 = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
        sn = s * r2
        out["y"] = (sn * pre).to(dt)
    if not case["backward"]:
        return out
    d = st["dstream"].float()
    if pre is not None:
        dy = st["dy"].float()
        out["dpre"] = (dy * sn).sum(0).to(pd)
        e = dy * pre
        d = d + r2 * (e - sn * (e * sn).mean(1, keepdim=True))
    out["dresidual"] = d.to(sd)
    if st["gate"] is not None:
        dgate = (d * u * scale).view(B, T // B, H).sum(1)
        out["dgate"] = dgate.view(st["gate"].shape).to(pd)
    e = gate * d
    if post is not None:
        out["dpost"] = (e * xn).sum(0).to(pd)
        e = e * post
        e = r1 * (e - xn * (e * xn).mean(1, keepdim=True))
    out["dx"] = e.to(dt)
    return out


def _in_eight_bits(x):
    """The values that x [rows, cols] stands for in the 8-bit form, in 32 bits:
    per 32 values a step of 2^(floor(log2 max |x|) - 6), at least 2^-127."""
    R, C = x.shape
    b = torch.zeros((R, _up(C, BLOCK)), device=x.device)
    b[:, :C] = x
    b = b.view(R, -1, BLOCK)
    e = ((b.abs().amax(-1).view(torch.int32) >> 23) - 6).clamp_min(0)[..., None]
    step = torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23).view(torch.float32)
    inverse = ((254 - e.clamp_max(253)) << 23).view(torch.float32)
    q = torch.round(b * inverse).clamp_(-127, 127) * step
    return q.view(R, -1)[:, :C]


def _plain_act(st):
    case = st["case"]
    I, dt = case["inter"], st["u"].dtype
    u = st["u"].float()
    gate, up = u[:, :I], u[:, I:]
    if case["act"] == "silu":
        h = gate / (1 + torch.exp(-gate)) * up
    else:
        h = torch.where(gate > 0, gate, 0.0) * up
    h = h.to(dt)
    if not case["backward"]:
        return dict(h=h)
    gate, up = _in_eight_bits(gate), _in_eight_bits(up)
    dh = st["dh"].float()
    du = torch.empty_like(st["u"])
    if case["act"] == "silu":
        s = 1 / (1 + torch.exp(-gate))
        du[:, :I] = dh * up * s * (1 + gate * (1 - s))
        du[:, I:] = dh * gate * s
    else:
        on = gate > 0
        du[:, :I] = torch.where(on, dh * up, 0.0)
        du[:, I:] = torch.where(on, dh * gate, 0.0)
    return dict(h=h, du=du)


def _plain_combine(st):
    case = st["case"]
    rows, token_row, w = st["rows"], st["token_row"].long(), st["weights"]
    has = token_row >= 0
    part = rows[token_row.clamp_min(0)].float() * w[..., None]
    out = dict(y=torch.where(has[..., None], part, 0.0).sum(1).to(DTYPES[case["out"]]))
    if not case["backward"]:
        return out
    t, slot = torch.nonzero(has, as_tuple=True)
    r = token_row[t, slot]
    dy = st["dy"].float()[t]
    drows = torch.zeros_like(rows)
    drows[r] = (dy * w[t, slot][:, None]).to(rows.dtype)
    dw = torch.zeros_like(w)
    dw[t, slot] = (dy * rows[r].float()).sum(1)
    out.update(drows=drows, dweights=dw)
    return out


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    with torch.enable_grad():
        return {"route": _exact_route, "norm": _exact_norm, "act": _exact_act,
                "combine": _exact_combine}[case["op"]](st)


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _exact_route(st):
    case = st["case"]
    T, E, k, G, cap = (case[n] for n in ("tokens", "experts", "top_k", "groups", "capacity"))
    x = _leaf(st["logits"])
    scores = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
    choice = scores.detach().clone()
    if st["bias"] is not None:
        choice += st["bias"].double()
    if G > 1:
        per = E // G
        ranked = choice.view(T, G, per).sort(dim=2, descending=True).values
        score = ranked[:, :, :case["group_top"]].sum(2)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices
        for g in range(case["top_groups"], G):
            cols = order[:, g:g + 1] * per + torch.arange(per, device="cuda")
            choice.scatter_(1, cols, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(scores, 1, ids)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    host = ids.cpu().reshape(-1)
    order = torch.sort(host, stable=True).indices
    counts = torch.bincount(host, minlength=E).tolist()
    M = _table_rows(case)
    row_token, row_slot = torch.full((M,), -1), torch.zeros(M, dtype=torch.int64)
    token_row = torch.full((T * k,), -1)
    first, rows, taken, at = [], [], 0, 0
    for e in range(E):
        mine = order[taken:taken + counts[e]]
        taken += counts[e]
        if cap:
            at, mine = e * cap, mine[:cap]
        n = len(mine)
        row_token[at:at + n] = mine // k
        row_slot[at:at + n] = mine % k
        token_row[mine] = torch.arange(at, at + n)
        first.append(at)
        rows.append(n)
        at += _up(n, ROWS)
    dev = lambda t: torch.as_tensor(t).int().cuda()
    out = dict(ids=ids.int(), weights=w.detach(), row_token=dev(row_token),
               row_slot=dev(row_slot), token_row=dev(token_row.view(T, k)),
               expert_first=dev(first), expert_rows=dev(rows))
    if case["backward"]:
        out["dlogits"], = torch.autograd.grad(w, x, st["dweights"].double())
    return out


def _exact_norm(st):
    case = st["case"]
    x, res, post, pre, gate = (_leaf(st[n]) for n in ("x", "residual", "post", "pre", "gate"))
    T, H = x.shape

    def normed(v, gain):
        return v / torch.sqrt((v ** 2).mean(1, keepdim=True) + EPS) * gain

    u = x if post is None else normed(x, post)
    if gate is not None:
        B = case["gates"]
        u = (u.reshape(B, T // B, H) * gate.reshape(B, 1, H)).reshape(T, H)
    s = res + case["scale"] * u
    y = None if pre is None else normed(s, pre)
    out = dict(stream=s.detach())
    if y is not None:
        out["y"] = y.detach()
    if not case["backward"]:
        return out
    into = dict(dx=x, dresidual=res, dpost=post, dgate=gate, dpre=pre)
    into = {name: t for name, t in into.items() if t is not None}
    ends, grads = [s], [st["dstream"].double()]
    if y is not None:
        ends.append(y)
        grads.append(st["dy"].double())
    got = torch.autograd.grad(ends, list(into.values()), grads)
    out.update(zip(into, got))
    return out


def _exact_act(st):
    case = st["case"]
    R, I = case["rows"], case["inter"]
    f = torch.nn.functional.silu if case["act"] == "silu" else torch.relu
    h = torch.empty((R, I), dtype=torch.float64, device="cuda")
    du = torch.empty((R, 2 * I), dtype=torch.float64, device="cuda") if case["backward"] else None
    for r in range(0, R, 2048):
        part = slice(r, min(R, r + 2048))
        gate, up = st["u"][part].double().split(I, dim=1)
        h[part] = f(gate) * up
        if not case["backward"]:
            continue
        kept = []
        for v in (gate, up):
            b = torch.nn.functional.pad(v, (0, -I % BLOCK)).view(len(v), -1, BLOCK)
            top = b.abs().amax(-1, keepdim=True)
            exponent = torch.where(top == 0, -127, (torch.frexp(top).exponent - 7).clamp_min(-127))
            step = ((exponent.long() + 1023) << 52).view(torch.float64)     # 2^exponent
            q = torch.round(b / step).clamp(-127, 127) * step
            kept.append(q.view(len(v), -1)[:, :I].contiguous().requires_grad_())
        got = torch.autograd.grad(f(kept[0]) * kept[1], kept, st["dh"][part].double())
        du[part] = torch.cat(got, 1)
    return dict(h=h, du=du) if case["backward"] else dict(h=h)


def _exact_combine(st):
    case = st["case"]
    # the rows that hold a token, and for each pair which of them it is
    held = torch.nonzero(st["row_token"] >= 0)[:, 0]
    at = torch.full((len(st["row_token"]),), len(held), device="cuda")
    at[held] = torch.arange(len(held), device="cuda")
    rows, w = _leaf(st["rows"][held]), _leaf(st["weights"])
    # a last row of zeros for the pairs that have none
    full = torch.cat((rows, torch.zeros((1, rows.shape[1]), dtype=rows.dtype, device="cuda")))
    at = torch.cat((at, at.new_tensor([len(held)])))        # (index -1: that row)
    pick = at[st["token_row"].long()]
    y = sum(full[pick[:, s]] * w[:, s:s + 1] for s in range(case["top_k"]))
    out = dict(y=y.detach())
    if case["backward"]:
        drows, dw = torch.autograd.grad(y, (rows, w), st["dy"].double())
        out["drows"] = torch.zeros(st["rows"].shape, dtype=torch.float64, device="cuda")
        out["drows"][held] = drows
        out["dweights"] = dw
    return out

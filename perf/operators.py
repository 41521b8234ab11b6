"""The mixture-of-experts operators: what is measured of them.

Four operators, as a serving or training program of the expert layer meets
them:

  route     router logits -> top-k experts, weights and the row tables of the
            grouped products, and the gradient of the weights
  quantize  bf16 / fp32 matrices -> microscaled 4-bit blocks (E2M1 codes, one
            power-of-two scale per 32 values), by rows, by gathered rows or
            transposed, and back to the values they stand for
  gemm      the product of two such matrices, plain or one per expert
  few       a whole expert layer (router, gated experts, combination) for a
            few tokens, with bf16 or 4-bit weights

``own = False`` computes each in its plain form (elementary torch operations
in 32 bits, rounded once at the end), ``own = True`` by the calls of
``communication_overlap_gb300.moe``.
"""
import math

import torch

own = False

BLOCK = 32          # values that share a scale
ROWS = 128          # rows of a block of scales, and an expert's row alignment
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token choosing 2 of 8 experts: pure latency
        dict(name="route_one_token", op="route", tokens=1, experts=8, top_k=2, dtype="f32",
             renormalize=True, capacity=0, backward=False),
        # a training batch over many small experts, with the gradient
        dict(name="route_train_128", op="route", tokens=16384, experts=128, top_k=8,
             dtype="bf16", renormalize=False, capacity=0, backward=True),
        # the All-to-All layer's tokens gathered into their experts' rows
        dict(name="quantize_gather", op="quantize", rows=32768, cols=4096, tokens=16384,
             dtype="bf16", transpose=False),
        # an expert's weight turned for the gradient of its input
        dict(name="quantize_transposed", op="quantize", rows=4096, cols=14336, tokens=0,
             dtype="bf16", transpose=True),
        # a small odd matrix in fp32: ragged rows, a ragged last block
        dict(name="quantize_odd", op="quantize", rows=333, cols=1000, tokens=0, dtype="f32",
             transpose=False),
        # one token through the up-projection: bound by reading the weight
        dict(name="gemm_one_row", op="gemm", rows=1, n=14336, k=4096, experts=1, out="bf16"),
        # the backward product of the ReduceScatter configuration, fp32 out
        dict(name="gemm_backward", op="gemm", rows=8192, n=4096, k=2752, experts=1, out="f32"),
        # the All-to-All expert layer: 32768 routed rows over 8 experts
        dict(name="gemm_experts", op="gemm", rows=32768, n=14336, k=4096, experts=8,
             out="bf16"),
        # the same layer's gated form for one generated token, bf16 weights
        dict(name="few_bf16_1", op="few", tokens=1, hidden=4096, inter=14336, experts=8,
             top_k=2, weights="bf16", renormalize=True),
        # a batch of generated tokens that reaches every expert
        dict(name="few_bf16_48", op="few", tokens=48, hidden=4096, inter=14336, experts=8,
             top_k=2, weights="bf16", renormalize=True),
        # one generated token with 4-bit weights
        dict(name="few_mx_1", op="few", tokens=1, hidden=4096, inter=14336, experts=8,
             top_k=2, weights="mx", renormalize=True),
        # a few tokens over many small experts of an odd width
        dict(name="few_mx_7_small", op="few", tokens=7, hidden=2048, inter=1416, experts=60,
             top_k=4, weights="mx", renormalize=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer in [lo, hi], uniform in its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, (v + step // 2) // step * step))
    return v - step if v == 3072 else v


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "few"])
    if op == "route":
        experts = _log_int(rng, 4, 256)
        tokens = _log_int(rng, 1, min(32768, 16384 * 128 // experts))
        top_k = rng.randint(1, min(8, experts))
        cap = rng.random() < 0.3
        # a capacity of 1.25 times the mean load, in whole tile rows
        capacity = -(-int(1.25 * tokens * top_k / experts + 1) // ROWS) * ROWS if cap else 0
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k,
                    dtype=rng.choice(["bf16", "f32"]), renormalize=rng.random() < 0.5,
                    capacity=capacity, backward=rng.random() < 0.5)
    if op == "quantize":
        cols = _log_int(rng, 32, 14336)
        rows = _log_int(rng, 1, min(32768, 32768 * 4096 // (2 * cols)))
        transpose = rng.random() < 0.4
        gather = not transpose and rng.random() < 0.5
        return dict(op=op, rows=rows, cols=cols, tokens=max(1, rows // 2) if gather else 0,
                    dtype=rng.choice(["bf16", "f32"]), transpose=transpose)
    if op == "gemm":
        experts = rng.choice([1, 1, 4, 8, 16])
        n = _log_int(rng, 64, 14336)
        k = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, min(32768, 32768 * 14336 * 4096 // (n * k)))
        return dict(op=op, rows=rows, n=n, k=k, experts=experts,
                    out=rng.choice(["bf16", "f32"]))
    hidden = _log_int(rng, 512, 8192, 8)
    experts = _log_int(rng, 4, 128)
    # no more weights than the largest listed layer
    inter = _log_int(rng, 256, min(14336, 8 * 14336 * 4096 // (experts * hidden)), 8)
    return dict(op=op, tokens=_log_int(rng, 1, 64), hidden=hidden, inter=inter,
                experts=experts, top_k=rng.randint(1, min(8, experts)),
                weights=rng.choice(["bf16", "mx"]), renormalize=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        es = 2 if case["dtype"] == "bf16" else 4
        M = _table_rows(case)
        # logits; ids, weights and token rows; row tables; experts' ranges
        b = T * E * es + 12 * T * k + 8 * M + 8 * E
        f = T * E * (k + 4)
        if case["backward"]:
            b += 4 * T * k + T * E * es     # weight gradients in, logit gradients out
            f += 4 * T * E
        return {"bytes": b, "flops": f}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        es = 2 if case["dtype"] == "bf16" else 4
        src = case["tokens"] if case["tokens"] else R
        # the source once, the 4-bit form, the values it stands for
        return {"bytes": src * C * es + R * C * 17 / 32 + R * C * es, "flops": 4 * R * C}
    if op == "gemm":
        R, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        E = min(E, R)
        es = 2 if case["out"] == "bf16" else 4
        return {"bytes": (R + E * N) * K * 17 / 32 + R * N * es, "flops": 2 * R * N * K}
    T, H, I, E, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "top_k"))
    # experts that T tokens reach on average
    reached = E * (1 - (1 - k / E) ** T)
    per = 2 if case["weights"] == "bf16" else 17 / 32
    return {"bytes": reached * 3 * H * I * per + 2 * E * H + 4 * T * H,
            "flops": 2 * T * k * 3 * H * I + 2 * T * E * H}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(g, rows, cols, dtype):
    """Rows with a few strong channels, as a model's hidden states have."""
    chan = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return (torch.randn((rows, cols), generator=g, device="cuda") * chan).to(dtype)


def _up(n, m):
    return -(-n // m) * m


def _block_values(x):
    """(codes 0..15, biased scale exponents) of x [rows, cols], cols % 32 == 0."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    e = b.abs().amax(-1).view(torch.int32) >> 23
    s = torch.where(e == 255, e, (e - 2).clamp_min(0))
    inv = ((254 - s.clamp_max(252)) << 23).view(torch.float32)
    v = b * inv[..., None]
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    c = c + 8 * torch.signbit(v)
    return c.reshape(x.shape[0], -1).to(torch.uint8), s.to(torch.uint8)


def _values(codes, scales):
    """fp32 values of codes [rows, cols] and scales [rows, cols / 32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    s = scales.to(torch.int32)
    scale = torch.where(s == 0, torch.full_like(s, 1 << 22), s << 23).view(torch.float32)
    scale = torch.where(s == 255, torch.full_like(scale, float("nan")), scale)
    v = table[codes.int()].reshape(codes.shape[0], -1, BLOCK) * scale[..., None]
    return v.reshape(codes.shape[0], -1)


def _packed(x):
    """A matrix [rows, cols] in the library's 4-bit layout: codes two to a
    byte, rows padded to 128 and columns to 128 with zeros; scales in blocks
    of 128 rows x 4 (512 bytes, row r's at (r % 32) * 16 + (r // 32) * 4)."""
    R, C = x.shape
    Rp, Cp = _up(R, ROWS), _up(C, 128)
    full = torch.zeros((Rp, Cp), device=x.device, dtype=torch.float32)
    full[:R, :C] = x
    c, s = _block_values(full)
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    scales = s.view(Rp // ROWS, 4, 32, Cp // 128, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes.contiguous(), scales.view(-1)


def _unpacked(codes, scales, rows, cols):
    Rp, Cp = codes.shape[0], codes.shape[1] * 2
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(Rp, Cp)
    s = scales.view(Rp // ROWS, Cp // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(Rp, Cp // 32)
    return c, s, rows, cols


def _decode(codes, scales, rows, cols):
    c, s, _, _ = _unpacked(codes, scales, rows, cols)
    return _values(c, s)[:rows, :cols]


def _stack(g, count, rows, cols, scale):
    """`count` matrices of N(0, scale) in the 4-bit layout, one after another."""
    parts = [_packed(_randn(g, (rows, cols), scale)) for _ in range(count)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _table_rows(case):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    return E * case["capacity"] if case["capacity"] else (T * k + E * (ROWS - 1)) // ROWS * ROWS


def _group_rows(case):
    """Rows of each expert: uneven, summing to the case's rows."""
    R, E = case["rows"], case["experts"]
    share = [1.0 + 0.5 * math.sin(1 + 2.3 * e) for e in range(E)]
    cuts = [int(R * sum(share[:e]) / sum(share)) for e in range(E)] + [R]
    return [cuts[e + 1] - cuts[e] for e in range(E)]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        st["logits"] = _randn(g, (T, E), 1.5, DTYPES[case["dtype"]])
        if case["backward"]:
            st["dweights"] = _randn(g, (T, k))
    elif op == "quantize":
        R, C, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        if case["transpose"]:
            st["x"] = _activations(g, C, R, dt)
        else:
            st["x"] = _activations(g, case["tokens"] or R, C, dt)
        st["index"] = None
        if case["tokens"]:
            idx = torch.randint(0, case["tokens"], (R,), generator=g, device="cuda")
            empty = torch.rand(R, generator=g, device="cuda") < 0.02
            st["index"] = torch.where(empty, -1, idx).to(torch.int32)
    elif op == "gemm":
        R, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        rows = _group_rows(case)
        first, at = [], 0
        for r in rows:
            first.append(at)
            at += _up(r, ROWS)
        st["span"] = span = at if E > 1 else R
        x = _activations(g, span, K, torch.float32)
        st["a"] = _packed(x)
        st["b"] = _stack(g, E, N, K, 1.0 / math.sqrt(K))
        st["groups"] = list(zip(first, rows)) if E > 1 else [(0, R)]
        st["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        st["rows"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        # the rows between the experts' ranges belong to no expert
        st["out"] = torch.zeros((span, N), dtype=DTYPES[case["out"]], device="cuda")
        if own:
            from communication_overlap_gb300 import moe
            st["qa"] = moe.MxTensor(st["a"][0], st["a"][1], 1, span, K)
            st["qb"] = moe.MxTensor(st["b"][0], st["b"][1], E, N, K)
    else:
        T, H, I, E = (case[n] for n in ("tokens", "hidden", "inter", "experts"))
        bf = torch.bfloat16
        st["x"] = _activations(g, T, H, bf)
        st["router"] = _randn(g, (E, H), 1.5 / math.sqrt(H), bf)
        if case["weights"] == "bf16":
            st["w1"] = torch.empty((E, 2 * I, H), dtype=bf, device="cuda")
            st["w2"] = torch.empty((E, H, I), dtype=bf, device="cuda")
            for e in range(E):
                st["w1"][e] = _randn(g, (2 * I, H), 1 / math.sqrt(H))
                st["w2"][e] = _randn(g, (H, I), 1 / math.sqrt(I))
        else:
            st["w1"] = _stack(g, E, 2 * I, H, 1 / math.sqrt(H))
            st["w2"] = _stack(g, E, H, I, 1 / math.sqrt(I))
        if own:
            from communication_overlap_gb300 import moe
            w1, w2 = st["w1"], st["w2"]
            if case["weights"] == "mx":
                w1 = moe.MxTensor(w1[0], w1[1], E, 2 * I, H)
                w2 = moe.MxTensor(w2[0], w2[1], E, H, I)
            st["layer"] = moe.FewTokenLayer(st["router"], w1, w2, case["top_k"],
                                            renormalize=case["renormalize"])
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "quantize": _plain_quantize, "gemm": _plain_gemm,
            "few": _plain_few}[state["case"]["op"]](state)


def _run_own(st):
    from communication_overlap_gb300 import moe
    case = st["case"]
    op = case["op"]
    if op == "route":
        r = moe.route(st["logits"], case["top_k"], renormalize=case["renormalize"],
                      capacity=case["capacity"])
        out = dict(ids=r.ids, weights=r.weights, row_token=r.row_token, row_slot=r.row_slot,
                   token_row=r.token_row, expert_first=r.expert_first,
                   expert_rows=r.expert_rows)
        if case["backward"]:
            out["dlogits"] = moe.route_backward(st["logits"], r.ids, r.weights, st["dweights"],
                                                renormalize=case["renormalize"])
        return out
    if op == "quantize":
        q = moe.quantize(st["x"], transpose=case["transpose"], row_index=st["index"])
        return moe.dequantize(q, st["x"].dtype)
    if op == "gemm":
        if case["experts"] == 1:
            return moe.mx_gemm(st["qa"], st["qb"], out=st["out"])
        return moe.mx_gemm(st["qa"], st["qb"], out=st["out"], group_first=st["first"],
                           group_rows=st["rows"])
    return st["layer"](st["x"])


def _choose(x, k):
    """The k largest of each row, ties to the lowest index (elementary ops)."""
    E = x.shape[1]
    iota = torch.arange(E, device=x.device)
    left, ids = x.clone(), []
    for _ in range(k):
        m = left.amax(1, keepdim=True)
        i = torch.where(left == m, iota, E).amin(1)
        ids.append(i)
        left.scatter_(1, i[:, None], float("-inf"))
    return torch.stack(ids, 1)


def _plain_weights(logits, ids, renormalize):
    x = logits.float()
    p = torch.exp(x - x.amax(1, keepdim=True))
    c = p.gather(1, ids)
    return c / (c if renormalize else p).sum(1, keepdim=True), p / p.sum(1, keepdim=True)


def _plain_route(st):
    case = st["case"]
    T, E, k, cap = case["tokens"], case["experts"], case["top_k"], case["capacity"]
    x = st["logits"].float()
    ids = _choose(x, k)
    w, p = _plain_weights(x, ids, case["renormalize"])
    flat = ids.reshape(-1)
    hot = (torch.arange(E, device=x.device)[:, None] == flat).to(torch.int32)
    before = hot.cumsum(1)
    pos = before.gather(0, flat[None])[0] - 1
    count = hot.sum(1)
    M = _table_rows(case)
    if cap:
        first = torch.arange(E, device=x.device) * cap
        kept, count = pos < cap, count.clamp_max(cap)
    else:
        span = (count + ROWS - 1) // ROWS * ROWS
        first, kept = span.cumsum(0) - span, pos >= 0
    row = torch.where(kept, first[flat] + pos, -1)
    i = torch.arange(T * k, device=x.device)
    at = torch.where(kept, row, M)     # dropped pairs land in a spare last entry
    row_token = torch.full((M + 1,), -1, dtype=torch.int64, device=x.device)
    row_slot = torch.zeros((M + 1,), dtype=torch.int64, device=x.device)
    row_token[at] = i // k
    row_slot[at] = i % k
    out = dict(ids=ids.int(), weights=w, row_token=row_token[:M].int(),
               row_slot=row_slot[:M].int(), token_row=row.reshape(T, k).int(),
               expert_first=first.int(), expert_rows=count.int())
    if case["backward"]:
        g = st["dweights"]
        dot = (w * g).sum(1, keepdim=True)
        if case["renormalize"]:
            d = torch.zeros_like(x).scatter_(1, ids, w * (g - dot))
        else:
            d = p * (torch.zeros_like(x).scatter_(1, ids, g) - dot)
        out["dlogits"] = d.to(st["logits"].dtype)
    return out


def _source(st):
    x = st["x"]
    if st["case"]["transpose"]:
        x = x.t()
    if st["index"] is not None:
        i = st["index"].long()
        x = x[i.clamp_min(0)] * (i >= 0)[:, None]
    return x


def _plain_quantize(st):
    x = _source(st).float()
    R, C = x.shape
    full = torch.zeros((R, _up(C, BLOCK)), device=x.device)
    full[:, :C] = x
    return _values(*_block_values(full))[:, :C].to(st["x"].dtype)


def _plain_gemm(st):
    case = st["case"]
    a = _decode(*st["a"], st["span"], case["k"])
    out = st["out"]
    for e, (r0, n) in enumerate(st["groups"]):
        if n:
            b = _decode(st["b"][0][e], st["b"][1][e], case["n"], case["k"])
            out[r0:r0 + n] = (a[r0:r0 + n] @ b.t()).to(out.dtype)
    return out


def _expert(st, e):
    case = st["case"]
    H, I = case["hidden"], case["inter"]
    if case["weights"] == "bf16":
        return st["w1"][e].float(), st["w2"][e].float()
    return (_decode(st["w1"][0][e], st["w1"][1][e], 2 * I, H),
            _decode(st["w2"][0][e], st["w2"][1][e], H, I))


def _plain_few(st):
    case = st["case"]
    I, E = case["inter"], case["experts"]
    x = st["x"].float()
    logits = x @ st["router"].float().t()
    ids = _choose(logits, case["top_k"])
    w, _ = _plain_weights(logits, ids, case["renormalize"])
    dense = torch.zeros_like(logits).scatter_(1, ids, w)
    y = torch.zeros_like(x)
    for e in range(E):
        w1, w2 = _expert(st, e)
        a = x @ w1.t()
        gate, up = a[:, :I], a[:, I:]
        h = gate / (1 + torch.exp(-gate)) * up
        y += dense[:, e:e + 1] * (h @ w2.t())
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = _inputs_only(case, seed)
    return {"route": _exact_route, "quantize": _exact_quantize, "gemm": _exact_gemm,
            "few": _exact_few}[case["op"]](st)


def _inputs_only(case, seed):
    """The inputs of prepare() without the framework's handles."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_choice(x, k, renormalize):
    """Experts, weights and probabilities by a stable descending sort."""
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(x, 1)
    w = torch.gather(p, 1, order)
    return order, (w / w.sum(1, keepdim=True) if renormalize else w), p


def _exact_route(st):
    case = st["case"]
    T, E, k, cap = case["tokens"], case["experts"], case["top_k"], case["capacity"]
    x = st["logits"].double()
    ids, w, p = _exact_choice(x, k, case["renormalize"])
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
    out = dict(ids=ids.int(), weights=w, row_token=dev(row_token), row_slot=dev(row_slot),
               token_row=dev(token_row.view(T, k)), expert_first=dev(first),
               expert_rows=dev(rows))
    if case["backward"]:
        # the Jacobian of softmax over the experts, or over the chosen ones
        g = st["dweights"].double()
        if case["renormalize"]:
            own_grad = w * g - w * (w * g).sum(1, keepdim=True)
            out["dlogits"] = torch.zeros_like(x).scatter(1, ids, own_grad)
        else:
            full = torch.zeros_like(x).scatter(1, ids, g)
            out["dlogits"] = p * full - p * (p * full).sum(1, keepdim=True)
    return out


def _power_of_two(e):
    """2^e in 64 bits, from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantize(st):
    x = _source(st).double()
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % BLOCK)).view(R, -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    exponent = (torch.frexp(top).exponent - 1 - 2).clamp_min(-127)
    exponent = torch.where(top == 0, torch.full_like(exponent, -127), exponent)
    unit = _power_of_two(exponent)
    u = b.abs() / unit
    step = torch.where(u < 2, 0.5, torch.where(u < 4, 1.0, 2.0)).double()
    q = (torch.round(u / step) * step).clamp_max(6.0)
    return (torch.copysign(q, b) * unit).view(R, -1)[:, :C]


def _exact_decode(codes, scales, rows, cols):
    c, s, _, _ = _unpacked(codes, scales, rows, cols)
    c, s = c[:rows].int(), s[:rows].int()
    m, e = (c & 1).double(), (c >> 1) & 3
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _power_of_two(e - 1))
    v = torch.where(c >= 8, -v, v).view(rows, -1, BLOCK)
    return (v * _power_of_two(s - 127)[..., None]).view(rows, -1)[:, :cols]


def _exact_gemm(st):
    case = st["case"]
    out = torch.zeros((st["span"], case["n"]), dtype=torch.float64, device="cuda")
    a = _exact_decode(*st["a"], st["span"], case["k"])
    for e, (r0, n) in enumerate(st["groups"]):
        b = _exact_decode(st["b"][0][e], st["b"][1][e], case["n"], case["k"])
        torch.matmul(a[r0:r0 + n], b.t(), out=out[r0:r0 + n])
    return out


def _exact_few(st):
    case = st["case"]
    H, I = case["hidden"], case["inter"]
    x = st["x"].double()
    ids, w, _ = _exact_choice(x @ st["router"].double().t(), case["top_k"],
                              case["renormalize"])
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        if case["weights"] == "bf16":
            w1, w2 = st["w1"][e].double(), st["w2"][e].double()
        else:
            w1 = _exact_decode(st["w1"][0][e], st["w1"][1][e], 2 * I, H)
            w2 = _exact_decode(st["w2"][0][e], st["w2"][1][e], H, I)
        gate, up = (x[tok] @ w1.t()).split(I, dim=1)
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, tok, (h @ w2.t()) * w[tok, slot][:, None])
    return y

"""Cases of two sets of operators around the routed expert FFN: the 8-bit integer form of its serving path, and the training
of its router.

``run`` computes an operator either from elementary torch operations in 32 bits (``own`` false; 64 for quotients next to a
rounding border) or through the library (``own`` true); ``exact`` computes the definition in 64 bits.

  * 8-bit integers: a row (one token's elements, or one output channel's weights) shares one scale s = amax / 127, rounded to
    32 bits; its codes are the integers nearest to x / s, ties to even, within +-127.  Products of codes are exact integers; a
    product's value is the integer sum times the token's and the channel's scale.  The routed FFN quantises the hidden rows
    silu(gate) * up between its two products, one scale per row over the whole row.
  * The router's training forward: softmax over the experts' logits, the k largest probabilities (equal ones: the lower expert
    first), the pairs and the tokens counted per expert, and two losses over the n tokens that count: balance =
    E / (k n) sum_e count_e mean_t p[t, e], and z = mean_t logsumexp(logits[t])^2.  Tokens that a mask leaves out (the padding
    of a batch, whatever their rows hold) get expert -1 and weight 0 and count nowhere.
  * Its backward pass: from the gradients of the routed weights (in the compact order that the expert FFN's backward pass
    leaves them in) and of the two losses, the gradients of the token rows and of the gate matrix.  Counts are constants.
  * The dispatch contract: pairs sorted by expert (stably), every expert's rows padded to (n // 128 + 1) * 128 rows, one
    expert id per 128-row block, routed weights in compact (unpadded) order.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}

# ---------------------------------------------------------------------------------------------------------------- cases


def _quant(name, batch, rows, cols, dtype):
    return {"name": name, "kind": "quantize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def _ffn(name, tokens, experts, top_k, hidden, inter, zipf=0.0):
    return {"name": name, "kind": "int8", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "inter": inter, "zipf": zipf}


def _router(kind, name, tokens, experts, top_k, hidden, left_out=0.0, add=False):
    case = {"name": name, "kind": kind, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "left_out": left_out}
    return dict(case, add=add) if kind == "backward" else case


def listed():
    return [
        # one decode step's token rows: a call whose latency counts
        _quant("int8_decode_tokens", 1, 64, 4096, "f16"),
        # fp32 rows of an odd count and length
        _quant("int8_ragged_rows", 3, 509, 2056, "f32"),
        # a checkpoint's expert matrices in bf16, converted once when a model is loaded
        _quant("int8_expert_weights", 8, 14336, 4096, "bf16"),
        # the framework's smallest layer: nine tokens, most of the time is launches
        _ffn("int8_tiny", 9, 4, 2, 256, 128),
        # serving, one step of 64 sequences: every expert's weights are read for a handful of rows
        _ffn("int8_decode", 64, 8, 2, 4096, 14336),
        # fine-grained experts under skewed routing
        _ffn("int8_fine", 8192, 64, 6, 2048, 1408, 1.1),
        # the largest layer: a long prompt batch over 128 skewed experts
        _ffn("int8_large", 16384, 128, 8, 7168, 2048, 1.2),
        # the training router of the smallest layer
        _router("router", "router_tiny", 9, 4, 2, 256),
        # and of the largest, its batch padded to a common length
        _router("router", "router_large", 16384, 128, 8, 7168, 0.125),
        # backward passes: of the smallest layer
        _router("backward", "router_backward_tiny", 9, 4, 2, 256),
        # of fine-grained experts, an odd number of tokens
        _router("backward", "router_backward_fine", 8191, 64, 6, 2048, 0.0),
        # of the largest layer, its padded batch, added to the token gradient that came through the experts
        _router("backward", "router_backward_large", 16384, 128, 8, 7168, 0.125, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "int8", "int8", "router", "backward", "backward"])
    if kind == "quantize":
        rows = _log(rng, 1, 100000)
        cols = 8 * _log(rng, 1, 2048)
        batch = rng.choice([1, 1, 3, 8])
        rows = max(1, min(rows, 400_000_000 // (cols * batch)))
        return {"kind": kind, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(["f16", "bf16", "f32"])}
    tokens = _log(rng, 1, 16384)
    if kind == "int8":
        experts = _log(rng, 1, 128)
        hidden, inter = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 112)
        # at most the largest listed case: weights and products
        while experts > 1 and experts * hidden * inter > 128 * 7168 * 2048:
            experts = (experts + 1) // 2
        top_k = rng.randint(1, min(8, experts))
        while tokens > 1 and tokens * top_k * hidden * inter > 16384 * 8 * 7168 * 2048:
            tokens = (tokens + 1) // 2
        return {"kind": kind, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "inter": inter,
                "zipf": rng.choice([0.0, 0.0, 1.1, 1.2])}
    experts = _log(rng, 1, 128)
    case = {"kind": kind, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(8, experts)),
            "hidden": 64 * _log(rng, 1, 112), "left_out": rng.choice([0.0, 0.0, 0.1, 0.5])}
    return dict(case, add=rng.choice([False, True])) if kind == "backward" else case


# ---------------------------------------------------------------------------------------------------------- the formats


def _plain_int8(x):
    """Codes (as fp32 integers) and scales [.., 1] of rows x [.., cols]; quotients in 64 bits: a code is decided by which
    side of a border between two integers its quotient lies on."""
    x = x.float()
    s = x.abs().amax(-1, keepdim=True) / 127
    q = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()).clamp_(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q)).float(), s


# -------------------------------------------------------------------------------------------------------------- inputs


def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + tag)
    return g


def _normal(shape, std, seed, tag, dtype=torch.float16):
    return (torch.randn(shape, generator=_gen(seed, tag), device="cuda") * std).to(dtype)


def _int8_weights(E, n, k, seed, tag):
    """Codes [E, n, k] and scales [E, n] of expert matrices of variance 1 / k, one expert at a time."""
    codes, scales = torch.empty((E, n, k), dtype=torch.int8, device="cuda"), torch.empty((E, n), device="cuda")
    g = _gen(seed, tag)
    for e in range(E):
        q, s = _plain_int8(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
        codes[e], scales[e] = q.to(torch.int8), s[:, 0]
    return codes, scales


def _tables(ids, E):
    """The contract's tables of expert ids [T, k] (-1: no expert)."""
    ids = ids.reshape(-1)
    live = np.flatnonzero(ids >= 0)
    n = np.bincount(ids[live], minlength=E)
    go = np.concatenate(([0], np.cumsum(n)))
    gpo = np.concatenate(([0], np.cumsum((n // 128 + 1) * 128)))
    M = -(-ids.size // 128) + E
    gidx = np.searchsorted(gpo[:-1], np.arange(M) * 128, side="right") - 1
    order = live[np.argsort(ids[live], kind="stable")]
    cpos = np.full(ids.size, -1)
    cpos[order] = np.arange(order.size)
    prow = np.where(ids >= 0, gpo[ids] + cpos - go[ids], -1)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return {"sizes": n.tolist(), "starts": gpo.tolist(), "offsets": go.tolist(), "padded": M * 128, "pairs": ids.size,
            "order": order, "gs": i32(n), "go": i32(go), "gpo": i32(gpo), "gidx": i32(gidx), "prow": i32(prow),
            "cpos": i32(cpos)}


def _routing(case, seed):
    """A routing of distinct experts per token, its routed weights [T, k] and the contract's tables."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    rng = np.random.default_rng([seed, T, E, k])
    logp = -case["zipf"] * np.log(np.arange(E) + 1.0)
    ids = np.argsort(-(logp[None] + rng.gumbel(size=(T, E))), axis=1, kind="stable")[:, :k]
    w = np.exp(rng.standard_normal((T, k)))
    w = (w / w.sum(1, keepdims=True)).astype(np.float32).reshape(-1)
    r = _tables(ids, E)
    return dict(r, topk_w=torch.from_numpy(w).cuda(), rw=torch.from_numpy(w[r["order"]]).cuda())


def prepare(case, seed):
    kind = case["kind"]
    if kind == "quantize":
        # rows whose magnitudes differ from channel to channel, as activations' and weights' do
        shape = (case["batch"], case["rows"], case["cols"])
        x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
        for b in range(case["batch"]):
            spread = torch.exp(torch.randn(case["cols"], generator=_gen(seed, 100 + b), device="cuda"))
            x[b] = torch.randn(shape[1:], generator=_gen(seed, 200 + b), device="cuda") * spread
        return {"case": case, "x": x}
    T, E, k, H = (case[n] for n in ("tokens", "experts", "top_k", "hidden"))
    zeros = lambda *shape, dtype=torch.float16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": case}
    if kind == "int8":
        I, r = case["inter"], _routing(case, seed)
        Tp = r["padded"]
        s["r"], s["x"] = r, _normal((T, H), 1.0, seed, 1)
        s["wg"], s["wu"] = _int8_weights(E, I, H, seed, 2), _int8_weights(E, I, H, seed, 3)
        s["wd"] = _int8_weights(E, H, I, seed, 4)
        # the program's buffers: packed token rows and their scales, routed weights, the hidden rows' workspace (their
        # codes, scales, and the rows in 32 bits), the output
        s["codes"], s["scales"] = zeros(Tp, H, dtype=torch.int8), zeros(Tp, dtype=torch.float32)
        s["w"], s["workspace"] = zeros(r["pairs"], dtype=torch.float32), zeros(Tp * (5 * I + 4), dtype=torch.uint8)
        s["out"] = zeros(Tp, H)
        return s
    # values on a grid (of 8-bit activations, of weights in steps of 2^-10) that leaves every sum of a logit exact in 32 bits
    # in any order: which experts are the largest, and which are equal, is then the same however the sums are taken
    s["x"] = (_normal((T, H), 32.0, seed, 1, torch.float32).round().clamp_(-127, 127) / 32).half()
    s["w"] = (_normal((E, H), 1024 / math.sqrt(H), seed, 2, torch.float32).round().clamp_(-1023, 1023) / 1024).half()
    mask = torch.rand(T, generator=_gen(seed, 3), device="cuda") >= case["left_out"]
    s["mask"] = mask.to(torch.uint8) if case["left_out"] else None
    # rows that are left out hold what was there before
    s["x"][~mask] = torch.where(torch.rand(H, generator=_gen(seed, 4), device="cuda") < 0.5, 65504.0, float("nan")).half()
    if kind == "router":
        return s
    # what the forward pass kept, and the gradients that reach the router
    s["ids"], _, s["probs"], s["lse"], s["counts"], _ = _plain_router(s["x"], s["w"], k, s["mask"])
    s["cpos"] = _tables(s["ids"].cpu().numpy(), E)["cpos"]
    s["drw"] = _normal((T * k,), 1.0, seed, 5, torch.float32)
    s["dlosses"] = torch.tensor([1e-2 * T, 1e-3 * T], device="cuda")  # of a loss summed over the tokens
    s["add"] = _normal((T, H), 2e-3, seed, 6) if case["add"] else None
    # the program's buffers: gradients, and scratch, made once
    s["dx"], s["dw"], s["scratch"] = zeros(T, H), zeros(E, H, dtype=torch.float32), {}
    return s


# ----------------------------------------------------------------------------------------------------------- one pass


def run(state):
    return {"quantize": _run_quantize, "int8": _run_int8, "router": _run_router, "backward": _run_backward}[state["case"]["kind"]](state)


def _run_quantize(s):
    """Quantises the rows; the codes are handed back as the values they stand for."""
    x = s["x"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        codes, scales = R.quantize_int8(x)
        return R.dequantize_int8(codes, scales, dtype=x.dtype), scales
    q, sc = _plain_int8(x)
    return (q * sc).to(x.dtype), sc.squeeze(-1)


def _groups(r):
    """(expert, first padded row, rows, first compact position) of the experts that hold rows."""
    return [(e, r["starts"][e], n, r["offsets"][e]) for e, n in enumerate(r["sizes"]) if n]


def _run_int8(s):
    """Quantises and packs the tokens, then the expert FFN on 8-bit weights: hidden rows are quantised between the two
    products, the output is scaled by the routed weights."""
    c, r = s["case"], s["r"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        R.pack_int8(s["x"], r["topk_w"], r["prow"], r["cpos"], s["codes"], s["scales"], s["w"])
        R.forward_int8(s["codes"], s["scales"], *s["wg"], *s["wu"], *s["wd"], s["w"], r["gs"], r["go"], r["gpo"], r["gidx"],
                       s["workspace"], s["out"])
        return s["out"]
    q, sc = _plain_int8(s["x"])
    at = torch.from_numpy(r["order"]).cuda() // c["top_k"]  # token of each pair in compact order
    out = torch.zeros((r["padded"], c["hidden"]), dtype=torch.float16, device="cuda")
    # one product per expert: a batched product would pad every expert to the largest group
    for e, p, n, o in _groups(r):
        x, xs = q[at[o:o + n]], sc[at[o:o + n]]
        g = (x @ s["wg"][0][e].float().T) * xs * s["wg"][1][e]
        u = (x @ s["wu"][0][e].float().T) * xs * s["wu"][1][e]
        h, hs = _plain_int8(g / (1 + torch.exp(-g)) * u)
        y = (h @ s["wd"][0][e].float().T) * hs * s["wd"][1][e]
        out[p:p + n] = (y * r["rw"][o:o + n, None]).half()
    return out


def _plain_router(x, w, k, mask):
    """Ids [T, k], their probabilities, all probabilities [T, E], logsumexp [T], counts [E + 1] (the last: tokens that
    count), losses [2]."""
    T, E = x.shape[0], w.shape[0]
    on = torch.ones(T, dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    logits = torch.where(on[:, None], x.float(), 0) @ w.float().T
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    p = torch.where(on[:, None], ex / total, 0)
    lse = torch.where(on, (top + torch.log(total))[:, 0], 0)
    vals, ids = torch.sort(p, dim=1, descending=True, stable=True)
    ids = torch.where(on[:, None], ids[:, :k], -1).int()
    counts = torch.cat(((ids[..., None] == torch.arange(E, device=x.device)).sum((0, 1)), on.sum()[None])).int()
    n = counts[E].double().clamp(min=1)  # long sums, over the tokens, in 64 bits
    balance = E / (k * n) * (counts[:E] * (p.double().sum(0) / n)).sum()
    return ids, vals[:, :k].contiguous(), p, lse, counts, torch.stack((balance, (lse.double() ** 2).sum() / n)).float()


def _run_router(s):
    """Routing of a training batch: what the experts need, what the backward pass needs, the losses."""
    k = s["case"]["top_k"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        s["out"] = R.router_train(s["x"], s["w"], k, token_mask=s["mask"], out=s.get("out"))
        return tuple(s["out"][n] for n in ("topk_ids", "topk_weights", "probs", "lse", "counts", "losses"))
    return _plain_router(s["x"], s["w"], k, s["mask"])


def _run_backward(s):
    """Gradients of the token rows and of the gate matrix."""
    E, k = s["case"]["experts"], s["case"]["top_k"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        if "bytes" not in s["scratch"]:
            n = R.router_backward_scratch_bytes(s["case"]["tokens"], s["case"]["hidden"], E)
            s["scratch"]["bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        R.router_backward(s["x"], s["w"], s["ids"], s["probs"], s["lse"], s["counts"], s["drw"], s["dlosses"], s["dx"], s["dw"],
                          s["scratch"]["bytes"], compact_pos_of_pair=s["cpos"], token_mask=s["mask"], dx_add=s["add"])
        return s["dx"], s["dw"]
    p, n = s["probs"], s["counts"][E].float().clamp(min=1)
    on = torch.ones_like(s["lse"], dtype=torch.bool) if s["mask"] is None else s["mask"].bool()
    pairs = torch.where(s["cpos"] >= 0, s["drw"][s["cpos"].clamp(min=0).long()], 0).view(-1, k)
    dp = (s["dlosses"][0] * E / (k * n * n) * s["counts"][:E]).expand_as(p).clone()
    dp.scatter_add_(1, s["ids"].clamp(min=0).long(), torch.where(s["ids"] >= 0, pairs, 0))
    dl = p * (dp - (p * dp).sum(1, keepdim=True)) + s["dlosses"][1] * 2 / n * s["lse"][:, None] * p
    dl = torch.where(on[:, None], dl, 0)
    dx = dl @ s["w"].float()
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return dx.half(), dl.T @ torch.where(on[:, None], s["x"].float(), 0)


# ------------------------------------------------------------------------------------------------- definition, 64 bits


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        if s["x"].numel() >= 1 << 29:
            return None
        got = [_exact_int8(x.double()) for x in s["x"]]
        return torch.stack([q * sc for q, sc in got]), torch.stack([sc[:, 0] for _, sc in got])
    E, k = case["experts"], case["top_k"]
    if kind == "int8":
        r, out = s["r"], torch.zeros((s["r"]["padded"], case["hidden"]), dtype=torch.float64, device="cuda")
        q, sc = _exact_int8(s["x"].double())
        token = torch.empty(r["pairs"], dtype=torch.long, device="cuda")
        token[r["cpos"].long()] = torch.arange(r["pairs"], device="cuda") // k
        value = lambda w, e: w[0][e].double() * w[1][e].double()[:, None]  # noqa: E731
        for e in range(E):
            if not r["sizes"][e]:
                continue
            at = slice(r["offsets"][e], r["offsets"][e] + r["sizes"][e])
            x = q[token[at]] * sc[token[at]]
            g = x @ value(s["wg"], e).T
            hq, hs = _exact_int8(g * torch.sigmoid(g) * (x @ value(s["wu"], e).T))
            y = (hq * hs) @ value(s["wd"], e).T
            out[r["starts"][e]:r["starts"][e] + r["sizes"][e]] = r["rw"][at].double()[:, None] * y
        return out
    on = torch.ones(case["tokens"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] > 0
    live = on.nonzero()[:, 0]
    x, w, n = s["x"][live].double(), s["w"].double(), live.numel()
    whole = lambda t, fill=0: torch.full((case["tokens"], *t.shape[1:]), fill, dtype=t.dtype, device="cuda").index_copy_(0, live, t)  # noqa: E731
    if kind == "router":
        logits = x @ w.T
        lse = torch.logsumexp(logits, 1)
        p = torch.exp(logits - lse[:, None])
        # logits are whole multiples of 2^-15: with the expert's index below them the order is one of whole numbers
        key = (logits * 2**15).round().long() * 256 + (255 - torch.arange(E, device="cuda"))
        ids = key.argsort(1, descending=True)[:, :k]
        counts = torch.zeros_like(p).scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.float64)).sum(0)
        losses = torch.stack((E / k * (counts / max(n, 1) * (p.sum(0) / max(n, 1))).sum(), (lse * lse).sum() / max(n, 1)))
        every = torch.cat((counts, torch.tensor([float(n)], device="cuda", dtype=torch.float64))).int()
        return whole(ids.int(), -1), whole(p.gather(1, ids)), whole(p), whole(lse), every, losses
    d, p, lse = s["dlosses"].double(), s["probs"][live].double(), s["lse"][live].double()
    drw = s["drw"].double()[s["cpos"].long().view(-1, k)[live]]
    dp = torch.zeros_like(p).scatter_add_(1, s["ids"][live].long(), drw)
    dp += d[0] * E / (k * max(n, 1)) * s["counts"][:E] / max(n, 1)
    dl = p * dp - p * (p * dp).sum(1, keepdim=True) + d[1] / max(n, 1) * 2 * lse[:, None] * p
    dx = whole(dl @ w)
    return (dx if s["add"] is None else dx + s["add"].double()), dl.T @ x


def _exact_int8(x):
    """Codes and scales of rows x [rows, cols] (64 bits): the scale is held in 32 bits, a code is the integer whose distance
    from the quotient is least, the even one of two."""
    s = (x.abs().amax(1, keepdim=True) / 127).float().double()
    r = torch.where(s > 0, x / s, torch.zeros_like(x))
    low = torch.floor(r)
    up = (r - low > 0.5) | ((r - low == 0.5) & (low % 2 != 0))
    return (low + up).clamp(-127, 127), s


# --------------------------------------------------------------------------------------------------------------- work


def work(case):
    """Each input read once and each output written once; products count two operations per multiply-add."""
    kind = case["kind"]
    if kind == "quantize":
        rows, size = case["batch"] * case["rows"], DTYPES[case["dtype"]].itemsize
        n = rows * case["cols"]
        # the rows in, codes and scales out; then codes and scales in, values out
        return {"bytes": 2 * n * (size + 1) + 8 * rows, "flops": 4 * n}
    T, E, k, H = (case[n] for n in ("tokens", "experts", "top_k", "hidden"))
    if kind == "int8":
        I, pairs = case["inter"], T * k
        used = min(E, pairs)  # experts that hold rows, at most
        weights = used * (3 * H * I + 4 * (2 * I + H))
        return {"bytes": weights + T * H * 2 + pairs * H * 2 + pairs * 8, "flops": 6 * pairs * H * I}
    kept = 4 * T * (E + 1)  # probabilities and logsumexps
    if kind == "router":
        return {"bytes": 2 * (T + E) * H + kept + 8 * T * k, "flops": 2 * T * E * H}
    rows = T * H * 2 * (3 if case["add"] else 2)
    return {"bytes": rows + 6 * E * H + kept + 12 * T * k, "flops": 4 * T * E * H}

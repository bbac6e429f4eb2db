"""Cases of the operators around the routed expert FFN: microscaled 4-bit (MXFP4) quantisation, the routed FFN on MXFP4
weights, the training forward of the gated gate/up stage, and the backward pass of the routed FFN.

``run`` computes an operator either from elementary torch operations in 32 bits (``own`` false) or through the library
(``own`` true); ``exact`` computes the definition in 64 bits.  Formats shared by both sides:

  * MXFP4: blocks of 32 consecutive elements of a row share one power-of-two scale 2^(floor(log2(amax)) - 2) held as an
    exponent byte (bias 127); elements are E2M1 codes (sign, 0 .5 1 1.5 2 3 4 6), low nibble first, rounded to nearest
    even and clamped at 6.  A row's codes are padded to whole chunks of 256 elements (128 bytes); scale bytes are stored
    chunk by chunk: [chunks, rows, 8], the 8 bytes ordered blocks 0 2 4 6 1 3 5 7 of the chunk.
  * The dispatch contract: pairs sorted by expert (stably), every expert's rows padded to (n // 128 + 1) * 128 rows, one
    expert id per 128-row block, routed weights in compact (unpadded) order.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCKS = (0, 2, 4, 6, 1, 3, 5, 7)  # order of a chunk's scale bytes

# ---------------------------------------------------------------------------------------------------------------- cases


def _ffn(kind, name, tokens, experts, top_k, hidden, inter, zipf=0.0):
    return {"name": name, "kind": kind, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "inter": inter, "zipf": zipf}


def _quant(name, batch, rows, cols, dtype):
    return {"name": name, "kind": "quantize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # one decode step's token rows, quantised before the expert products: a call whose latency counts
        _quant("quantize_decode_tokens", 1, 64, 4096, "f16"),
        # fp32 rows of an odd count whose last block is cut short
        _quant("quantize_ragged_rows", 1, 1021, 1416, "f32"),
        # a checkpoint's expert matrices in bf16, converted once when a model is loaded
        _quant("quantize_expert_weights", 8, 14336, 4096, "bf16"),
        # the framework's smallest layer: nine tokens, most of the time is launches
        _ffn("mx", "mx_tiny", 9, 4, 2, 256, 128),
        # serving, one step of 64 sequences: every expert's weights are read for a handful of rows
        _ffn("mx", "mx_decode", 64, 8, 2, 4096, 14336),
        # fine-grained experts under skewed routing, an intermediate size that is no multiple of a 256-element chunk
        _ffn("mx", "mx_fine", 8192, 64, 6, 2048, 1408, 1.1),
        # the largest layer: a long prompt batch over 128 skewed experts
        _ffn("mx", "mx_large", 16384, 128, 8, 7168, 2048, 1.2),
        # training forward of the gated stage: skewed fine-grained experts
        _ffn("train", "train_fine", 8192, 64, 6, 2048, 1408, 1.1),
        # and few large experts
        _ffn("train", "train_prefill", 4096, 8, 2, 4096, 14336),
        # the backward pass of nine tokens over four experts
        _ffn("backward", "backward_tiny", 9, 4, 2, 256, 128),
        # of skewed fine-grained experts, some of them with few rows
        _ffn("backward", "backward_fine", 8192, 64, 6, 2048, 1408, 1.1),
        # and of few large experts
        _ffn("backward", "backward_prefill", 4096, 8, 2, 4096, 14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "mx", "mx", "train", "backward", "backward"])
    if kind == "quantize":
        rows = _log(rng, 1, 100000)
        cols = 8 * _log(rng, 1, 2048)
        batch = rng.choice([1, 1, 3, 8])
        rows = max(1, min(rows, 400_000_000 // (cols * batch)))
        return {"kind": kind, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(["f16", "bf16", "f32"])}
    top = {"mx": 16384, "train": 8192, "backward": 8192}[kind]
    tokens = _log(rng, 1, top)
    experts = _log(rng, 1, 128)
    top_k = rng.randint(1, min(8, experts))
    hidden, inter = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 112)
    # at most the largest listed case of the kind: weights and products
    most = {"mx": (128 * 7168 * 2048, 16384 * 8 * 7168 * 2048)}.get(kind, (8 * 4096 * 14336, 8192 * 4096 * 14336))
    while experts > 1 and experts * hidden * inter > most[0]:
        experts = (experts + 1) // 2
    top_k = min(top_k, experts)
    while tokens > 1 and tokens * top_k * hidden * inter > most[1]:
        tokens = (tokens + 1) // 2
    return {"kind": kind, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "inter": inter,
            "zipf": rng.choice([0.0, 0.0, 1.1, 1.2])}


# ---------------------------------------------------------------------------------------------------------- the formats


def _chunks(cols):
    return -(-cols // 256)


def _plain_quantize(x):
    """(codes' values in E2M1 units, scales) of x [.., cols], block by block, in 32 bits: values [.., blocks, 32],
    scales [.., blocks, 1], with x rounded to values * scales."""
    cols = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, _chunks(cols) * 256 - cols))
    v = v.view(*v.shape[:-1], -1, 32)
    amax = v.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1): floor(log2(amax)) = e - 1
    e = torch.where(amax > 0, e - 3, torch.full_like(e, -127)).clamp_(min=-127)
    half = e // 2  # 2^e in two factors, each a normal number
    y = torch.ldexp(torch.ldexp(v, -half), half - e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp_(max=6.0), y)
    return q, e


def _values(q, e, cols):
    """What codes and scale exponents stand for, in 32 bits."""
    half = e // 2
    return torch.ldexp(torch.ldexp(q, half), e - half).flatten(-2)[..., :cols]


def _encode(q, e):
    """Code bytes [.., rows, bytes] and scale bytes [.., chunks, rows, 8] in the stored layout."""
    a = q.abs()
    idx = (2 * a).clamp(max=4) + (a > 2) * (a - 2).clamp(max=2) + (a > 4)  # 0 .5 1 1.5 2 | 3 4 | 6
    idx = (idx.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    codes = idx[..., 0::2] | (idx[..., 1::2] << 4)
    s = (e.squeeze(-1) + 127).to(torch.uint8)
    s = s.view(*s.shape[:-1], -1, 8)[..., list(BLOCKS)]  # [.., rows, chunks, 8]
    return codes.contiguous(), s.transpose(-3, -2).contiguous()


def _decode(codes, scales, cols, dtype):
    """Values [rows, cols] of stored codes [rows, bytes] and scales [chunks, rows, 8]."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=dtype, device=codes.device)
    idx = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    back = [BLOCKS.index(b) for b in range(8)]
    s = scales.transpose(0, 1)[..., back].flatten(1).to(dtype) - 127  # [rows, blocks]
    v = table[idx].view(codes.shape[0], -1, 32) * torch.exp2(s).unsqueeze(-1)
    return v.flatten(1)[:, :cols]


# -------------------------------------------------------------------------------------------------------------- inputs


def _gen(seed, tag):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + tag)
    return g


def _normal(shape, std, seed, tag, dtype=torch.float16):
    return (torch.randn(shape, generator=_gen(seed, tag), device="cuda") * std).to(dtype)


def _weights(E, n, k, seed, tag):
    """fp16 expert matrices [E, n, k] of variance 1 / k, one expert at a time."""
    w, g = torch.empty((E, n, k), dtype=torch.float16, device="cuda"), _gen(seed, tag)
    for e in range(E):
        w[e] = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
    return w


def _mx_weights(E, n, k, seed, tag):
    """The same as MXFP4 codes and scales."""
    ch, g = _chunks(k), _gen(seed, tag)
    codes = torch.empty((E, n, 128 * ch), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, ch, n, 8), dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _encode(*_plain_quantize(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)))
    return codes, scales


def _routing(case, seed):
    """Expert ids [T, k] (distinct per token), routed weights [T, k] and the contract's tables."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    rng = np.random.default_rng([seed, T, E, k])
    logp = -case["zipf"] * np.log(np.arange(E) + 1.0)
    ids = np.argsort(-(logp[None] + rng.gumbel(size=(T, E))), axis=1, kind="stable")[:, :k].reshape(-1)
    w = np.exp(rng.standard_normal((T, k)))
    w = (w / w.sum(1, keepdims=True)).astype(np.float32).reshape(-1)
    n = np.bincount(ids, minlength=E)
    go = np.concatenate(([0], np.cumsum(n)))
    gpo = np.concatenate(([0], np.cumsum((n // 128 + 1) * 128)))
    M = -(-ids.size // 128) + E
    gidx = np.searchsorted(gpo[:-1], np.arange(M) * 128, side="right") - 1
    order = np.argsort(ids, kind="stable")
    cpos = np.empty_like(order)
    cpos[order] = np.arange(ids.size)
    prow = gpo[ids] + cpos - go[ids]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return {"sizes": n.tolist(), "starts": gpo.tolist(), "offsets": go.tolist(), "padded": M * 128, "pairs": ids.size,
            "topk_w": torch.from_numpy(w).cuda(), "rw": torch.from_numpy(w[order]).cuda(), "gs": i32(n), "go": i32(go),
            "gpo": i32(gpo), "gidx": i32(gidx), "prow": i32(prow), "cpos": i32(cpos)}


def _rows(r, cols, seed, tag, std=1.0):
    """Rows of the padded layout, fp16; padding rows are zero."""
    x = torch.zeros((r["padded"], cols), dtype=torch.float16, device="cuda")
    x[r["prow"].long()] = _normal((r["pairs"], cols), std, seed, tag)
    return x


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
    E, H, I = case["experts"], case["hidden"], case["inter"]
    r = _routing(case, seed)
    Tp = r["padded"]
    s = {"case": case, "r": r}
    zeros = lambda *shape, dtype=torch.float16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    if kind == "mx":
        s["x"] = _normal((case["tokens"], H), 1.0, seed, 1)
        s["wg"], s["wu"] = _mx_weights(E, I, H, seed, 2), _mx_weights(E, I, H, seed, 3)
        s["wd"] = _mx_weights(E, H, I, seed, 4)
        # the program's buffers: packed token rows, routed weights, the hidden rows' workspace, the output
        s["codes"], s["scales"] = zeros(Tp, 128 * _chunks(H), dtype=torch.uint8), zeros(_chunks(H), Tp, 8, dtype=torch.uint8)
        s["w"] = zeros(r["pairs"], dtype=torch.float32)
        s["workspace"] = zeros(Tp * 136 * _chunks(I), dtype=torch.uint8)
        s["out"] = zeros(Tp, H)
        return s
    s["x"] = _rows(r, H, seed, 1)
    s["wg"], s["wu"] = _weights(E, I, H, seed, 2), _weights(E, I, H, seed, 3)
    if kind == "train":
        s["gate"], s["up"], s["hidden"] = zeros(Tp, I), zeros(Tp, I), zeros(Tp, I)
        return s
    s["wd"] = _weights(E, H, I, seed, 4)
    # what the forward pass kept, and the gradient of its output
    s["gate"], s["up"], s["dout"] = _rows(r, I, seed, 5), _rows(r, I, seed, 6), _rows(r, H, seed, 7)
    # the program's buffers: gradients of the pre-activations, the weighted hidden rows, scratch, the results
    s["dgate"], s["dup"], s["hidden"] = zeros(Tp, I), zeros(Tp, I), zeros(Tp, I)
    s["scratch"] = zeros(r["pairs"] * -(-I // 128), dtype=torch.float32)
    s["dx"], s["drw"] = zeros(Tp, H), zeros(r["pairs"], dtype=torch.float32)
    s["dwg"], s["dwu"], s["dwd"] = zeros(E, I, H), zeros(E, I, H), zeros(E, H, I)
    return s


# ----------------------------------------------------------------------------------------------------------- one pass


def run(state):
    kind = state["case"]["kind"]
    if kind == "quantize":
        return _run_quantize(state)
    return {"mx": _run_mx, "train": _run_train, "backward": _run_backward}[kind](state)


def _run_quantize(s):
    """Quantises the rows; the codes are handed back as the values they stand for."""
    x = s["x"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        codes, scales = R.quantize_mxfp4(x)
        return R.dequantize_mxfp4(codes, scales, x.shape[-1], dtype=x.dtype)
    q, e = _plain_quantize(x)
    return _values(q, e, x.shape[-1]).to(x.dtype)


def _groups(r):
    """(expert, first padded row, rows, first compact position) of the experts that hold rows."""
    return [(e, r["starts"][e], n, r["offsets"][e]) for e, n in enumerate(r["sizes"]) if n]


def _run_mx(s):
    """Quantises and packs the tokens, then the expert FFN on MXFP4 weights: hidden rows are quantised between the two
    products, the output is scaled by the routed weights."""
    c, r = s["case"], s["r"]
    H, I = c["hidden"], c["inter"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        R.pack_mxfp4(s["x"], r["topk_w"], r["prow"], r["cpos"], s["codes"], s["scales"], s["w"])
        R.forward_mxfp4(s["codes"], s["scales"], *s["wg"], *s["wu"], *s["wd"], s["w"], r["gs"], r["go"], r["gpo"], r["gidx"],
                        s["workspace"], s["out"])
        return s["out"]
    x = _values(*_plain_quantize(s["x"]), H)
    stacked = torch.zeros((r["padded"], H), device="cuda")
    stacked[r["prow"].long()] = x.repeat_interleave(c["top_k"], 0)
    out = torch.zeros((r["padded"], H), dtype=torch.float16, device="cuda")
    # one product per expert: a batched product would pad every expert to the largest group
    for e, p, n, q in _groups(r):
        rows = stacked[p:p + n]
        g = rows @ _decode(s["wg"][0][e], s["wg"][1][e], H, torch.float32).T
        u = rows @ _decode(s["wu"][0][e], s["wu"][1][e], H, torch.float32).T
        h = _values(*_plain_quantize(g / (1 + torch.exp(-g)) * u), I)
        y = h @ _decode(s["wd"][0][e], s["wd"][1][e], I, torch.float32).T
        out[p:p + n] = (y * r["rw"][q:q + n, None]).half()
    return out


def _run_train(s):
    """The gated stage of the training forward: gate and up projections, kept for the backward pass, and hidden rows."""
    r = s["r"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        R.gate_up_train(s["x"], s["wg"], s["wu"], r["gs"], r["gpo"], r["gidx"], s["gate"], s["up"], s["hidden"])
        return s["gate"], s["up"], s["hidden"]
    gate, up, hidden = (torch.zeros_like(s[n]) for n in ("gate", "up", "hidden"))
    for e, p, n, _ in _groups(r):
        x = s["x"][p:p + n].float()
        g, u = x @ s["wg"][e].float().T, x @ s["wu"][e].float().T
        gate[p:p + n], up[p:p + n] = g.half(), u.half()
        hidden[p:p + n] = (g / (1 + torch.exp(-g)) * u).half()
    return gate, up, hidden


def _run_backward(s):
    """Gradients of the routed FFN: of the token rows, the three expert matrices and the routed weights."""
    r = s["r"]
    if own:
        import mixture_experts_routed_grouped_amd as R
        R.backward(s["x"], s["dout"], s["wg"], s["wu"], s["wd"], r["rw"], s["gate"], s["up"], r["gs"], r["go"], r["gpo"],
                   r["gidx"], s["dgate"], s["dup"], s["hidden"], s["scratch"], s["dx"], s["dwg"], s["dwu"], s["dwd"], s["drw"])
        return s["dx"], s["dwg"], s["dwu"], s["dwd"], s["drw"]
    dx, dwg, dwu, dwd, drw = (torch.zeros_like(s[n]) for n in ("dx", "dwg", "dwu", "dwd", "drw"))
    for e, p, n, q in _groups(r):
        got = _gradients(*(s[m][p:p + n].float() for m in ("x", "dout", "gate", "up")),
                         *(s[m][e].float() for m in ("wg", "wu", "wd")), r["rw"][q:q + n])
        dx[p:p + n], dwg[e], dwu[e], dwd[e], drw[q:q + n] = got
    return dx, dwg, dwu, dwd, drw


def _gradients(x, dout, g, u, wg, wu, wd, w):
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    h = silu * u
    back = dout @ wd  # the gradient of the hidden row before the routed weight
    dh = back * w[:, None]
    dg = dh * u * (sig + silu * (1 - sig))
    du = dh * silu
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, (dout * w[:, None]).T @ h, (back * h).sum(1)


# ------------------------------------------------------------------------------------------------- definition, 64 bits


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        return torch.stack([_exact_mx(x.double()) for x in s["x"]]) if s["x"].numel() < 1 << 29 else None
    r = s["r"]
    E, H, I = case["experts"], case["hidden"], case["inter"]
    f64 = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    sizes, starts, offsets = r["sizes"], r["starts"], r["offsets"]
    live = [e for e in range(E) if sizes[e]]
    rows = lambda t, e: t[starts[e]:starts[e] + sizes[e]].double()  # noqa: E731
    if kind == "mx":
        out = f64(r["padded"], H)
        x = _exact_mx(s["x"].double())
        token = torch.empty(r["pairs"], dtype=torch.long, device="cuda")
        token[r["cpos"].long()] = torch.arange(r["pairs"], device="cuda") // case["top_k"]
        for e in live:
            at = slice(offsets[e], offsets[e] + sizes[e])
            xe = x[token[at]]
            wg, wu, wd = (_decode(w[0][e], w[1][e], k, torch.float64) for w, k in ((s["wg"], H), (s["wu"], H), (s["wd"], I)))
            g = xe @ wg.T
            h = _exact_mx(g * torch.sigmoid(g) * (xe @ wu.T))
            out[starts[e]:starts[e] + sizes[e]] = r["rw"][at].double()[:, None] * (h @ wd.T)
        return out
    if kind == "train":
        gate, up, hidden = (f64(r["padded"], I) for _ in range(3))
        for e in live:
            to = slice(starts[e], starts[e] + sizes[e])
            xe = rows(s["x"], e)
            gate[to], up[to] = xe @ s["wg"][e].double().T, xe @ s["wu"][e].double().T
            hidden[to] = gate[to] * torch.sigmoid(gate[to]) * up[to]
        return gate, up, hidden
    dx, drw = f64(r["padded"], H), f64(r["pairs"])
    dwg, dwu, dwd = f64(E, I, H), f64(E, I, H), f64(E, H, I)
    for e in live:
        at = slice(offsets[e], offsets[e] + sizes[e])
        x, dy, g, u = (rows(s[n], e) for n in ("x", "dout", "gate", "up"))
        w = r["rw"][at].double()[:, None]
        sig = torch.sigmoid(g)
        dh = dy @ s["wd"][e].double()
        drw[at] = (dh * g * sig * u).sum(1)
        dg, du = w * dh * u * sig * (1 + g * (1 - sig)), w * dh * g * sig
        dx[starts[e]:starts[e] + sizes[e]] = dg @ s["wg"][e].double() + du @ s["wu"][e].double()
        dwg[e], dwu[e], dwd[e] = dg.T @ x, du.T @ x, (w * dy).T @ (g * sig * u)
    return dx, dwg, dwu, dwd, drw


def _exact_mx(x):
    """The MXFP4 value of every element of x [rows, cols] (64 bits): the nearest of the block's 15 levels, ties to the
    level of even code."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))), torch.full_like(top, -125.0))
    # log2 may round across a power of two
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    unit = torch.exp2((e - 2).clamp(min=-127))
    a = v.abs() / unit
    out = torch.zeros_like(a)
    for i in range(1, 8):  # level i from the midpoint below it on; the midpoint itself belongs to the even code
        mid = (LEVELS[i - 1] + LEVELS[i]) / 2
        out = torch.where((a > mid) | ((a == mid) & (i % 2 == 0)), LEVELS[i], out)
    return torch.copysign(out * unit, v).flatten(1)[:, :cols]


# --------------------------------------------------------------------------------------------------------------- work


def work(case):
    """Each input read once and each output written once; products count two operations per multiply-add."""
    kind = case["kind"]
    if kind == "quantize":
        n, size = case["batch"] * case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize
        stored = case["batch"] * case["rows"] * 136 * _chunks(case["cols"])
        # the rows in, codes and scales out; then codes and scales in, values out
        return {"bytes": 2 * n * size + 2 * stored, "flops": 4 * n}
    T, E, k, H, I = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "inter"))
    pairs = T * k
    used = min(E, pairs)  # experts that hold rows, at most
    if kind == "mx":
        weights = used * (2 * I * 136 * _chunks(H) + H * 136 * _chunks(I))
        return {"bytes": weights + T * H * 2 + pairs * H * 2 + pairs * 8, "flops": 6 * pairs * H * I}
    if kind == "train":
        return {"bytes": 2 * (2 * used * I * H + pairs * H + 3 * pairs * I), "flops": 4 * pairs * H * I}
    weights = 2 * 3 * I * H * (used + E)  # the matrices in, their gradients out
    return {"bytes": weights + 2 * (3 * pairs * H + 2 * pairs * I) + 8 * pairs, "flops": 12 * pairs * H * I}

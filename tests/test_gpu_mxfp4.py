"""GPU tests of the MXFP4 entry points against the 64-bit oracle
(oracle/mxfp4.py): quantisation bit for bit, the products within bounds that
follow from fp32 accumulation and one final rounding.

Bounds.  A product of two MXFP4 values is exact in fp32, so a sum of K of
them carries at most K additions' rounding: |error| <= K 2^-23 sum|x w| (2^-23
per addition allows for a truncating adder).  silu's hardware exp2 and
reciprocal add a relative 2^-20.  An output rounded to fp16 adds half a step,
2^-11 of the value (2^-25 absolute below the normal numbers); a hidden value
must be the E2M1 number nearest to some value within the bound of the true
one, under a scale byte that such a block maximum gives."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import workloads
from oracle import mxfp4 as MX

pytestmark = pytest.mark.gpu
F16_HALF_STEP = 2.0 ** -11
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------ quantisation
def _patterns(dtype):
    """Rows of every 16-bit pattern of the type that is a finite number
    (fp32: the same patterns as high halves, with varied low bits, subnormals
    among them), in an order that mixes magnitudes, and rows of close ones."""
    bits = np.arange(65536, dtype=np.uint32)
    if dtype == "f16":
        v = bits.astype(np.uint16).view(np.float16)
        bits = bits[np.isfinite(v)]
    else:
        v = (bits << 16).view(np.float32)
        bits = bits[np.isfinite(v)]
    rng = np.random.default_rng(11)
    order = np.argsort(bits & 0x7FFF, kind="stable")
    both = np.concatenate([bits[order], rng.permutation(bits)])
    both = np.concatenate([both, np.zeros(-both.size % 512, np.uint32)])
    if dtype == "f32":
        full = ((both << 16) | rng.integers(0, 65536, both.size).astype(np.uint32)).view(np.float32)
        return torch.from_numpy(full.reshape(-1, 512).copy())
    t = torch.from_numpy(both.astype(np.uint16).view(np.int16).reshape(-1, 512).copy())
    return t.view(DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantize_all_patterns(dtype):
    x = _patterns(dtype)
    codes, scales = R.quantize_mxfp4(x.cuda())
    torch.cuda.synchronize()
    wc, ws = MX.stored(*MX.quantize(x.double().numpy()))
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy(), wc)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 8), (1, 1, 256), (1, 3, 24), (2, 5, 264), (3, 7, 1416),
                                             (1, 130, 4096), (2, 33, 512 + 32), (1, 1100, 8192)])
def test_quantize_shapes_and_way_back(dtype, batch, rows, cols):
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((batch, rows, cols)) * np.exp(rng.standard_normal(cols))
    x = torch.from_numpy(x).to(DTYPES[dtype])
    codes, scales = R.quantize_mxfp4(x.cuda())
    back = R.dequantize_mxfp4(codes, scales, cols, dtype=x.dtype)
    torch.cuda.synchronize()
    some = range(rows) if rows < 200 else [0, 1, 7, 8, 511, rows - 1]
    for b in range(batch):
        wc, ws = MX.stored(*MX.quantize(x[b].double().numpy()[list(some)]))
        assert np.array_equal(codes[b].cpu().numpy()[list(some)], wc)
        assert np.array_equal(scales[b].cpu().numpy()[:, list(some)], ws)
        assert np.array_equal(_np(back[b])[list(some)], MX.values(wc, ws, cols))
    two, s2 = R.quantize_mxfp4(x[0].cuda())          # a matrix by itself is the batch's first
    assert torch.equal(two, codes[0]) and torch.equal(s2, scales[0])


def test_quantize_nonfinite_blocks():
    x = torch.randn(4, 256)
    x[0, 3], x[1, 40], x[2, 255], x[3, 64] = float("nan"), float("inf"), -float("inf"), 65504.0
    for t in DTYPES.values():
        codes, scales = R.quantize_mxfp4(x.to(t).cuda())
        back = R.dequantize_mxfp4(codes, scales, 256, dtype=t).cpu()
        wc, ws = MX.stored(*MX.quantize(x.to(t).double().numpy()))
        assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(scales.cpu().numpy(), ws)
        assert torch.isnan(back[0, :32]).all() and not torch.isnan(back[0, 32:]).any()
        assert torch.isnan(back[1, 32:64]).all() and torch.isnan(back[2, 224:]).all()
        assert torch.isnan(back).sum() == 96


def test_dequantize_every_code_and_scale():
    """Every code under every scale byte, in each type: exact in fp32, one
    rounding in fp16 and bf16."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(32, 1)[:, :256].contiguous().view(64, 128)
    scales = torch.arange(256).to(torch.uint8).repeat(2).view(1, 64, 8).contiguous()
    want = MX.values(codes.numpy(), scales.numpy(), 256)
    for t in DTYPES.values():
        got = R.dequantize_mxfp4(codes.cuda(), scales.cuda(), 256, dtype=t).cpu()
        ref = torch.from_numpy(want).to(t)           # 64 bits to the type: one rounding
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        ok = ~torch.isnan(ref)
        assert torch.equal(got[ok], ref[ok])


def test_quantize_past_32_bit_offsets():
    """More than 2^32 elements: rows on both sides of the border."""
    rows, cols = (1 << 21) + 5, 2048
    x = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    some = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 21) - 1, 1 << 21, rows - 1]
    g = torch.Generator().manual_seed(3)
    v = torch.randn((len(some), cols), generator=g).half()
    x[some] = v.cuda()
    codes, scales = R.quantize_mxfp4(x)
    back = R.dequantize_mxfp4(codes, scales, cols)
    torch.cuda.synchronize()
    want = MX.quantized_values(v.double().numpy())
    assert np.array_equal(_np(back[some]), want)
    assert int(torch.count_nonzero(codes.view(torch.int32).any(1))) == len(some)
    assert torch.count_nonzero(back.view(torch.int32).any(1)) == len(some)


def test_quantize_many_short_rows():
    """More rows than one pass of the largest grid takes (2^20 workgroups of
    32 rows), 8 elements each: rows before, at and behind the border."""
    rows = (1 << 25) + 70
    x = torch.zeros((rows, 8), dtype=torch.float16, device="cuda")
    some = [0, 31, 32, (1 << 23) - 1, 1 << 23, (1 << 25) - 1, 1 << 25, rows - 1]
    v = torch.randn((len(some), 8), generator=torch.Generator().manual_seed(4)).half()
    x[some] = v.cuda()
    codes, scales = R.quantize_mxfp4(x)
    back = R.dequantize_mxfp4(codes, scales, 8)
    torch.cuda.synchronize()
    assert np.array_equal(_np(back[some]), MX.quantized_values(v.double().numpy()))
    assert int((back != 0).any(1).sum()) == len(some)


# -------------------------------------------------------------------- pack
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (5, 3, 264), (130, 2, 512), (700, 8, 1408)])
def test_pack(T, k, H):
    rng = np.random.default_rng(T)
    E = 16
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    c = R.build_contract(ids, E)
    prow, cpos = c["padded_row_of_pair"].copy(), c["compact_pos_of_pair"].copy()
    if T > 4:                                         # pairs that the device contract left out
        prow[3], cpos[3] = -1, -1
        prow[4] = c["total_padded_tokens"]
    x = torch.from_numpy(rng.standard_normal((T, H))).half().cuda()
    w = torch.rand(T * k, device="cuda")
    Tp = c["total_padded_tokens"]
    cs, ss = R.mxfp4_shapes((Tp, H))
    codes = torch.full(cs, 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full(ss, 0xFF, dtype=torch.uint8, device="cuda")
    wc = torch.full((T * k,), -7.0, device="cuda")
    i32 = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    R.pack_mxfp4(x, w, i32(prow), i32(cpos), codes, scales, wc)
    qc, qs = R.quantize_mxfp4(x)
    torch.cuda.synchronize()
    moved = np.zeros(Tp, bool)
    for p in range(T * k):
        r = prow[p]
        if 0 <= r < Tp:
            moved[r] = True
            assert torch.equal(codes[r], qc[p // k]) and torch.equal(scales[:, r], qs[:, p // k])
        if cpos[p] >= 0:
            assert wc[cpos[p]] == w[p]
    rest = torch.from_numpy(~moved).cuda()
    assert (codes[rest] == 0x5A).all() and (scales[:, rest] == 0xFF).all()


# ---------------------------------------------------------------- products
def _case(counts, H, I, seed=0):
    """Tables for exact group sizes and random operands; token rows outside
    the groups hold NaN scales, outputs and workspaces a sentinel."""
    E = len(counts)
    ids = workloads.routing_from_counts(counts, seed=seed)
    c = R.build_contract(ids, E)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    Tp, pairs = c["total_padded_tokens"], c["pairs"]
    d = {"c": c, "E": E, "H": H, "I": I, "Tp": Tp, "pairs": pairs, "counts": counts}
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    d["gs"], d["go"], d["gpo"], d["gidx"] = (i32(c[k]) for k in ("group_sizes", "group_offsets",
                                                                 "group_padded_offsets", "group_idx_for_bx"))
    d["wg"], d["wu"] = R.quantize_mxfp4(rnd(E, I, H) / H ** 0.5), R.quantize_mxfp4(rnd(E, I, H) / H ** 0.5)
    d["wd"] = R.quantize_mxfp4(rnd(E, H, I) / I ** 0.5)
    cs, ss = R.mxfp4_shapes((Tp, H))
    d["codes"] = torch.randint(0, 256, cs, generator=g, device="cuda", dtype=torch.uint8)
    d["scales"] = torch.full(ss, 0xFF, dtype=torch.uint8, device="cuda")
    d["rw"] = torch.rand(max(pairs, 1), generator=g, device="cuda")[:pairs]
    x = rnd(pairs, H).half()
    prow, cpos = i32(c["padded_row_of_pair"]), i32(c["compact_pos_of_pair"])
    if pairs:
        scratch = torch.empty(pairs, device="cuda")
        R.pack_mxfp4(x, d["rw"], prow, cpos, d["codes"], d["scales"], scratch)
    hc, hs = R.mxfp4_shapes((Tp, I))
    d["hc"] = torch.full(hc, 0x5A, dtype=torch.uint8, device="cuda")
    d["hs"] = torch.full(hs, 0xA5, dtype=torch.uint8, device="cuda")
    d["out"] = torch.full((Tp, H), 0x7E5A, dtype=torch.int16, device="cuda").view(torch.float16)
    return d


def _gate_up(d, variant, **kw):
    R.gate_up_mxfp4(d["codes"], d["scales"], *d["wg"], *d["wu"], d["gs"], d["gpo"], d["gidx"], d["hc"], d["hs"],
                    d["H"], d["pairs"], variant=variant, **kw)


def _down(d, variant, **kw):
    R.down_mxfp4(d["hc"], d["hs"], *d["wd"], d["rw"], d["gs"], d["go"], d["gpo"], d["gidx"], d["out"], d["I"],
                 variant=variant, **kw)


def _val(c, s, cols):
    return torch.from_numpy(MX.values(c.cpu().numpy(), s.cpu().numpy(), cols)).cuda()


MID_LO = torch.tensor([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
MID_HI = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e30], dtype=torch.float64)


def _check(d):
    """Hidden rows and out rows of every group against 64 bits; every other
    row as it was."""
    H, I, c = d["H"], d["I"], d["c"]
    valid = torch.zeros(d["Tp"], dtype=torch.bool, device="cuda")
    lo, hi = MID_LO.cuda(), MID_HI.cuda()
    back = [MX.ORDER.index(b) for b in range(8)]
    for e, n in enumerate(d["counts"]):
        if not n:
            continue
        p, q = int(c["group_padded_offsets"][e]), int(c["group_offsets"][e])
        rows = slice(p, p + n)
        valid[rows] = True
        x = _val(d["codes"][rows], d["scales"][:, rows], H)
        wg, wu = (_val(w[0][e], w[1][e], H) for w in (d["wg"], d["wu"]))
        g, u = x @ wg.T, x @ wu.T
        eg, eu = (H * 2.0 ** -23 * (x.abs() @ w.abs().T) for w in (wg, wu))
        sig = torch.sigmoid(g)
        h = g * sig * u
        err = 1.1 * eg * (u.abs() + eu) + (g * sig).abs() * eu + h.abs() * 2.0 ** -20
        # the stored block scale, the codes under it
        sb = d["hs"][:, rows].transpose(0, 1)[..., back].reshape(n, -1)[:, :I // 32].double() - 127
        unit = torch.exp2(sb).repeat_interleave(32, 1)
        top, et = h.abs().view(n, -1, 32).amax(-1), err.view(n, -1, 32).amax(-1)
        assert (torch.exp2(sb + 2) <= top + et).all() and (top - et < torch.exp2(sb + 3)).all(), (e, n)
        cb = d["hc"][rows]
        code = torch.stack([cb & 15, cb >> 4], -1).view(n, -1)[:, :I].long()
        mag, sign = code & 7, torch.where((code & 8) > 0, -1.0, 1.0)
        a, ea = h * sign / unit, err / unit           # the code's own side is positive
        assert (a >= torch.where(mag == 0, torch.zeros_like(a), lo[mag]) - ea).all(), (e, n)
        assert (a <= hi[mag] + ea).all(), (e, n)
        pad = torch.stack([cb & 15, cb >> 4], -1).view(n, -1)[:, I:]
        assert not pad.any() and not (d["hs"][:, rows].transpose(0, 1)[..., back].reshape(n, -1)[:, I // 32:]).any()
        # out from the hidden rows that were stored
        hq = _val(cb, d["hs"][:, rows], I)
        wd = _val(d["wd"][0][e], d["wd"][1][e], I)
        w = d["rw"][q:q + n].double()[:, None]
        y = (hq @ wd.T) * w
        ey = I * 2.0 ** -23 * (hq.abs() @ wd.abs().T) * w
        bound = ey + (y.abs() + ey) * (F16_HALF_STEP + 2.0 ** -23) + 2.0 ** -25
        assert ((d["out"][rows].double() - y).abs() <= bound).all(), (e, n)
    rest = ~valid
    assert (d["hc"][rest] == 0x5A).all() and (d["hs"][:, rest] == 0xA5).all()
    assert (d["out"][rest].view(torch.int16) == 0x7E5A).all()


SHAPES = [
    ([1], 128, 128), ([0, 1, 0], 256, 128), ([5, 0, 9, 31], 128, 384), ([32, 33, 64, 65], 512, 256),
    ([96, 97, 127, 128, 129], 384, 640), ([255, 256, 257, 0, 300], 640, 384), ([7] * 20, 256, 1408),
    ([1, 500, 2, 90], 2048, 256), ([3, 17], 4096, 128), ([16, 200], 256, 4096),
]


@pytest.mark.parametrize("variant", ["stream", "tile"])
@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_stages(counts, H, I, variant):
    print(f"[mx] {variant} counts={counts} H={H} I={I}", flush=True)
    d = _case(counts, H, I, seed=H + I)
    _gate_up(d, variant)
    _down(d, variant)
    torch.cuda.synchronize()
    _check(d)


@pytest.mark.parametrize("H,I", [(1 << 20, 128), (128, 1 << 20)])
def test_maximum_hidden_and_intermediate(H, I):
    """The largest H and I that the entries take, three rows over two experts:
    both families' out rows against 64 bits on the codes that each stored."""
    print(f"[mx] H={H} I={I}", flush=True)
    d = _case([1, 2], H, I, seed=1)
    val = lambda c, s, cols: R.dequantize_mxfp4(c.contiguous(), s.contiguous(), cols, dtype=torch.float32).double()  # noqa: E731
    for variant in ("stream", "tile"):
        _gate_up(d, variant)
        _down(d, variant)
        torch.cuda.synchronize()
        for e, n in enumerate(d["counts"]):
            p, q = int(d["c"]["group_padded_offsets"][e]), int(d["c"]["group_offsets"][e])
            rows = slice(p, p + n)
            x = val(d["codes"][rows], d["scales"][:, rows], H)
            g, u = x @ val(d["wg"][0][e], d["wg"][1][e], H).T, x @ val(d["wu"][0][e], d["wu"][1][e], H).T
            h, hq = g * torch.sigmoid(g) * u, val(d["hc"][rows], d["hs"][:, rows], I)
            top = h.abs().view(n, -1, 32).amax(-1).repeat_interleave(32, 1)
            # half of E2M1's widest step, or the clamp at 6, of a maximum in [4, 8)
            assert ((hq - h).abs() <= top * 0.5 * (1 + 2.0 ** -10)).all(), (variant, e)
            wd, w = val(d["wd"][0][e], d["wd"][1][e], I), d["rw"][q:q + n].double()[:, None]
            y, ey = (hq @ wd.T) * w, I * 2.0 ** -23 * (hq.abs() @ wd.abs().T) * w
            bound = ey + (y.abs() + ey) * (F16_HALF_STEP + 2.0 ** -23) + 2.0 ** -25
            assert ((d["out"][rows].double() - y).abs() <= bound).all(), (variant, e)


@pytest.mark.parametrize("variant", ["stream", "tile", "auto"])
def test_forward_is_its_stages(variant):
    d = _case([40, 0, 130, 3], 640, 384, seed=4)
    _gate_up(d, variant)
    _down(d, variant)
    ws = torch.full((R.mxfp4_workspace_bytes(d["Tp"], d["I"]),), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full_like(d["out"].view(torch.int16), 0x7E5A).view(torch.float16)
    R.forward_mxfp4(d["codes"], d["scales"], *d["wg"], *d["wu"], *d["wd"], d["rw"], d["gs"], d["go"], d["gpo"],
                    d["gidx"], ws, out, variant=variant)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), d["out"].view(torch.int16))
    rows = torch.from_numpy(np.asarray(d["c"]["padded_row_of_pair"])).long().cuda()
    n = d["hc"].numel()
    assert torch.equal(ws[:n].view(d["hc"].shape)[rows], d["hc"][rows])
    assert torch.equal(ws[n:].view(d["hs"].shape)[:, rows], d["hs"][:, rows])


@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_nan_stays_in_its_row(variant):
    """A token row with an infinity gives NaN in its own row and nowhere else."""
    d = _case([70, 5], 256, 256, seed=9)
    bad = int(d["c"]["group_padded_offsets"][0]) + 33
    d["scales"][0, bad, 2] = 0xFF
    _gate_up(d, variant)
    _down(d, variant)
    torch.cuda.synchronize()
    rows = torch.from_numpy(np.sort(d["c"]["padded_row_of_pair"])).long().cuda()
    nan = torch.isnan(d["out"][rows]).any(1)
    assert torch.isnan(d["out"][bad]).all()
    assert rows[nan].tolist() == [bad]


@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_corrupted_block_table_leaves_rows_unwritten(variant):
    d = _case([140, 20], 256, 128, seed=2)
    d["gidx"][1] = 1                                   # the second block of expert 0
    d["counts"] = [128, 20]
    _gate_up(d, variant)
    _down(d, variant)
    torch.cuda.synchronize()
    _check(d)


@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_graph_replays_on_another_stream(variant):
    d = _case([40, 0, 130, 3], 384, 256, seed=5)
    x = torch.randn(d["pairs"], d["H"], device="cuda").half()
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    prow, cpos = i32(d["c"]["padded_row_of_pair"]), i32(d["c"]["compact_pos_of_pair"])
    wc = torch.empty(d["pairs"], device="cuda")
    ws = torch.empty(R.mxfp4_workspace_bytes(d["Tp"], d["I"]), dtype=torch.uint8, device="cuda")
    other = [torch.empty_like(t) for t in (d["codes"], d["scales"], ws)]

    def layer(codes, scales, work, out):
        R.pack_mxfp4(x, d["rw"], prow, cpos, codes, scales, wc)
        R.forward_mxfp4(codes, scales, *d["wg"], *d["wu"], *d["wd"], wc, d["gs"], d["go"], d["gpo"], d["gidx"], work,
                        out, variant=variant)

    def quantized():
        return R.quantize_mxfp4(x)

    rows = prow.long()
    layer(d["codes"], d["scales"], ws, d["out"])
    torch.cuda.synchronize()
    want, wq = d["out"][rows].clone(), quantized()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qc, qs = torch.empty_like(wq[0]), torch.empty_like(wq[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            layer(d["codes"], d["scales"], ws, d["out"])
            R.quantize_mxfp4(x, qc, qs)
    torch.cuda.synchronize()
    eager = torch.empty_like(d["out"])
    for i in range(4):
        d["out"].fill_(0.0)
        qc.fill_(0)
        layer(other[0], other[1], other[2], eager)    # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d["out"][rows].view(torch.int16), want.view(torch.int16)), i
        assert torch.equal(eager[rows].view(torch.int16), want.view(torch.int16)), i
        assert torch.equal(qc, wq[0]) and torch.equal(qs, wq[1]), i


def test_binding_refusals():
    """Types, shapes, strides, devices and sizes are refused by name before
    anything is launched."""
    d = _case([33, 140], 256, 384, seed=3)
    ws = torch.empty(R.mxfp4_workspace_bytes(d["Tp"], d["I"]), dtype=torch.uint8, device="cuda")
    good = [d["codes"], d["scales"], *d["wg"], *d["wu"], *d["wd"], d["rw"], d["gs"], d["go"], d["gpo"], d["gidx"], ws,
            d["out"]]
    for i, t in enumerate(good):
        bad = [t.cpu(), t.double() if t.dtype is not torch.float64 else t.float()]
        bad += [t.transpose(0, 1)] if t.dim() > 1 else []
        if i == 13:
            bad.append(t[:-1])
        elif i not in (8, 12, 14):                     # counts that define the call's sizes
            bad.append(torch.cat([t, t]))
        for b in bad:
            with pytest.raises((TypeError, ValueError, R.RmoeError)):
                R.forward_mxfp4(*good[:i], b, *good[i + 1:])
    x = torch.zeros(4, 256, device="cuda")
    for kw in (dict(x=x.double()), dict(x=x[:, ::2]), dict(x=x[0]), dict(x=x, codes=torch.zeros(4, 64, device="cuda")),
               dict(x=x, scales=torch.zeros(1, 4, 4, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            R.quantize_mxfp4(**kw)
    with pytest.raises(R.RmoeError):
        R.quantize_mxfp4(torch.zeros(4, 12, device="cuda"))
    torch.cuda.synchronize()
    assert (d["out"].view(torch.int16) == 0x7E5A).all()


def test_two_streams_at_once():
    """Two forwards on different streams share nothing but the weights."""
    d = _case([60, 200, 9], 512, 384, seed=6)
    rows = torch.from_numpy(np.asarray(d["c"]["padded_row_of_pair"])).long().cuda()
    outs, wss, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, variant in zip(streams, ("stream", "tile")):
        outs.append(torch.zeros_like(d["out"]))
        wss.append(torch.empty(R.mxfp4_workspace_bytes(d["Tp"], d["I"]), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, variant, ws, out in zip(streams, ("stream", "tile"), wss, outs):
            R.forward_mxfp4(d["codes"], d["scales"], *d["wg"], *d["wu"], *d["wd"], d["rw"], d["gs"], d["go"],
                            d["gpo"], d["gidx"], ws, out, variant=variant, stream=s)
    torch.cuda.synchronize()
    for variant, out in zip(("stream", "tile"), outs):
        _gate_up(d, variant)
        _down(d, variant)
        torch.cuda.synchronize()
        assert torch.equal(out[rows].view(torch.int16), d["out"][rows].view(torch.int16))
        d["out"].fill_(0)


def test_layer_from_router_to_combine():
    """Router, device contract, MXFP4 pack, forward and combine as a program
    runs them; the sum over a token's experts against the stored rows."""
    T, E, k, H, I = 37, 8, 2, 256, 384
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").half()
    wr = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).half()
    d = _case([3] * E, H, I, seed=8)                   # for its weights
    ids, vals = R.router(x, wr, k)
    t = R.build_contract_device(ids, E)
    Tp = t["total_padded_tokens"]
    cs, ss = R.mxfp4_shapes((Tp, H))
    codes, scales = torch.empty(cs, dtype=torch.uint8, device="cuda"), torch.empty(ss, dtype=torch.uint8, device="cuda")
    w = torch.empty(T * k, device="cuda")
    ws = torch.empty(R.mxfp4_workspace_bytes(Tp, I), dtype=torch.uint8, device="cuda")
    out, y = torch.zeros((Tp, H), dtype=torch.float16, device="cuda"), torch.empty((T, H), dtype=torch.float16, device="cuda")
    R.pack_mxfp4(x, vals.reshape(-1), t["padded_row_of_pair"], t["compact_pos_of_pair"], codes, scales, w)
    R.forward_mxfp4(codes, scales, *d["wg"], *d["wu"], *d["wd"], w, t["group_sizes"], t["group_offsets"],
                    t["group_padded_offsets"], t["group_idx_for_bx"], ws, out)
    R.combine(out, t["padded_row_of_pair"], k, y)
    torch.cuda.synchronize()
    # the tokens' own rows through the oracle's quantisation, each step from the stored one before it
    xq = torch.from_numpy(MX.quantized_values(x.double().cpu().numpy())).cuda()
    n = R.lib().rmoe_mxfp4_code_bytes(Tp, I)
    hcs, hss = R.mxfp4_shapes((Tp, I))
    hq = _val(ws[:n].view(hcs), ws[n:].view(hss), I)
    prow = t["padded_row_of_pair"].view(T, k).long()
    for tok in range(T):
        want, bound = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
        for j in range(k):
            e, r = int(ids[tok, j]), int(prow[tok, j])
            gate = _val(d["wg"][0][e], d["wg"][1][e], H) @ xq[tok]
            up = _val(d["wu"][0][e], d["wu"][1][e], H) @ xq[tok]
            h = gate * torch.sigmoid(gate) * up
            top = h.abs().view(-1, 32).amax(1, keepdim=True).expand(-1, 32).reshape(-1)
            # E2M1's widest half step is 1 of a maximum in [4, 8); clamping at 6 loses up to 2
            assert ((hq[r] - h).abs() <= top * (2 / 4) * (1 + 2.0 ** -18)).all()
            wd = _val(d["wd"][0][e], d["wd"][1][e], I)
            yj = (wd @ hq[r]) * vals[tok, j].double()
            ej = I * 2.0 ** -23 * (wd.abs() @ hq[r].abs()) * vals[tok, j].double()
            want += yj
            bound += ej + (yj.abs() + ej) * (F16_HALF_STEP + 2.0 ** -23) + 2.0 ** -25
        bound += (want.abs() + bound) * (F16_HALF_STEP + 2.0 ** -22) + 2.0 ** -25
        assert ((y[tok].double() - want).abs() <= bound).all(), tok

"""GPU tests of the 8-bit integer entry points against the 64-bit oracle
(oracle/int8.py): quantisation bit for bit, the products within bounds that
follow from their fp32 steps and one final rounding.

Bounds.  Sums of codes' products are exact integers.  Their conversion to
fp32, the product of two scales and its product with the sum round once each:
3 half steps of 2^-24.  silu(g) of a g that is off by a relative d is off by
(1 + |g|) d; its own exponent's argument (2^-24 |g|), the hardware exp2 and
reciprocal (2^-23 each), the addition and the product (2^-24 each) and up's
three half steps and the last product's add up to less than (1 + |g|) 2^-20.
The hidden rows are held in fp32 before they are quantised, so their codes are
the oracle's of the stored rows.  An out value has four half steps of fp32
(less than 2^-21) and fp16's half step, 2^-11 (2^-25 absolute below the normal
numbers)."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import workloads
from oracle import int8 as Q

pytestmark = pytest.mark.gpu
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _same(x, codes, scales):
    """codes and scales are the oracle's of x [rows, cols]."""
    wc, ws = Q.quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), wc)


# ------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_quantize_all_patterns(dtype):
    """Every finite 16-bit pattern (fp32: as high halves, with varied low
    bits), rows of close magnitudes and rows of mixed ones, subnormal rows
    among them."""
    bits = np.arange(65536, dtype=np.uint32)
    v = bits.astype(np.uint16).view(np.float16) if dtype == "f16" else (bits << 16).view(np.float32)
    bits = bits[np.isfinite(v)]
    rng = np.random.default_rng(3)
    order = np.argsort(bits & 0x7FFF, kind="stable")
    both = np.concatenate([bits[order], rng.permutation(bits)])
    both = np.concatenate([both, np.zeros(-both.size % 512, np.uint32)])
    if dtype == "f32":
        x = torch.from_numpy(((both << 16) | rng.integers(0, 65536, both.size).astype(np.uint32)).view(np.float32).reshape(-1, 512).copy())
    else:
        x = torch.from_numpy(both.astype(np.uint16).view(np.int16).reshape(-1, 512).copy()).view(DTYPES[dtype])
    codes, scales = R.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    _same(x, codes, scales)


def test_quantize_next_to_every_border():
    """fp32 values at, right above and right below every midpoint between two
    codes, under many scales, far from one and below the normal numbers."""
    rng = np.random.default_rng(5)
    rows = []
    for i, s in enumerate(rng.uniform(1, 2, 96)):
        s = np.float32(s * 2.0 ** [0, 40, -40, 120, -125, -135][i % 6])
        mid = ((np.arange(-126, 126) + 0.5) * float(s)).astype(np.float32)
        row = np.concatenate([mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(-np.inf))])
        row = np.concatenate([row, [np.float32(127 * float(s))], np.zeros(-(row.size + 1) % 8, np.float32)])
        rows.append(row.astype(np.float32))
    x = torch.from_numpy(np.stack(rows))
    codes, scales = R.quantize_int8(x.cuda())
    torch.cuda.synchronize()
    _same(x, codes, scales)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8), (1, 256), (3, 24), (2, 5, 264), (3, 7, 1416), (130, 4096), (2, 33, 544),
                                   (5000, 512), (4100, 2048), (9, 8200), (3, 16384), (3, 20008), (2, 50000), (40,)])
def test_quantize_shapes_and_way_back(dtype, shape):
    rng = np.random.default_rng(sum(shape))
    x = torch.from_numpy(rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[-1]))).to(DTYPES[dtype])
    codes, scales = R.quantize_int8(x.cuda())
    back = R.dequantize_int8(codes, scales, dtype=x.dtype)
    torch.cuda.synchronize()
    assert codes.shape == x.shape and scales.shape == x.shape[:-1]
    rows = x.reshape(-1, shape[-1])
    some = list(range(rows.shape[0])) if rows.shape[0] < 200 else [0, 1, 3, 4, 1023, rows.shape[0] // 2, rows.shape[0] - 1]
    c, s = codes.reshape(rows.shape).cpu()[some], scales.reshape(-1).cpu()[some]
    _same(rows[some], c, s)
    # a product in fp32, then one rounding to the type
    want = (c.float() * s[:, None]).to(x.dtype)
    assert torch.equal(back.reshape(rows.shape).cpu()[some], want)
    every = (codes.float() * scales[..., None]).to(x.dtype)
    assert torch.equal(back, every)
    # half a code, and the scale's own rounding
    far = (codes.double() * scales.double()[..., None] - x.double().cuda()).abs()
    assert (far <= scales.double()[..., None] * (0.5 + 127 * 2.0 ** -23)).all()


def test_quantize_nonfinite_zero_and_largest_rows():
    x = torch.randn(7, 256)
    x[0, 3], x[1, 40], x[2, 255] = float("nan"), float("inf"), -float("inf")
    x[4], x[5, 7] = 0.0, 65504.0
    for t in DTYPES.values():
        codes, scales = R.quantize_int8(x.to(t).cuda())
        back = R.dequantize_int8(codes, scales, dtype=t).cpu()
        _same(x.to(t), codes, scales)
        assert torch.isnan(back[:3]).all() and torch.isfinite(back[3:]).all() and not back[4].any()
    big = torch.tensor([[torch.finfo(torch.float32).max] + [1e38, -3e38, 1.0, 0, 0, 0, 2e38]])
    _same(big, *R.quantize_int8(big.cuda()))


def test_quantize_past_32_bit_offsets():
    """More than 2^32 elements: rows on both sides of the border."""
    rows, cols = (1 << 21) + 5, 2048
    x = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    some = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 21) - 1, 1 << 21, rows - 1]
    v = torch.randn((len(some), cols), generator=torch.Generator().manual_seed(3)).half()
    x[some] = v.cuda()
    codes, scales = R.quantize_int8(x)
    back = R.dequantize_int8(codes, scales)
    torch.cuda.synchronize()
    _same(v, codes[some], scales[some])
    assert torch.equal(back[some], (codes[some].float() * scales[some][:, None]).half())
    assert int((scales != 0).sum()) == len(some)
    assert int(codes.view(torch.int32).any(1).sum()) == len(some) and int(back.view(torch.int32).any(1).sum()) == len(some)


def test_quantize_many_short_rows():
    rows = (1 << 23) + 70
    x = torch.zeros((rows, 8), dtype=torch.float16, device="cuda")
    some = [0, 31, 32, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, rows - 1]
    v = torch.randn((len(some), 8), generator=torch.Generator().manual_seed(4)).half()
    x[some] = v.cuda()
    codes, scales = R.quantize_int8(x)
    back = R.dequantize_int8(codes, scales)
    torch.cuda.synchronize()
    _same(v, codes[some], scales[some])
    assert int((back != 0).any(1).sum()) == len(some)


# -------------------------------------------------------------------- pack
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 16, 24, 64, 72, 128, 136, 248, 256, 264, 504, 512, 520])
def test_quantize_rows_that_share_a_wave(cols, dtype):
    """One to 64 lanes per row; the last workgroup partly filled; rows of NaN,
    zeros and the largest values beside others."""
    kind = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn((515, cols), generator=g, device="cuda") * torch.exp(3 * torch.randn((515, 1), generator=g, device="cuda"))).to(kind)
    x[3], x[8], x[9] = 0, torch.finfo(kind).max, -torch.finfo(kind).max
    x[5, cols - 1], x[514, 0] = float("nan"), float("inf")
    codes, scales = R.quantize_int8(x)
    alone = [R.quantize_int8(x[r:r + 1]) for r in (0, 4, 6, 256, 513)]
    torch.cuda.synchronize()
    bad = torch.tensor([5, 514], device="cuda")
    good = torch.ones(515, dtype=torch.bool, device="cuda")
    good[bad] = False
    _same(x[good], codes[good], scales[good])
    assert scales[bad].isnan().all() and not codes[bad].any()
    for r, (c, s) in zip((0, 4, 6, 256, 513), alone):
        assert torch.equal(c[0], codes[r]) and torch.equal(s[0], scales[r])


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (5, 3, 264), (130, 2, 512), (700, 8, 1408), (3, 40, 7168), (4, 2, 20000)])
def test_pack(T, k, H):
    rng = np.random.default_rng(T)
    E = max(16, k)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    c = R.build_contract(ids, E)
    prow, cpos = c["padded_row_of_pair"].copy(), c["compact_pos_of_pair"].copy()
    if T > 4:                                         # pairs that the device contract left out
        prow[3], cpos[3] = -1, -1
        prow[4] = c["total_padded_tokens"]
    x = torch.from_numpy(rng.standard_normal((T, H))).half().cuda()
    w = torch.rand(T * k, device="cuda")
    Tp = c["total_padded_tokens"]
    codes = torch.full((Tp, H), 0x5A, dtype=torch.int8, device="cuda")
    scales = torch.full((Tp,), -5.0, device="cuda")
    wc = torch.full((T * k,), -7.0, device="cuda")
    i32 = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    R.pack_int8(x, w, i32(prow), i32(cpos), codes, scales, wc)
    qc, qs = R.quantize_int8(x)
    torch.cuda.synchronize()
    moved = np.zeros(Tp, bool)
    for p in range(T * k):
        r = prow[p]
        if 0 <= r < Tp:
            moved[r] = True
            assert torch.equal(codes[r], qc[p // k]) and scales[r] == qs[p // k]
        if cpos[p] >= 0:
            assert wc[cpos[p]] == w[p]
    rest = torch.from_numpy(~moved).cuda()
    assert (codes[rest] == 0x5A).all() and (scales[rest] == -5.0).all()


# ---------------------------------------------------------------- products
def _case(counts, H, I, seed=0, k=1):
    """Tables for exact group sizes and random operands; token rows outside
    the groups hold garbage under NaN scales, outputs a sentinel."""
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
    d["wg"], d["wu"] = R.quantize_int8(rnd(E, I, H) / H ** 0.5), R.quantize_int8(rnd(E, I, H) / H ** 0.5)
    d["wd"] = R.quantize_int8(rnd(E, H, I) / I ** 0.5)
    d["codes"] = torch.randint(-128, 128, (Tp, H), generator=g, device="cuda", dtype=torch.int8)
    d["scales"] = torch.full((Tp,), float("nan"), device="cuda")
    d["rw"] = torch.rand(max(pairs, 1), generator=g, device="cuda")[:pairs]
    d["x"] = rnd(pairs, H).half()
    d["prow"], d["cpos"] = i32(c["padded_row_of_pair"]), i32(c["compact_pos_of_pair"])
    if pairs:
        R.pack_int8(d["x"], d["rw"], d["prow"], d["cpos"], d["codes"], d["scales"], torch.empty(pairs, device="cuda"))
    d["rows"] = torch.full((Tp, I), 1e30, device="cuda")
    d["hc"] = torch.full((Tp, I), 0x5A, dtype=torch.int8, device="cuda")
    d["hs"] = torch.full((Tp,), -3.0, device="cuda")
    d["out"] = torch.full((Tp, H), 0x7E5A, dtype=torch.int16, device="cuda").view(torch.float16)
    return d


def _tables(d):
    return d["gs"], d["go"], d["gpo"], d["gidx"]


def _gate_up(d, variant, **kw):
    R.gate_up_int8(d["codes"], d["scales"], *d["wg"], *d["wu"], d["gs"], d["gpo"], d["gidx"], d["rows"], d["hc"], d["hs"],
                   d["pairs"], variant=variant, **kw)


def _down(d, variant, **kw):
    R.down_int8(d["hc"], d["hs"], *d["wd"], d["rw"], *_tables(d), d["out"], variant=variant, **kw)


def _forward(d, ws, out, variant, **kw):
    R.forward_int8(d["codes"], d["scales"], *d["wg"], *d["wu"], *d["wd"], d["rw"], *_tables(d), ws, out, variant=variant, **kw)


def _workspace(d, fill=0x5A):
    return torch.full((R.int8_workspace_bytes(d["Tp"], d["I"]),), fill, dtype=torch.uint8, device="cuda")


def _check(d):
    """Hidden rows, their codes and out rows of every group against 64 bits;
    every other row as it was."""
    c = d["c"]
    valid = torch.zeros(d["Tp"], dtype=torch.bool, device="cuda")
    for e, n in enumerate(d["counts"]):
        if not n:
            continue
        p, q = int(c["group_padded_offsets"][e]), int(c["group_offsets"][e])
        rows = slice(p, p + n)
        valid[rows] = True
        x, xs = d["codes"][rows].double(), d["scales"][rows].double()[:, None]
        g, u = ((x @ w[0][e].double().T) * xs * w[1][e].double() for w in (d["wg"], d["wu"]))
        h = g * torch.sigmoid(g) * u
        off = (d["rows"][rows].double() - h).abs()
        assert (off <= h.abs() * (1 + g.abs()) * 2.0 ** -20 + 2.0 ** -120).all(), (e, n)
        _same(d["rows"][rows], d["hc"][rows], d["hs"][rows])
        y = (d["hc"][rows].double() @ d["wd"][0][e].double().T) * d["hs"][rows].double()[:, None] * d["wd"][1][e].double()
        y = y * d["rw"][q:q + n].double()[:, None]
        off = (d["out"][rows].double() - y).abs()
        assert (off <= y.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25).all(), (e, n)
    rest = ~valid
    assert (d["rows"][rest] == 1e30).all() and (d["hc"][rest] == 0x5A).all() and (d["hs"][rest] == -3.0).all()
    assert (d["out"][rest].view(torch.int16) == 0x7E5A).all()


SHAPES = [
    ([1], 128, 128), ([0, 1, 0], 256, 128), ([5, 0, 9, 31], 128, 384), ([32, 33, 64, 65], 512, 256),
    ([96, 97, 127, 128, 129], 384, 640), ([255, 256, 257, 0, 300], 640, 384), ([7] * 20, 256, 1408),
    ([1, 500, 2, 90], 2048, 256), ([3, 17], 4096, 128), ([16, 200], 256, 4096), ([2, 130], 128, 16512),
]


@pytest.mark.parametrize("variant", ["stream", "tile"])
@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_stages(counts, H, I, variant):
    print(f"[int8] {variant} counts={counts} H={H} I={I}", flush=True)
    d = _case(counts, H, I, seed=H + I)
    _gate_up(d, variant)
    _down(d, variant)
    torch.cuda.synchronize()
    _check(d)


@pytest.mark.parametrize("counts,I", [([3, 0, 40], 2048), ([3, 0, 40], 2176), ([3, 0, 40], 8320), ([3, 0, 40], 24576),
                                      ([1, 33], 33024), ([1024], 2176), ([5, 1020], 2176)])
def test_few_and_many_long_hidden_rows(counts, I):
    """Hidden rows shared by 4 and by 16 waves, of one to eight vectors a lane and of more."""
    print(f"[int8] counts={counts} I={I}", flush=True)
    d = _case(counts, 128, I, seed=I)
    _gate_up(d, "auto")
    _down(d, "auto")
    torch.cuda.synchronize()
    _check(d)


@pytest.mark.parametrize("H,I", [(133120, 128), (128, 133120)])
@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_maximum_hidden_and_intermediate(H, I, variant):
    """The largest H and I that the entries take, every code 127 or -127: the
    sums reach 127^2 133120, next to 2^31."""
    print(f"[int8] {variant} H={H} I={I}", flush=True)
    d = _case([1, 2], H, I, seed=1)
    d["codes"].fill_(127)
    d["wg"][0].fill_(127)
    d["wu"][0].fill_(-127)
    if H > I:
        for w in (d["wg"], d["wu"]):
            w[1].fill_(1.0 / (127 * 127 * H))
        d["scales"].fill_(1.0)
    _gate_up(d, variant)
    if I > H:
        # as if the hidden rows had come out equal
        d["hc"].fill_(127)
        d["hs"].fill_(1.0 / (127 * I))
        d["wd"][0].fill_(-127)
        _down(d, variant)
        torch.cuda.synchronize()
        for e, n in enumerate(d["counts"]):
            p, q = int(d["c"]["group_padded_offsets"][e]), int(d["c"]["group_offsets"][e])
            y = -127.0 * 127 * I * d["hs"][p].double() * d["wd"][1][e].double() * d["rw"][q:q + n].double()[:, None]
            assert ((d["out"][p:p + n].double() - y).abs() <= y.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25).all()
    else:
        _down(d, variant)
        torch.cuda.synchronize()
        _check(d)


@pytest.mark.parametrize("variant", ["stream", "tile", "auto"])
def test_forward_is_its_stages(variant):
    d = _case([40, 0, 130, 3], 640, 384, seed=4)
    _gate_up(d, variant)
    _down(d, variant)
    ws, out = _workspace(d), torch.full_like(d["out"].view(torch.int16), 0x7E5A).view(torch.float16)
    _forward(d, ws, out, variant)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), d["out"].view(torch.int16))
    rows, n = d["prow"].long(), d["hc"].numel()
    assert torch.equal(ws[:n].view(torch.int8).view(d["hc"].shape)[rows], d["hc"][rows])
    assert torch.equal(ws[5 * n:].view(torch.float32)[rows], d["hs"][rows])


@pytest.mark.parametrize("counts,H,I", [([40, 0, 130, 3], 128, 4096), ([256], 256, 2176), ([700], 384, 8320), ([1], 128, 16384),
                                        ([300, 129], 1152, 2432), ([5, 0, 260], 640, 2048), ([128] * 9, 512, 3968)])
def test_forward_in_parts_of_k(counts, H, I):
    """Few tiles of out and a long K: the forward cuts the sums into parts,
    whose results are those of the stage alone, which has no room for them."""
    print(f"[int8] parts counts={counts} H={H} I={I}", flush=True)
    d = _case(counts, H, I, seed=I)
    _gate_up(d, "tile")
    _down(d, "tile")
    ws, out = _workspace(d), torch.full_like(d["out"].view(torch.int16), 0x7E5A).view(torch.float16)
    for _ in range(2):
        _forward(d, ws, out, "tile")
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), d["out"].view(torch.int16))
    _check(d)


def test_families_agree_bit_for_bit():
    d = _case([60, 200, 9, 0, 128], 512, 384, seed=6)
    got = []
    for variant in ("stream", "tile"):
        _gate_up(d, variant)
        _down(d, variant)
        torch.cuda.synchronize()
        got.append((d["rows"].clone(), d["hc"].clone(), d["hs"].clone(), d["out"].view(torch.int16).clone()))
        d["out"].view(torch.int16).fill_(0x7E5A)
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_nan_and_zero_rows_stay_by_themselves(variant):
    """A token row with an infinity gives NaN in its own row and nowhere else;
    a row of zeros gives zeros."""
    d = _case([70, 5], 256, 256, seed=9)
    x = d["x"].clone()
    prow = d["prow"].long()
    x[3, 7], x[11, 100], x[20] = float("inf"), float("nan"), 0.0
    R.pack_int8(x, d["rw"], d["prow"], d["cpos"], d["codes"], d["scales"], torch.empty(d["pairs"], device="cuda"))
    _gate_up(d, variant)
    _down(d, variant)
    torch.cuda.synchronize()
    out = d["out"][prow]
    assert torch.isnan(out[[3, 11]]).all() and int(torch.isnan(out).any(1).sum()) == 2
    assert not out[20].any()


def test_corrupted_block_table_in_parts_of_k():
    d = _case([300, 129], 256, 4096, seed=12)
    _gate_up(d, "tile")
    _down(d, "tile")
    torch.cuda.synchronize()
    want, blocks = d["out"].view(torch.int16).clone(), d["gidx"].clone()
    for bad in (1, -1, 7, 2 ** 31 - 1):              # block 1 belongs to expert 0
        d["gidx"].copy_(blocks)
        d["gidx"][1] = bad
        ws, out = _workspace(d), torch.full_like(want, 0x7E5A)
        _forward(d, ws, out.view(torch.float16), "tile")
        torch.cuda.synchronize()
        assert (out[128:256] == 0x7E5A).all()
        assert torch.equal(out[:128], want[:128]) and torch.equal(out[256:], want[256:])


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
    wc, ws = torch.empty(d["pairs"], device="cuda"), _workspace(d)
    other = [torch.empty_like(t) for t in (d["codes"], d["scales"], ws)]

    def layer(codes, scales, work, out):
        R.pack_int8(d["x"], d["rw"], d["prow"], d["cpos"], codes, scales, wc)
        R.forward_int8(codes, scales, *d["wg"], *d["wu"], *d["wd"], wc, *_tables(d), work, out, variant=variant)

    rows = d["prow"].long()
    layer(d["codes"], d["scales"], ws, d["out"])
    wq = R.quantize_int8(d["x"])
    torch.cuda.synchronize()
    want = d["out"][rows].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qc, qs = torch.empty_like(wq[0]), torch.empty_like(wq[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            layer(d["codes"], d["scales"], ws, d["out"])
            R.quantize_int8(d["x"], qc, qs)
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


def test_graph_replays_in_parts_of_k():
    d = _case([200, 64], 128, 4096, seed=13)
    ws, out = _workspace(d), torch.full_like(d["out"].view(torch.int16), 0x7E5A).view(torch.float16)
    _forward(d, ws, out, "tile")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _forward(d, ws, out, "tile")
    for i in range(3):
        d["codes"].copy_(d["codes"].roll(i + 1, 1))
        graph.replay()
        _gate_up(d, "stream")
        _down(d, "stream")
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), d["out"].view(torch.int16))
        ws.fill_(0x11)


def test_two_streams_at_once():
    """Two forwards on different streams share nothing but the weights."""
    d = _case([60, 200, 9], 512, 384, seed=6)
    rows = d["prow"].long()
    both, streams = ("stream", "tile"), [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.zeros_like(d["out"]) for _ in both], [_workspace(d) for _ in both]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, variant, ws, out in zip(streams, both, wss, outs):
            _forward(d, ws, out, variant, stream=s)
    torch.cuda.synchronize()
    _gate_up(d, "tile")
    _down(d, "tile")
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out[rows].view(torch.int16), d["out"][rows].view(torch.int16))


def test_binding_refusals():
    """Types, shapes, strides, devices and sizes are refused by name before
    anything is launched."""
    d = _case([33, 140], 256, 384, seed=3)
    good = [d["codes"], d["scales"], *d["wg"], *d["wu"], *d["wd"], d["rw"], *_tables(d), _workspace(d), d["out"]]
    for i, t in enumerate(good):
        bad = [t.cpu(), t.double() if t.dtype is not torch.float64 else t.float()]
        bad += [t.transpose(0, 1)] if t.dim() > 1 else []
        if i == 13:
            bad.append(t[:-1])
        elif i not in (8, 12, 14):                     # counts that define the call's sizes
            bad.append(torch.cat([t, t]))
        for b in bad:
            with pytest.raises((TypeError, ValueError, R.RmoeError)):
                R.forward_int8(*good[:i], b, *good[i + 1:])
    x = torch.zeros(4, 256, device="cuda")
    for kw in (dict(x=x.double()), dict(x=x[:, ::2]), dict(x=x, codes=torch.zeros(4, 256, device="cuda")),
               dict(x=x, scales=torch.zeros(5, device="cuda")), dict(x=x, scales=torch.zeros(4, 1, device="cuda")),
               dict(x=x, codes=torch.zeros(4, 128, dtype=torch.int8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            R.quantize_int8(**kw)
    with pytest.raises(R.RmoeError):
        R.quantize_int8(torch.zeros(4, 12, device="cuda"))
    torch.cuda.synchronize()
    assert (d["out"].view(torch.int16) == 0x7E5A).all()


def test_layer_from_router_to_combine():
    """Router, device contract, 8-bit pack, forward and combine as a program
    runs them, against 64 bits from the stored hidden codes on."""
    T, E, k, H, I = 37, 8, 2, 256, 384
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").half()
    wr = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).half()
    d = _case([3] * E, H, I, seed=8)                   # for its weights
    ids, vals = R.router(x, wr, k)
    t = R.build_contract_device(ids, E)
    Tp = t["total_padded_tokens"]
    codes, scales = torch.empty((Tp, H), dtype=torch.int8, device="cuda"), torch.empty(Tp, device="cuda")
    w = torch.empty(T * k, device="cuda")
    ws = torch.empty(R.int8_workspace_bytes(Tp, I), dtype=torch.uint8, device="cuda")
    out, y = torch.zeros((Tp, H), dtype=torch.float16, device="cuda"), torch.empty((T, H), dtype=torch.float16, device="cuda")
    R.pack_int8(x, vals.reshape(-1), t["padded_row_of_pair"], t["compact_pos_of_pair"], codes, scales, w)
    R.forward_int8(codes, scales, *d["wg"], *d["wu"], *d["wd"], w, t["group_sizes"], t["group_offsets"],
                   t["group_padded_offsets"], t["group_idx_for_bx"], ws, out)
    R.combine(out, t["padded_row_of_pair"], k, y)
    torch.cuda.synchronize()
    xq = torch.from_numpy(Q.values(*Q.quantize(x.double().cpu().numpy()))).cuda()
    n = Tp * I
    hc, hs = ws[:n].view(torch.int8).view(Tp, I).double(), ws[5 * n:].view(torch.float32).double()
    prow = t["padded_row_of_pair"].view(T, k).long()
    value = lambda m, e: m[0][e].double() * m[1][e].double()[:, None]  # noqa: E731
    for tok in range(T):
        want, bound = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
        for j in range(k):
            e, r = int(ids[tok, j]), int(prow[tok, j])
            gate, up = value(d["wg"], e) @ xq[tok], value(d["wu"], e) @ xq[tok]
            h = gate * torch.sigmoid(gate) * up
            # half a code under the stored scale, and fp32's steps
            assert ((hc[r] * hs[r] - h).abs() <= hs[r] * 0.5 + h.abs() * (1 + gate.abs()) * 2.0 ** -19).all()
            yj = (value(d["wd"], e) @ (hc[r] * hs[r])) * vals[tok, j].double()
            want += yj
            bound += yj.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25
        bound += (want.abs() + bound) * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25
        assert ((y[tok].double() - want).abs() <= bound).all(), tok

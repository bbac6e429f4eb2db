"""GPU tests of the training forward and the backward pass against 64 bits
(oracle/train.py), stage by stage: each stage's outputs from the stored
inputs of that stage, so that a bound covers that stage's own roundings.

Bounds.  A product of two fp16 numbers is exact in fp32; a sum of K of them
carries at most K additions' rounding, |error| <= K 2^-23 sum|a b| (2^-23 per
addition allows for a truncating adder).  The sigmoid (hardware exp2 and
reciprocal) and the few fp32 operations around it add a relative 2^-19 of
each term.  An fp16 output adds half a step: 2^-11 of the value, 2^-25 below
the normal numbers."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import workloads
from oracle import train as TR

pytestmark = pytest.mark.gpu
SUM, FN = 2.0 ** -23, 2.0 ** -19
BITS = 0x7E5A    # sentinel of rows that no call may write (an fp16 NaN)


def _near(got, want, err, what):
    """got (fp16) is want within err and one rounding."""
    off = (got.double() - want).abs()
    bound = err + (want.abs() + err) * 2.0 ** -11 + 2.0 ** -25
    bad = off > bound
    assert not bad.any() and not torch.isnan(got).any(), \
        f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((off / bound).max()):.3g} of the bound"


def _case(counts, H, I, seed=0, tables=None):
    """Tables for exact group sizes and random inputs; padding rows of every
    input hold NaN, every output the sentinel."""
    E = len(counts)
    c = R.build_contract(workloads.routing_from_counts(counts, seed=seed), E)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    Tp, pairs = c["total_padded_tokens"], c["pairs"]
    d = {"c": c, "E": E, "H": H, "I": I, "Tp": Tp, "pairs": pairs, "counts": list(counts)}
    d["gs"], d["go"], d["gpo"], d["gidx"] = (i32(c[k]) for k in ("group_sizes", "group_offsets",
                                                                 "group_padded_offsets", "group_idx_for_bx"))
    rows = i32(c["padded_row_of_pair"]).long()
    d["rows"] = rows
    bits = lambda *s: torch.full(s, BITS, dtype=torch.int16, device="cuda").view(torch.float16)  # noqa: E731

    def padded(cols, scale=1.0):
        t = bits(Tp, cols)
        t[rows] = rnd(pairs, cols) * scale
        return t

    d["x"], d["dout"] = padded(H), padded(H)
    d["wg"], d["wu"], d["wd"] = rnd(E, I, H) / H ** 0.5, rnd(E, I, H) / H ** 0.5, rnd(E, H, I) / I ** 0.5
    d["rw"] = torch.rand(max(pairs, 1), generator=g, device="cuda")[:pairs]
    for n in ("gate", "up", "hidden", "dgate", "dup", "whidden"):
        d[n] = bits(Tp, I)
    d["dx"] = bits(Tp, H)
    d["dgw"], d["duw"], d["ddw"] = bits(E, I, H), bits(E, I, H), bits(E, H, I)
    d["drw"] = torch.full((pairs,), float("nan"), device="cuda")
    d["scratch"] = torch.full((R.backward_scratch_bytes(pairs, I) // 4 or 1,), float("nan"), device="cuda")
    return d


def _forward(d, **kw):
    R.gate_up_train(d["x"], d["wg"], d["wu"], d["gs"], d["gpo"], d["gidx"], d["gate"], d["up"], d["hidden"], **kw)


def _backward(d, dgate="dgate", dup="dup", **kw):
    R.backward(d["x"], d["dout"], d["wg"], d["wu"], d["wd"], d["rw"], d["gate"], d["up"], d["gs"], d["go"], d["gpo"],
               d["gidx"], d[dgate], d[dup], d["whidden"], d["scratch"], d["dx"], d["dgw"], d["duw"], d["ddw"],
               d["drw"], **kw)


def _groups(d):
    c = d["c"]
    for e, n in enumerate(d["counts"]):
        p, q = int(c["group_padded_offsets"][e]), int(c["group_offsets"][e])
        yield e, n, slice(p, p + n), slice(q, q + n)


def _untouched(d, names):
    rest = torch.ones(d["Tp"], dtype=torch.bool, device="cuda")
    for _, _, rows, _ in _groups(d):
        rest[rows] = False
    for n in names:
        assert (d[n][rest].view(torch.int16) == BITS).all(), n


def _check_forward(d):
    for e, n, rows, _ in _groups(d):
        if not n:
            continue
        x, wg, wu = d["x"][rows].double(), d["wg"][e].double(), d["wu"][e].double()
        g, u = x @ wg.T, x @ wu.T
        eg, eu = d["H"] * SUM * (x.abs() @ wg.abs().T), d["H"] * SUM * (x.abs() @ wu.abs().T)
        _near(d["gate"][rows], g, eg, f"gate {e}")
        _near(d["up"][rows], u, eu, f"up {e}")
        sl = g * torch.sigmoid(g)
        _near(d["hidden"][rows], sl * u, 1.1 * eg * (u.abs() + eu) + sl.abs() * eu + (sl * u).abs() * FN, f"hidden {e}")
    _untouched(d, ["gate", "up", "hidden"])


def _check_backward(d, gate="gate", up="up"):
    H, I = d["H"], d["I"]
    for e, n, rows, at in _groups(d):
        if not n:
            for m in ("dgw", "duw", "ddw"):
                assert (d[m][e].view(torch.int16) == 0).all(), (m, e)
            continue
        x, dy, g, u = (d[m][rows].double() for m in ("x", "dout", gate, up))
        wg, wu, wd, w = d["wg"][e].double(), d["wu"][e].double(), d["wd"][e].double(), d["rw"][at].double()
        b, dg, du, hw, drw = TR.hidden_grads(dy, wd, w, g, u)
        eb = H * SUM * (dy.abs() @ wd.abs())
        s = torch.sigmoid(g)
        terms = w[:, None] * (s + (g * s).abs() * (1 - s))           # silu' without cancellation
        _near(d["dgate"][rows], dg, u.abs() * terms * (eb + (b.abs() + eb) * FN), f"dgate {e}")
        _near(d["dup"][rows], du, w[:, None] * (g * s).abs() * (eb + (b.abs() + eb) * FN), f"dup {e}")
        _near(d["whidden"][rows], hw, hw.abs() * FN, f"whidden {e}")
        h = (g * s * u).abs()
        bound = (eb * h).sum(1) + (FN + I * 2.0 ** -24) * ((b.abs() + eb) * h).sum(1)
        assert ((d["drw"][at].double() - drw).abs() <= bound).all(), f"drw {e}"
        # the products of the stored dgate, dup and whidden
        dg, du, hw = (d[m][rows].double() for m in ("dgate", "dup", "whidden"))
        _near(d["dx"][rows], dg @ wg + du @ wu, 2 * I * SUM * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()), f"dx {e}")
        for m, l, r in (("dgw", dg, x), ("duw", du, x), ("ddw", dy, hw)):
            _near(d[m][e], l.T @ r, n * SUM * (l.abs().T @ r.abs()), f"{m} {e}")


SHAPES = [
    ([1], 128, 128), ([0, 1, 0], 256, 128), ([5, 0, 9, 31], 128, 384), ([32, 33, 63, 64, 65], 512, 256),
    ([96, 97, 127, 128, 129], 384, 640), ([191, 192, 193, 0, 300], 640, 384), ([255, 256, 257], 256, 256),
    ([7] * 20, 256, 1408), ([1, 500, 2, 90], 2048, 256), ([3, 17], 4096, 128), ([16, 200], 256, 4096),
    ([0, 0, 0], 128, 256),
]


@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_forward_and_backward(counts, H, I):
    print(f"[train] counts={counts} H={H} I={I}", flush=True)
    d = _case(counts, H, I, seed=H + I)
    _forward(d)
    torch.cuda.synchronize()
    _check_forward(d)
    print("[train] backward", flush=True)
    _backward(d)
    torch.cuda.synchronize()
    _check_backward(d)
    _untouched(d, ["dgate", "dup", "whidden", "dx"])


def test_hidden_rows_are_the_tiled_forwards():
    """gate_up_train's hidden rows are gate_up's, bit for bit."""
    d = _case([40, 0, 130, 3], 640, 384, seed=4)
    _forward(d)
    other = torch.full_like(d["hidden"].view(torch.int16), BITS).view(torch.float16)
    R.gate_up(d["x"], d["wg"], d["wu"], d["gs"], d["gpo"], d["gidx"], other, d["pairs"], variant="tile")
    torch.cuda.synchronize()
    assert torch.equal(other.view(torch.int16), d["hidden"].view(torch.int16))


def test_in_place_and_equal_bits():
    """dgate and dup may take the memory of gate and up; a second call gives
    the same bits."""
    d = _case([70, 5, 0, 300], 384, 384, seed=7)
    _forward(d)
    _backward(d)
    torch.cuda.synchronize()
    names = ("dgate", "dup", "whidden", "dx", "dgw", "duw", "ddw")
    want = {n: d[n].clone() for n in names}
    drw = d["drw"].clone()
    d["whidden"].fill_(0)
    _backward(d, dgate="gate", dup="up")
    torch.cuda.synchronize()
    r = d["rows"]
    assert torch.equal(d["gate"][r], want["dgate"][r]) and torch.equal(d["up"][r], want["dup"][r])
    for n in ("whidden", "dx"):
        assert torch.equal(d[n][r], want[n][r]), n
    for n in ("dgw", "duw", "ddw"):
        assert torch.equal(d[n], want[n]), n
    assert torch.equal(d["drw"], drw)


# two items of 256 rows; few long items, so that most workgroups start on the
# weight gradients while the others work on dx; more items than workgroups and
# a last, partly free round of them; uneven and empty groups
@pytest.mark.parametrize("counts,H,I", [([33, 140], 256, 384), ([700, 600, 700, 500], 1024, 4096),
                                        ([2000, 0, 30, 900, 6000], 2048, 8192), ([0, 0, 3, 0], 384, 1152),
                                        ([1] * 40, 512, 512)])
def test_stages_are_the_whole(counts, H, I):
    d = _case(counts, H, I, seed=3)
    _forward(d)
    _backward(d)
    torch.cuda.synchronize()
    w = {n: d[n].clone() for n in ("dgate", "dup", "whidden", "dx", "dgw", "duw", "ddw", "drw")}
    for n in w:
        d[n].fill_(7.0)
    R.down_backward(d["dout"], d["wd"], d["rw"], d["gate"], d["up"], d["gs"], d["go"], d["gpo"], d["gidx"], d["dgate"],
                    d["dup"], d["whidden"], d["scratch"], d["drw"])
    R.gate_up_backward(d["dgate"], d["dup"], d["wg"], d["wu"], d["gs"], d["gpo"], d["gidx"], d["dx"])
    R.weight_grad(d["x"], d["dout"], d["dgate"], d["dup"], d["whidden"], d["gs"], d["gpo"], d["dgw"], d["duw"], d["ddw"])
    torch.cuda.synchronize()
    r = d["rows"]
    for n in ("dgate", "dup", "whidden", "dx"):
        assert torch.equal(d[n][r], w[n][r]), n
    for n in ("dgw", "duw", "ddw", "drw"):
        assert torch.equal(d[n], w[n]), n


def test_gradients_against_differences():
    """The gradients along random directions against central differences of
    the 64-bit forward.  Each gradient carries the fp16 roundings of the kept
    gate and up (each through a factor of silu or silu' of at most about 2),
    of dgate, dup or whidden, and its own: under 8 half steps of 2^-11 of its
    norm, whatever the direction."""
    d = _case([50, 21], 256, 128, seed=5)
    _forward(d)
    _backward(d)
    torch.cuda.synchronize()
    for e, n, rows, at in _groups(d):
        x, dy = d["x"][rows].double(), d["dout"][rows].double()
        base = [x, d["wg"][e].double(), d["wu"][e].double(), d["wd"][e].double(), d["rw"][at].double()]
        got = [d["dx"][rows], d["dgw"][e], d["duw"][e], d["ddw"][e], d["drw"][at]]
        for i in range(5):
            g = torch.Generator(device="cuda").manual_seed(10 * e + i)
            v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
            lo, hi = list(base), list(base)
            lo[i], hi[i] = base[i] - 1e-5 * v, base[i] + 1e-5 * v
            diff = float(((TR.forward(*hi) - TR.forward(*lo)) * dy).sum() / 2e-5)
            gi = got[i].double()
            assert abs(diff - float((gi * v).sum())) <= 8 * 2.0 ** -11 * float(gi.norm() * v.norm()), (e, i)


def test_extreme_gates():
    """Gates at both ends of fp16, zeros of both signs: finite gradients that
    follow the formula."""
    d = _case([40], 128, 256, seed=6)
    _forward(d)
    g = torch.tensor([65504.0, -65504.0, 100.0, -100.0, 20.0, -20.0, 0.0, -0.0, 2.0 ** -24, -2.0 ** -14],
                     device="cuda").half()
    d["gate"][d["rows"]] = g.repeat(26)[:256].expand(40, 256).clone()
    d["up"][d["rows"]] = d["up"][d["rows"]].clamp(-0.01, 0.01)   # products stay inside fp16
    d["wd"].mul_(0.1)
    _backward(d)
    torch.cuda.synchronize()
    r = d["rows"]
    keep = (d["dgate"], d["dup"], d["whidden"])
    kept = {n: d[n][r].clone() for n in ("dgate", "dup", "whidden", "gate", "up")}
    fin = torch.isfinite
    ok = fin(keep[0][r]) & fin(keep[2][r])
    assert ok.all()
    x, dy, gg, u = (d[m][r].double() for m in ("x", "dout", "gate", "up"))
    order = torch.from_numpy(np.asarray(d["c"]["compact_pos_of_pair"])).long().cuda()
    w = d["rw"][order].double()
    b, dg, du, hw, _ = TR.hidden_grads(dy, d["wd"][0].double(), w, gg, u)
    eb = 128 * SUM * (dy.abs() @ d["wd"][0].double().abs())
    s = torch.sigmoid(gg)
    _near(d["dgate"][r], dg, u.abs() * w[:, None] * (s + (gg * s).abs() * (1 - s)) * (eb + (b.abs() + eb) * FN), "dgate")
    _near(d["whidden"][r], hw, hw.abs() * FN, "whidden")
    # a gate or up row that left fp16's range counts as the largest number
    inf = torch.full_like(d["gate"][r], float("inf"))
    for n in ("gate", "up"):
        d[n][r] = torch.where(kept[n].abs() == 65504, torch.copysign(inf, kept[n]), kept[n])
    assert torch.isinf(d["gate"][r]).any()
    _backward(d)
    torch.cuda.synchronize()
    for n in ("dgate", "dup", "whidden"):
        assert torch.equal(d[n][r], kept[n]), n
    d["gate"][int(r[3])] = float("nan")               # and NaN stays NaN
    _backward(d)
    torch.cuda.synchronize()
    assert torch.isnan(d["dgate"][int(r[3])]).all() and not torch.isnan(d["dgate"][int(r[4])]).any()


def test_pairs_left_out_by_the_contract():
    """Pairs with an expert id out of range have no row and no compact place:
    the places past the last valid pair keep what they held."""
    T, k, E, H, I = 30, 2, 4, 128, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)   # repeats allowed
    ids[5, 1], ids[20, 0] = E, -1
    t = R.build_contract_device(ids, E)
    Tp, pairs = t["total_padded_tokens"], t["pairs"]
    tables = (t["group_sizes"], t["group_offsets"], t["group_padded_offsets"], t["group_idx_for_bx"])
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    bits = lambda *s: torch.full(s, BITS, dtype=torch.int16, device="cuda").view(torch.float16)  # noqa: E731
    w, prow = torch.full((pairs,), float("nan"), device="cuda"), t["padded_row_of_pair"]
    xs, dys = bits(Tp, H), bits(Tp, H)
    for src, dst in ((rnd(T, H), xs), (rnd(T, H), dys)):
        R.pack(src, torch.rand(pairs, generator=g, device="cuda"), prow, t["compact_pos_of_pair"], dst, w)
    d = {"c": R.build_contract(ids.cpu().clamp(0, E - 1).numpy(), E), "E": E, "H": H, "I": I, "Tp": Tp, "pairs": pairs}
    torch.cuda.synchronize()
    sizes, offsets, starts = (x.cpu().numpy() for x in tables[:3])
    d["c"] = {"group_padded_offsets": starts, "group_offsets": offsets}
    d["counts"] = sizes.tolist()
    assert sum(d["counts"]) == pairs - 2
    d.update(x=xs, dout=dys, wg=rnd(E, I, H), wu=rnd(E, I, H), wd=rnd(E, H, I), rw=w, gs=tables[0], go=tables[1],
             gpo=tables[2], gidx=tables[3])
    for n in ("gate", "up", "hidden", "dgate", "dup", "whidden"):
        d[n] = bits(Tp, I)
    d["dx"], d["dgw"], d["duw"], d["ddw"] = bits(Tp, H), bits(E, I, H), bits(E, I, H), bits(E, H, I)
    d["drw"] = torch.full((pairs,), -7.0, device="cuda")
    d["scratch"] = torch.full((R.backward_scratch_bytes(pairs, I) // 4,), float("nan"), device="cuda")
    _forward(d)
    torch.cuda.synchronize()
    _check_forward(d)
    _backward(d)
    torch.cuda.synchronize()
    _check_backward(d)
    _untouched(d, ["dgate", "dup", "whidden", "dx"])
    assert (d["drw"][-2:] == -7.0).all()


@pytest.mark.parametrize("H,I", [(1 << 20, 128), (128, 1 << 20)])
def test_maximum_hidden_and_intermediate(H, I):
    """The largest H and I that the entries take, three rows over two experts."""
    print(f"[train] H={H} I={I}", flush=True)
    d = _case([1, 2], H, I, seed=1)
    _forward(d)
    torch.cuda.synchronize()
    _check_forward(d)
    _backward(d)
    torch.cuda.synchronize()
    _check_backward(d)


def test_corrupted_tables_read_nothing_out_of_bounds():
    """A block mapped to another expert leaves its rows unwritten; a group
    that would reach past the last row is left out of the weight gradients."""
    d = _case([140, 20], 256, 128, seed=2)
    _forward(d)
    torch.cuda.synchronize()
    saved = d["gidx"].clone()
    d["gidx"][1] = 1
    R.gate_up_backward(d["gate"], d["up"], d["wg"], d["wu"], d["gs"], d["gpo"], d["gidx"], d["dx"])
    torch.cuda.synchronize()
    assert (d["dx"][128:256].view(torch.int16) == BITS).all()
    assert not torch.isnan(d["dx"][:128]).any()
    d["gidx"].copy_(saved)
    d["dgate"].fill_(0), d["dup"].fill_(0), d["whidden"].fill_(0)
    d["gpo"][1] = d["Tp"] - 64 + 128
    R.weight_grad(d["x"], d["dout"], d["dgate"], d["dup"], d["whidden"], d["gs"], d["gpo"], d["dgw"], d["duw"], d["ddw"])
    torch.cuda.synchronize()
    assert (d["dgw"][1].view(torch.int16) == BITS).all() and (d["ddw"][1].view(torch.int16) == BITS).all()
    assert (d["dgw"][0] == 0).all()


def test_binding_refusals():
    """Types, shapes, strides, devices and sizes are refused by name before
    anything is launched."""
    d = _case([33, 140], 256, 384, seed=3)
    good = [d[n] for n in ("x", "dout", "wg", "wu", "wd", "rw", "gate", "up", "gs", "go", "gpo", "gidx", "dgate", "dup",
                           "whidden", "scratch", "dx", "dgw", "duw", "ddw", "drw")]
    for i, t in enumerate(good):
        bad = [t.cpu(), t.double() if t.dtype is not torch.int32 else t.long()] + ([t.t()] if t.dim() == 2 else [])
        if i != 15:                                    # scratch: any shape and type that is long enough
            bad.append(torch.cat([t, t]))
        else:
            bad = [t.cpu(), t[:-1]]
        for b in bad:
            if i == 5 and b.shape != t.shape:
                continue                               # the routed weights' count is the pair count itself
            with pytest.raises((TypeError, ValueError, R.RmoeError)):
                R.backward(*good[:i], b, *good[i + 1:])
    with pytest.raises(TypeError):
        R.backward(None, *good[1:])
    torch.cuda.synchronize()
    assert (d["dx"].view(torch.int16) == BITS).all() and (d["dgw"].view(torch.int16) == BITS).all()


def test_graph_replays_and_two_streams():
    d = _case([60, 0, 200, 9], 384, 256, seed=8)
    names = ("dgate", "dup", "whidden", "dx", "dgw", "duw", "ddw", "drw", "gate", "up", "hidden")

    def step(t, **kw):
        _forward(t, **kw)
        _backward(t, **kw)

    step(d)
    torch.cuda.synchronize()
    r = d["rows"]
    pick = lambda t, n: t[n] if n in ("dgw", "duw", "ddw", "drw") else t[n][r]  # noqa: E731
    want = {n: pick(d, n).clone() for n in names}
    other = dict(d)
    for n in (*names, "scratch"):
        other[n] = torch.zeros_like(d[n])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(d)
    torch.cuda.synchronize()
    for i in range(4):
        for n in names:
            d[n].fill_(0.0)
            other[n].fill_(0.0)
        step(other)                                    # eager work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(pick(d, n), want[n]), (i, n)
            assert torch.equal(pick(other, n), want[n]), (i, n)
    s2 = torch.cuda.Stream()
    for t in (d, other):
        for n in names:
            t[n].fill_(0.0)
    torch.cuda.synchronize()
    step(d, stream=side)                               # two calls at once, buffers of their own
    step(other, stream=s2)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(pick(d, n), want[n]) and torch.equal(pick(other, n), want[n]), n


def test_layer_step():
    """A training step of the whole routed layer as a program runs it: router,
    device contract, pack, training forward, combine; then the gradient of the
    output packed, the backward pass, and the tokens' gradient combined."""
    T, E, k, H, I = 45, 6, 2, 256, 384
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    x, dy, wr = rnd(T, H), rnd(T, H), rnd(E, H) / H ** 0.5
    wg, wu, wd = rnd(E, I, H) / H ** 0.5, rnd(E, I, H) / H ** 0.5, rnd(E, H, I) / I ** 0.5
    ids, vals = R.router(x, wr, k)
    t = R.build_contract_device(ids, E)
    Tp, pairs = t["total_padded_tokens"], t["pairs"]
    tables = (t["group_sizes"], t["group_offsets"], t["group_padded_offsets"], t["group_idx_for_bx"])
    z = lambda *s: torch.full(s, float("nan"), dtype=torch.float16, device="cuda")  # noqa: E731
    xs, dys, gate, up, hid, out = z(Tp, H), z(Tp, H), z(Tp, I), z(Tp, I), z(Tp, I), z(Tp, H)
    w, drw = torch.empty(pairs, device="cuda"), torch.empty(pairs, device="cuda")
    y, dx_t = z(T, H), z(T, H)
    R.pack(x, vals.reshape(-1), t["padded_row_of_pair"], t["compact_pos_of_pair"], xs, w)
    R.gate_up_train(xs, wg, wu, tables[0], tables[2], tables[3], gate, up, hid)
    R.down(hid, wd, w, *tables, out)
    R.combine(out, t["padded_row_of_pair"], k, y)
    R.pack(dy, vals.reshape(-1), t["padded_row_of_pair"], t["compact_pos_of_pair"], dys, w)
    dx, dgw, duw, ddw = z(Tp, H), z(E, I, H), z(E, I, H), z(E, H, I)
    scratch = torch.empty(R.backward_scratch_bytes(pairs, I), dtype=torch.uint8, device="cuda")
    R.backward(xs, dys, wg, wu, wd, w, gate, up, *tables, gate, up, hid, scratch, dx, dgw, duw, ddw, drw)
    R.combine(dx, t["padded_row_of_pair"], k, dx_t)
    torch.cuda.synchronize()
    # the same in 64 bits through autograd
    leaves = [a.double().requires_grad_() for a in (x, wg, wu, wd, vals)]
    X, WG, WU, WD, V = leaves
    ids64 = ids.long()
    tot = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = torch.nonzero(ids64 == e, as_tuple=True)
        tot = tot.index_add(0, tok, TR.forward(X[tok], WG[e], WU[e], WD[e], V[tok, slot]))
    (tot * dy.double()).sum().backward()
    # norms: roundings of the kept rows, the operands, the k slots and the result, 2^-11 each with factors up to 2
    close = lambda a, b: float((a.double() - b).norm()) <= 10 * 2.0 ** -11 * float(b.norm())  # noqa: E731
    assert close(y, tot.detach())
    for got, leaf in zip((dx_t, dgw, duw, ddw), leaves):
        assert close(got, leaf.grad)
    assert close(drw[t["compact_pos_of_pair"].long()].view(T, k), V.grad)

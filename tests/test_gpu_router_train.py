"""GPU tests of the training router against the 64-bit oracle
(oracle/router_train.py).

Inputs of the parity tests lie on a grid (tokens in steps of 2^-5, gate rows in
steps of 2^-10) on which every partial sum of a logit is exact in fp32: ids and
counts must be the oracle's.  With D the largest distance of a logit from its
row's maximum, u = 2^-24 and the hardware exp2, log2 and reciprocal good to 4 u:

  * a probability: the exponent's argument (2 D u relative), exp2, a sum of at
    most E / 4 + 2 additions, a reciprocal and a product: (2 D + E / 2 + 16) u;
  * lse: the sum's error and log2's, absolute, and its own rounding:
    (2 D + E / 2 + 32) u + 2 u |lse|;
  * the losses' sums run over at most 64 terms in fp32, then in 64 bits.

Backward: dl in fp32 from sums of E / 4 + k / 4 + 6 additions at most; its two
fp16 parts leave 2^-22 of the value and 2^-38 of the largest one that shares
its scale; an fp32 sum of K products carries K 2^-23 of the sum of their
magnitudes (2^-23 per addition allows for a truncating adder)."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import workloads
from oracle import router_train as RB

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(T, E, H, seed, left_out=0.0):
    """x, w on the grid; a mask (None: every token counts), with NaN and
    infinities in the rows that are left out."""
    rng = np.random.default_rng(seed)
    x = np.clip(np.round(rng.standard_normal((T, H)) * 32), -127, 127) / 32
    w = np.clip(np.round(rng.standard_normal((E, H)) * 1024 / H ** 0.5), -1023, 1023) / 1024
    mask = (rng.random(T) >= left_out).astype(np.uint8) if left_out else None
    bad = x.astype(np.float16)
    if mask is not None:
        bad[mask == 0] = np.where(rng.random((int((mask == 0).sum()), H)) < 0.5, np.nan, np.inf)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return x, w, mask, dev(bad), dev(w.astype(np.float16)), None if mask is None else dev(mask)


def _np(t):
    return t.cpu().numpy().astype(np.float64)


def _check_forward(got, x, w, k, mask):
    T, E = x.shape[0], w.shape[0]
    f = RB.forward(x, w, k, mask)
    assert np.array_equal(got["topk_ids"].cpu().numpy(), f["ids"])
    assert np.array_equal(got["counts"].cpu().numpy(), f["counts"])
    D = (f["logits"].max(1) - f["logits"].min(1))[:, None] if T else np.zeros((0, 1))
    rel = (2 * D + E / 2 + 16) * U
    assert (np.abs(_np(got["probs"]) - f["probs"]) <= f["probs"] * rel + 1e-37).all()
    assert (np.abs(_np(got["topk_weights"]) - f["vals"]) <= f["vals"] * rel + 1e-37).all()
    el = ((2 * D + E / 2 + 32) * U)[:, 0] + 2 * U * np.abs(f["lse"])
    assert (np.abs(_np(got["lse"]) - f["lse"]) <= el).all()
    n = max(1, int(f["counts"][E]))
    most = float(rel.max()) if T else 0.0
    l = _np(got["losses"])
    assert abs(l[0] - f["losses"][0]) <= f["losses"][0] * (most + 66 * U) + 1e-37
    ez = (2 * np.abs(f["lse"]) * el + el ** 2)[f["lse"] != 0].sum() / n + f["losses"][1] * 68 * U
    assert abs(l[1] - f["losses"][1]) <= ez
    return f


SIZES = [(1, 1, 1, 64, 0), (9, 4, 2, 256, 0), (9, 4, 2, 256, 0.4), (64, 8, 2, 4096, 0), (65, 7, 3, 512, 0.2),
         (1000, 64, 6, 2048, 0.1), (300, 128, 8, 7168, 0), (130, 256, 16, 1024, 0.3), (65, 32, 32, 64, 0),
         (63, 33, 32, 192, 0.5), (257, 96, 4, 320, 0.1), (200, 160, 5, 128, 0), (129, 192, 7, 448, 0.2),
         (70, 224, 8, 64, 0), (40001, 16, 2, 128, 0.3), (33000, 40, 3, 64, 0), (128, 3, 1, 8192, 0.9)]


@pytest.mark.parametrize("T,E,k,H,left_out", SIZES)
def test_forward(T, E, k, H, left_out):
    print(f"[router_train] T={T} E={E} k={k} H={H}", flush=True)
    x, w, mask, xg, wg, mg = _inputs(T, E, H, T + E, left_out)
    got = R.router_train(xg, wg, k, token_mask=mg)
    torch.cuda.synchronize()
    _check_forward(got, x, w, k, mask)
    if mask is None:                                  # the serving router's choice, bit for bit
        ids, vals = R.router(xg, wg, k)
        assert torch.equal(ids, got["topk_ids"]) and torch.equal(vals, got["topk_weights"])


@pytest.mark.parametrize("T,E,k,H", [(333, 64, 6, 1024), (40000, 8, 2, 64), (100, 130, 4, 192)])
def test_forward_is_the_serving_router_on_any_values(T, E, k, H):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = torch.randn((T, H), generator=g, device="cuda").half(), (torch.randn((E, H), generator=g, device="cuda") / 4).half()
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    got = R.router_train(x, w, k, token_mask=mask)
    ids, vals = R.router(x, w, k)
    torch.cuda.synchronize()
    assert torch.equal(got["topk_ids"], torch.where(mask[:, None], ids, -1))
    assert torch.equal(got["topk_weights"], torch.where(mask[:, None], vals, 0))
    n = torch.bincount(ids[mask].reshape(-1).long(), minlength=E)
    assert torch.equal(got["counts"].long(), torch.cat((n, mask.sum()[None])))
    again = R.router_train(x, w, k, token_mask=mask.to(torch.uint8), out={n: torch.empty_like(t) for n, t in got.items()})
    torch.cuda.synchronize()
    for n in ("topk_ids", "topk_weights", "probs", "lse", "counts", "losses"):
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("E,H", [(100, 448), (128, 64), (256, 1024), (64, 128)])
def test_serving_and_training_rows_do_not_depend_on_the_batch(E, H):
    """A token's ids and scores are the same bits whatever follows it, up to
    two workgroups of 64 tokens per compute unit: 64 tokens per workgroup from
    one on are two halves that sum as workgroups of 32 do."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    T = 128 * cus - 37
    g = torch.Generator(device="cuda").manual_seed(E)
    x, w = torch.randn((T, H), generator=g, device="cuda").half(), (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).half()
    ids, vals = R.router(x, w, 4)
    got = R.router_train(x, w, 4)
    for few in (1, 95, 64 * cus - 1):
        i, v = R.router(x[:few], w, 4)
        t = R.router_train(x[:few], w, 4)
        torch.cuda.synchronize()
        assert torch.equal(i, ids[:few]) and torch.equal(v, vals[:few])
        assert torch.equal(t["topk_ids"], i) and torch.equal(t["probs"], got["probs"][:few])
    assert torch.equal(got["topk_ids"], ids) and torch.equal(got["topk_weights"], vals)


def test_forward_of_nothing():
    """No tokens, and no token that counts."""
    w = torch.randn((8, 128), device="cuda").half()
    got = R.router_train(torch.empty((0, 128), dtype=torch.float16, device="cuda"), w, 2)
    torch.cuda.synchronize()
    assert not got["counts"].any() and not got["losses"].any() and got["topk_ids"].shape == (0, 2)
    x = torch.full((70, 128), float("nan"), device="cuda").half()
    mask = torch.zeros(70, dtype=torch.bool, device="cuda")
    got = R.router_train(x, w, 2, token_mask=mask)
    torch.cuda.synchronize()
    assert not got["counts"].any() and not got["losses"].any() and not got["probs"].any() and not got["lse"].any()
    assert (got["topk_ids"] == -1).all() and not got["topk_weights"].any()
    dx, dw = torch.full_like(x, 7), torch.full((8, 128), 7.0, device="cuda")
    scratch = torch.empty(R.router_backward_scratch_bytes(70, 128, 8), dtype=torch.uint8, device="cuda")
    R.router_backward(x, w, got["topk_ids"], got["probs"], got["lse"], got["counts"],
                      torch.full((140,), float("nan"), device="cuda"), torch.ones(2, device="cuda"), dx, dw, scratch,
                      token_mask=mask)
    torch.cuda.synchronize()
    assert not dx.any() and not dw.any()
    dw.fill_(7)
    none = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    R.router_backward(x[:0], w, none(0, 2, t=torch.int32), none(0, 8), none(0), got["counts"], none(0), None, x[:0], dw, scratch)
    torch.cuda.synchronize()
    assert not dw.any()


def test_a_token_with_nan_shows_itself_and_no_other():
    x, w, _, xg, wg, _ = _inputs(70, 8, 128, 3)
    xg[5, 3] = float("nan")
    got = R.router_train(xg, wg, 2)
    torch.cuda.synchronize()
    rest = [t for t in range(70) if t != 5]
    assert torch.isnan(got["probs"][5]).all() and torch.isnan(got["lse"][5]) and torch.isnan(got["losses"]).all()
    assert (got["topk_ids"][5] == 2 ** 31 - 1).all() and torch.isfinite(got["probs"][rest]).all()
    assert int(got["counts"][:8].sum()) == 2 * 69 and int(got["counts"][8]) == 70
    t = R.build_contract_device(got["topk_ids"], 8)
    assert int(t["bad_ids"]) == 2


# ---------------------------------------------------------------- backward
def _backward(f, xg, wg, mg, g, ab, add=None, compact=False, alias=False, seed=0):
    """Calls the library on the kept values f; returns (dx, dw)."""
    T, E = f["probs"].shape
    k, H = f["ids"].shape[1], xg.shape[1]
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    drw, cpos = f32(g).reshape(-1), None
    if compact:                                       # a random order, pairs of left-out tokens nowhere
        perm = np.random.default_rng(seed).permutation(T * k).astype(np.int32)
        buf = torch.full((T * k,), float("nan"), device="cuda")
        buf[torch.from_numpy(perm).long().cuda()] = drw
        dead = f["ids"].reshape(-1) < 0
        perm[dead] = -1
        drw, cpos = buf, i32(perm)
    dx = torch.full((T, H), float("nan"), device="cuda").half()
    if alias:
        dx.copy_(add)
        add = dx
    dw = torch.full((E, H), float("nan"), device="cuda")
    scratch = torch.full((R.router_backward_scratch_bytes(T, H, E),), 0xFF, dtype=torch.uint8, device="cuda")
    R.router_backward(xg, wg, i32(f["ids"]), f32(f["probs"]), f32(f["lse"]), i32(f["counts"]), drw,
                      None if ab is None else f32(ab), dx, dw, scratch, compact_pos_of_pair=cpos, token_mask=mg, dx_add=add)
    torch.cuda.synchronize()
    return dx, dw


def _check_backward(dx, dw, f, x, w, mask, g, ab, add=None):
    """x, w, f: what the library was given (f and g in the fp32 it took)."""
    f = {n: (v.astype(np.float32).astype(np.float64) if n in ("probs", "lse") else v) for n, v in f.items()}
    g = np.asarray(g, np.float32).astype(np.float64)
    T, E = f["probs"].shape
    k, n = f["ids"].shape[1], max(1, int(f["counts"][E]))
    on = np.ones(T, bool) if mask is None else mask.astype(bool)
    dl = RB.dlogits(f["probs"], f["lse"], f["ids"], f["counts"], np.where(on[:, None], g, 0), ab, mask)
    want_x, want_w = RB.backward(np.where(on[:, None], x, 0), w, dl)
    # dl's own error: its sums and products in fp32
    a, b = (0.0, 0.0) if ab is None else (abs(ab[0]), abs(ab[1]))
    ca = a * E * np.abs(f["counts"][:E]) / (k * n * n)
    cz = 2 * b * np.abs(f["lse"])[:, None] / n
    ag = np.where(on[:, None] & (f["ids"] >= 0), np.abs(g), 0).sum(1, keepdims=True)
    size = ca[None] + cz + ag + (f["probs"] * ca[None]).sum(1, keepdims=True) + ag
    edl = f["probs"] * size * (E / 4 + k / 4 + 16) * U
    # and that of its two fp16 parts
    blocks = np.pad(np.abs(dl), ((0, -T % 64), (0, 0))).reshape(-1, 64, E).max(1).repeat(64, 0)[:T]
    top = np.maximum(np.abs(dl).max(1, keepdims=True, initial=0), blocks)
    part = edl + np.abs(dl) * 2.0 ** -22 + top * 2.0 ** -38
    EP = -(-E // 32) * 32
    ax, aw = np.abs(np.where(on[:, None], x, 0)), np.abs(w)
    bx = part @ aw + 2 * EP * 2.0 ** -23 * (np.abs(dl) @ aw)
    if add is not None:
        want_x = want_x + add
    bx += (np.abs(want_x) + bx) * (2.0 ** -11 + U) + 2.0 ** -25
    assert (np.abs(_np(dx) - want_x) <= bx).all()
    nb = -(-T // 64)
    bw = part.T @ ax + (128 + nb + 300) * 2.0 ** -23 * (np.abs(dl).T @ ax)
    assert (np.abs(_np(dw) - want_w) <= bw + 1e-37).all()


@pytest.mark.parametrize("T,E,k,H,left_out", SIZES)
def test_backward(T, E, k, H, left_out):
    print(f"[router_backward] T={T} E={E} k={k} H={H}", flush=True)
    x, w, mask, xg, wg, mg = _inputs(T, E, H, T + E, left_out)
    f = RB.forward(x, w, k, mask)
    rng = np.random.default_rng(T)
    g, ab = rng.standard_normal((T, k)), (0.02 * T, -0.003 * T)
    add = torch.from_numpy(rng.standard_normal((T, H)) * 1e-2).half()
    dx, dw = _backward(f, xg, wg, mg, g, ab)
    _check_backward(dx, dw, f, x, w, mask, g, ab)
    # compact order and an added gradient, apart and in place
    dx2, dw2 = _backward(f, xg, wg, mg, g, ab, add=add.cuda(), compact=True)
    _check_backward(dx2, dw2, f, x, w, mask, g, ab, _np(add))
    assert torch.equal(dw, dw2)
    dx3, _ = _backward(f, xg, wg, mg, g, ab, add=add.cuda(), compact=True, alias=True)
    assert torch.equal(dx2, dx3)
    # the losses' gradients alone, the weights' alone
    dx, dw = _backward(f, xg, wg, mg, g, None)
    _check_backward(dx, dw, f, x, w, mask, g, None)
    dx, dw = _backward(f, xg, wg, mg, 0 * g, ab)
    _check_backward(dx, dw, f, x, w, mask, 0 * g, ab)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e-3, 1e12])
def test_backward_of_small_and_large_gradients(size):
    """Power-of-two scales carry gradients far outside fp16's range (dx itself
    is fp16)."""
    x, w, mask, xg, wg, mg = _inputs(130, 40, 256, 5, 0.2)
    f = RB.forward(x, w, 3, mask)
    g = np.random.default_rng(1).standard_normal((130, 3)) * size
    g[64:100] *= 1e-6
    dx, dw = _backward(f, xg, wg, mg, g, None)
    if size < 1:
        _check_backward(dx, dw, f, x, w, mask, g, None)
    else:
        assert torch.isfinite(dw).all()
        _check_backward(torch.zeros_like(dx), dw, f, x, 0 * w, mask, g, None)


def test_backward_of_ids_twice_and_out_of_range():
    x, w, _, xg, wg, _ = _inputs(67, 9, 128, 7)
    f = RB.forward(x, w, 4)
    f["ids"][3] = [2, 2, 2, 5]
    f["ids"][4] = [-1, 9, 2 ** 31 - 1, 0]
    f["ids"][66] = [8, 8, -5, -(2 ** 31)]
    g = np.random.default_rng(2).standard_normal((67, 4))
    dx, dw = _backward(f, xg, wg, None, g, (3.0, 1.0))
    _check_backward(dx, dw, f, x, w, None, g, (3.0, 1.0))


@pytest.mark.parametrize("E", [1, 40])
def test_backward_where_one_expert_has_all_the_probability(E):
    """p = 1: the routed weights' gradients cancel exactly, however large, and
    leave the z loss's, with the roundings of its own products only (a fp32
    constant, lse, p, n: 4; two fp16 parts 2^-22; the sums of dW)."""
    T, H = 130, 128
    x, w, _, xg, wg, _ = _inputs(T, E, H, 9)
    f = RB.forward(x, w, 1)
    f["ids"][:] = E - 1
    f["probs"][:] = 0
    f["probs"][:, E - 1] = 1
    g = np.random.default_rng(3).standard_normal((T, 1)) * 1e4
    dx, dw = _backward(f, xg, wg, None, g, (0.0, 0.01))
    dl = np.zeros((T, E))
    dl[:, E - 1] = 2 * 0.01 * f["lse"].astype(np.float32).astype(np.float64) / T
    top = np.abs(dl).max()
    size = np.abs(dl).T @ np.abs(x)
    assert (np.abs(_np(dw) - dl.T @ x) <= size * (6 * U + 2.0 ** -22 + 431 * 2.0 ** -23) + T * top * 2.0 ** -36).all()
    assert (np.abs(_np(dx) - dl @ w) <= (np.abs(dl) @ np.abs(w)) * (2.0 ** -10) + 2.0 ** -24).all()


def test_backward_counts_may_come_from_elsewhere():
    """Counts summed over several ranks: constants of the loss."""
    x, w, mask, xg, wg, mg = _inputs(90, 12, 192, 8, 0.1)
    f = RB.forward(x, w, 2, mask)
    f["counts"] = f["counts"] * 3 + 5
    g = np.random.default_rng(3).standard_normal((90, 2))
    dx, dw = _backward(f, xg, wg, mg, g, (9.0, 2.0))
    _check_backward(dx, dw, f, x, w, mask, g, (9.0, 2.0))


def test_backward_nan_stays_with_its_token():
    x, w, _, xg, wg, _ = _inputs(70, 8, 128, 3)
    f = RB.forward(x, w, 2)
    g = np.random.default_rng(4).standard_normal((70, 2))
    g[5, 1] = np.nan
    dx, dw = _backward(f, xg, wg, None, g, None)
    rest = [t for t in range(70) if t != 5]
    assert torch.isnan(dx[5]).all() and torch.isfinite(dx[rest]).all() and torch.isnan(dw).all()


def test_graph_replays_and_streams():
    """Forward and backward captured on a side stream and replayed between
    eager calls; two eager runs on streams of their own."""
    T, E, k, H = 500, 24, 3, 320
    _, _, _, xg, wg, mg = _inputs(T, E, H, 9, 0.2)
    drw, ab = torch.randn(T * k, device="cuda"), torch.tensor([4.0, 0.5], device="cuda")
    n = R.router_backward_scratch_bytes(T, H, E)

    def buffers():
        return (torch.zeros((T, H), dtype=torch.float16, device="cuda"), torch.zeros((E, H), device="cuda"),
                torch.empty(n, dtype=torch.uint8, device="cuda"))

    def step(out, bufs, stream=None):
        out = R.router_train(xg, wg, k, token_mask=mg, out=out, stream=stream)
        R.router_backward(xg, wg, out["topk_ids"], out["probs"], out["lse"], out["counts"], drw, ab, *bufs, token_mask=mg,
                          stream=stream)
        return out

    want, wb = step(None, buffers()), buffers()
    step(want, wb)
    torch.cuda.synchronize()
    names = ("topk_ids", "topk_weights", "probs", "lse", "counts", "losses")
    keep = {m: want[m].clone() for m in names}
    mine, mb = {m: torch.empty_like(t) for m, t in want.items()}, buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(mine, mb)
    torch.cuda.synchronize()
    for i in range(4):
        for t in (*mb[:2], mine["probs"], mine["losses"]):
            t.fill_(0)
        step(want, wb)                                # eager work between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(mine[m], keep[m]) and torch.equal(want[m], keep[m]) for m in names), i
        assert torch.equal(mb[0], wb[0]) and torch.equal(mb[1], wb[1]), i
    streams, outs, bufs = [torch.cuda.Stream() for _ in range(2)], [], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for s, b in zip(streams, bufs):
        outs.append(step(None, b, stream=s))
    torch.cuda.synchronize()
    for o, b in zip(outs, bufs):
        assert all(torch.equal(o[m], keep[m]) for m in names)
        assert torch.equal(b[0], wb[0]) and torch.equal(b[1], wb[1])


def test_binding_refusals():
    T, E, k, H = 20, 8, 2, 128
    _, _, _, xg, wg, mg = _inputs(T, E, H, 1, 0.2)
    out = R.router_train(xg, wg, k, token_mask=mg)
    for kw in (dict(x=xg.float()), dict(x=xg[:, ::2]), dict(x=xg.cpu()), dict(router_w=wg[:, :64]), dict(router_w=wg.float()),
               dict(token_mask=mg[:-1]), dict(token_mask=mg.int()), dict(token_mask=mg.cpu()),
               dict(out={n: t[:-1] for n, t in out.items()}), dict(out=dict(out, probs=out["probs"].double()))):
        with pytest.raises((TypeError, ValueError)):
            R.router_train(**{"x": xg, "router_w": wg, "top_k": k, **kw})
    with pytest.raises(R.RmoeError):
        R.router_train(xg, wg, 9)
    with pytest.raises(R.RmoeError):
        R.router_train(xg, wg, 0)
    good = dict(x=xg, router_w=wg, topk_ids=out["topk_ids"], probs=out["probs"], lse=out["lse"], counts=out["counts"],
                drw=torch.zeros(T * k, device="cuda"), dlosses=torch.zeros(2, device="cuda"),
                dx=torch.zeros((T, H), dtype=torch.float16, device="cuda"), drouter_w=torch.zeros((E, H), device="cuda"),
                scratch=torch.empty(R.router_backward_scratch_bytes(T, H, E), dtype=torch.uint8, device="cuda"),
                compact_pos_of_pair=torch.zeros(T * k, dtype=torch.int32, device="cuda"), token_mask=mg,
                dx_add=torch.zeros((T, H), dtype=torch.float16, device="cuda"))
    R.router_backward(**good)
    for name, t in good.items():
        for bad in (t.cpu(), t.double(), t[:-1], t.unsqueeze(0).expand(2, *t.shape)):
            if name == "scratch" and bad.dtype is torch.float64:
                continue                              # scratch is bytes of any type
            with pytest.raises((TypeError, ValueError, R.RmoeError)):
                R.router_backward(**{**good, name: bad})


def test_mask_types():
    T, E, k, H = 20, 8, 2, 128
    _, _, _, xg, wg, mg = _inputs(T, E, H, 2, 0.3)
    a, b = R.router_train(xg, wg, k, token_mask=mg), R.router_train(xg, wg, k, token_mask=mg.bool())
    assert all(torch.equal(a[n], b[n]) for n in ("topk_ids", "topk_weights", "probs", "lse", "counts", "losses"))
    with pytest.raises(TypeError):
        R.router_train(xg, wg, k, token_mask=mg.tolist())


def test_training_step_of_a_whole_layer():
    """Router, contract, pack, expert FFN, combine, and all of it backwards, as
    a program runs them, with padding tokens: the gradients of the tokens, the
    gate matrix and the expert matrices against 64-bit autograd through the
    same choice of experts."""
    T, E, k, H, I = 150, 8, 2, 256, 128
    x, w, mask, xg, wr, mg = _inputs(T, E, H, 4, 0.2)
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wg, wu, wd = (rnd(E, I, H) / H ** 0.5).half(), (rnd(E, I, H) / H ** 0.5).half(), (rnd(E, H, I) / I ** 0.5).half()
    dy, ab = rnd(T, H).half(), torch.tensor([30.0, 2.0], device="cuda")
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731

    r = R.router_train(xg, wr, k, token_mask=mg)
    t = R.build_contract_device(r["topk_ids"], E)
    Tp, pairs = t["total_padded_tokens"], T * k
    prow, cpos = t["padded_row_of_pair"], t["compact_pos_of_pair"]
    tables = (t["group_sizes"], t["group_offsets"], t["group_padded_offsets"], t["group_idx_for_bx"])
    xs, rw, dout = f16(Tp, H), torch.zeros(pairs, device="cuda"), f16(Tp, H)
    gate, up, hidden, out, y = f16(Tp, I), f16(Tp, I), f16(Tp, I), f16(Tp, H), f16(T, H)
    R.pack(xg, r["topk_weights"].view(-1), prow, cpos, xs, rw)
    R.gate_up_train(xs, wg, wu, t["group_sizes"], t["group_padded_offsets"], t["group_idx_for_bx"], gate, up, hidden)
    R.down(hidden, wd, rw, *tables, out)
    R.combine(out, prow, k, y)
    # backwards
    R.pack(dy, r["topk_weights"].view(-1), prow, cpos, dout, rw)
    dgate, dup, whidden, dxs = f16(Tp, I), f16(Tp, I), f16(Tp, I), f16(Tp, H)
    dwg, dwu, dwd, drw = torch.zeros_like(wg), torch.zeros_like(wu), torch.zeros_like(wd), torch.zeros(pairs, device="cuda")
    scratch = torch.empty(R.backward_scratch_bytes(pairs, I), dtype=torch.uint8, device="cuda")
    R.backward(xs, dout, wg, wu, wd, rw, gate, up, *tables, dgate, dup, whidden, scratch, dxs, dwg, dwu, dwd, drw)
    dx, dwr = f16(T, H), torch.zeros((E, H), device="cuda")
    R.combine(dxs, prow, k, dx)
    scratch2 = torch.empty(R.router_backward_scratch_bytes(T, H, E), dtype=torch.uint8, device="cuda")
    R.router_backward(xg, wr, r["topk_ids"], r["probs"], r["lse"], r["counts"], drw, ab, dx, dwr, scratch2,
                      compact_pos_of_pair=cpos, token_mask=mg, dx_add=dx)
    torch.cuda.synchronize()

    leaf = lambda a: a.double().cpu().requires_grad_()  # noqa: E731
    on = torch.from_numpy(mask > 0)
    x64, w64 = torch.from_numpy(x).requires_grad_(), leaf(wr)
    g64, u64, d64 = leaf(wg), leaf(wu), leaf(wd)
    logits = x64[on] @ w64.T
    p = torch.softmax(logits, 1)
    ids = r["topk_ids"].cpu().long()[on]
    total, parts = torch.zeros((int(on.sum()), H), dtype=torch.float64), []
    for e in range(E):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        xe = x64[on][tok]
        h = torch.nn.functional.silu(xe @ g64[e].T) * (xe @ u64[e].T)
        parts.append((tok, (h @ d64[e].T) * p[tok, e][:, None]))
    for tok, v in parts:
        total = total.index_add(0, tok, v)
    n = int(on.sum())
    counts = torch.bincount(ids.reshape(-1), minlength=E).double()
    balance = E / (k * n) * (counts * p.mean(0)).sum()
    z = (torch.logsumexp(logits, 1) ** 2).mean()
    loss = (total * dy.double().cpu()[on]).sum() + ab[0].double().cpu() * balance + ab[1].double().cpu() * z
    loss.backward()
    assert abs(float(r["losses"][0]) - float(balance.detach())) <= 1e-5 and abs(float(r["losses"][1]) - float(z.detach())) <= 1e-5
    assert not y[~on.cuda()].any() and not dx[~on.cuda()].any()
    # every step rounds its fp16 results once (2^-11 of a value) and adds up: the chain behind a gradient holds at most
    # seven of them (x, gate or up, hidden, out, dgate, dx of a row, dx of a token), and their squares add up
    far = lambda got, want: float((got.double().cpu() - want).norm() / want.norm())  # noqa: E731
    assert far(y[on.cuda()], total.detach()) <= 7 * 2.0 ** -11
    for got, want in ((dx[on.cuda()], x64.grad[on]), (dwr, w64.grad), (dwg, g64.grad), (dwu, u64.grad), (dwd, d64.grad)):
        assert far(got, want) <= 7 * 2.0 ** -11

"""GPU tests of the router, its training forward and its backward pass at its
fewest experts and at the token counts whose workgroups pass 2^32 threads in
one dimension of a grid (the host takes such a launch modulo 2^32: rows were
left unwritten and nothing was reported).

In the latter nearly all token rows are zero, so that every logit of theirs is
0: probability 1 / E each, the first expert, lse = ln E.  Rows with values
stand at the start, at the edge between two rows of the grid and at the end.

Tolerances, u = 2^-24: logits are whole multiples of 2^-15 below 2^9, exact in
fp32; with D a row's largest distance of a logit from its maximum a
probability is good to (2 D + E / 2 + 16) u of it, lse to (2 D + E / 2 + 32) u
+ 2 u |lse| (the exponent's argument, hardware exp2, log2 and reciprocal of 4 u,
the sums), the losses to 68 u and the probabilities' own error."""
import math

import pytest
import torch

import mixture_experts_routed_grouped_amd as R
from test_gpu_router_train import _check_forward, _inputs

pytestmark = pytest.mark.gpu
ROW = 1 << 21                     # workgroups in a row of the grid
U = 2.0 ** -24


def _room(nbytes):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < nbytes + (4 << 30):
        pytest.skip(f"needs {nbytes >> 30} GiB of GPU memory, {free >> 30} are free")


def _tokens(T, H, per_group):
    """x [T, H], and the tokens whose rows are not zero."""
    edge = ROW * per_group
    at = torch.cat((torch.arange(70), torch.arange(edge - 70, edge + 70), torch.arange(T - 200, T))).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((T, H), dtype=torch.float16, device="cuda")
    x[at] = (torch.randint(-127, 128, (at.numel(), H), generator=g, device="cuda") / 32).half()
    w = (torch.randint(-100, 101, (2, H), generator=g, device="cuda") / 1024).half()
    return x, w, at


def _differ(t, value, at):
    """Whether t equals value but for the rows at: looked at in pieces."""
    bad = []
    for i in range(0, t.shape[0], 1 << 26):
        rows = (t[i:i + (1 << 26)] != value).view(min(1 << 26, t.shape[0] - i), -1).any(1).nonzero()[:, 0] + i
        bad.append(rows)
    bad = torch.cat(bad)
    return bad[~torch.isin(bad, at)]


def test_forward_past_2_32_threads():
    T, H, E = (2 ** 32 // 320 + 4) * 64 + 5, 64, 2
    _room(T * (2 * H + 4 * 8))
    print(f"[router sizes] T={T}", flush=True)
    x, w, at = _tokens(T, H, 64)
    logits = x[at].double() @ w.double().T          # exact in fp32 in any order
    p = torch.softmax(logits, 1)
    first = (logits[:, 1] > logits[:, 0]).int()
    D = (logits[:, :1] - logits[:, 1:]).abs()
    rel, want_lse = (2 * D + 17) * U, torch.logsumexp(logits, 1)
    ids, vals = torch.full((T, 1), -7, dtype=torch.int32, device="cuda"), torch.full((T, 1), -7.0, device="cuda")
    R.router(x, w, 1, topk_ids=ids, topk_weights=vals)
    torch.cuda.synchronize()
    assert _differ(ids, 0, at).numel() == 0 and _differ(vals, 0.5, at).numel() == 0
    assert torch.equal(ids[at, 0], first)
    assert ((vals[at].double() - p.max(1, keepdim=True).values).abs() <= rel).all()
    print("[router sizes] training", flush=True)
    got = R.router_train(x, w, 1)
    torch.cuda.synchronize()
    assert torch.equal(got["topk_ids"], ids) and torch.equal(got["topk_weights"], vals)
    assert _differ(got["probs"], 0.5, at).numel() == 0
    assert ((got["probs"][at].double() - p).abs() <= rel * p).all()
    lse = got["lse"]
    assert _differ((lse - math.log(2)).abs() <= 35 * U, True, at).numel() == 0
    assert ((lse[at].double() - want_lse).abs() <= (2 * D[:, 0] + 33) * U + 2 * U * want_lse.abs()).all()
    ones = int(first.sum())
    assert got["counts"].tolist() == [T - ones, ones, T]
    rest = T - at.numel()
    sum_p = p.sum(0).cpu() + rest / 2
    balance = 2 / T * float((sum_p[0] * (T - ones) + sum_p[1] * ones) / T)
    z = (rest * math.log(2) ** 2 + float((want_lse ** 2).sum())) / T
    assert abs(float(got["losses"][0]) - balance) <= 1e-5 and abs(float(got["losses"][1]) - z) <= 1e-5


def test_backward_past_2_32_threads():
    T, H, E = 2 ** 28 + 64 * 3 + 5, 64, 2
    need = R.router_backward_scratch_bytes(T, H, E)
    _room(T * (4 * H + 8 + 16) + need)
    print(f"[router backward sizes] T={T}", flush=True)
    x, w, at = _tokens(T, H, 64)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    probs, lse = torch.full((T, E), 0.5, device="cuda"), torch.full((T,), 0.75, device="cuda")
    counts = torch.tensor([T, 0, T], dtype=torch.int32, device="cuda")
    drw = torch.zeros(T, device="cuda")
    drw[at] = torch.linspace(-1, 1, at.numel(), device="cuda")
    dlosses = torch.tensor([0.0, float(2 ** 28)], device="cuda")
    dx, dw = torch.full((T, H), 7, dtype=torch.float16, device="cuda"), torch.full((E, H), 7.0, device="cuda")
    R.router_backward(x, w, ids, probs, lse, counts, drw, dlosses, dx, dw,
                      torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    dl = 2 * float(dlosses[1]) * 0.75 * probs[at].double() / T
    dl[:, 0] += 0.25 * drw[at].double()
    dl[:, 1] -= 0.25 * drw[at].double()
    # fp32 sums of 2 x 32 products (2^-17 of their magnitudes), dl's own 20 roundings of terms up to 2.5 times it, its two
    # fp16 parts; then one rounding to fp16
    def near(got, dl):
        want, size = dl @ w.double(), dl.abs() @ w.double().abs()
        return ((got.double() - want).abs() <= want.abs() * 2.0 ** -10 + size * 2.0 ** -16 + 2.0 ** -24).all()
    assert near(dx[at], dl)
    plain = dx[100]                                  # of a row that carries the z loss's gradient alone
    assert near(plain, torch.full((2,), float(dlosses[1]) * 0.75 / T, dtype=torch.float64, device="cuda"))
    assert _differ(dx, plain, at).numel() == 0
    # only the rows with values add to the gate matrix's gradient: at most 128 + 300 + 410 additions
    want, size = dl.T @ x[at].double(), dl.abs().T @ x[at].double().abs()
    assert ((dw.double() - want).abs() <= size * 2.0 ** -13).all()


@pytest.mark.parametrize("H", [64, 576])
@pytest.mark.parametrize("E", [1, 2, 5, 8, 9])
@pytest.mark.parametrize("T", [77, 40003])
def test_forward_of_few_experts(T, E, H):
    """Up to 8 experts the lanes hold two scores each; every expert chosen."""
    x, w, mask, xg, wg, mg = _inputs(T, E, H, T + E, 0.1)
    got = R.router_train(xg, wg, E, token_mask=mg)
    torch.cuda.synchronize()
    _check_forward(got, x, w, E, mask)
    x, w, _, xg, wg, _ = _inputs(T, E, H, T + E)
    got = R.router_train(xg, wg, E)
    ids, vals = R.router(xg, wg, E)
    torch.cuda.synchronize()
    _check_forward(got, x, w, E, None)
    assert torch.equal(ids, got["topk_ids"]) and torch.equal(vals, got["topk_weights"])

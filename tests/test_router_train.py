"""The training router without a GPU: the oracle's gradients against
differences of its own losses, the library's sizes, and every refusal of the
entry points (checked before any HIP call)."""
import ctypes

import numpy as np
import pytest

import mixture_experts_routed_grouped_amd as R
from oracle import router_train as RB

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
P = ctypes.c_void_p


def test_oracle_balance_of_equal_and_of_one_sided_routers():
    x = np.zeros((8, 4))
    f = RB.forward(x, np.zeros((4, 4)), 2)               # equal logits: the first two experts
    assert f["ids"].tolist() == [[0, 1]] * 8 and f["counts"].tolist() == [8, 8, 0, 0, 8]
    assert np.allclose(f["losses"], [1.0, np.log(4) ** 2])
    w = np.zeros((4, 4))
    w[2] = 50
    f = RB.forward(np.ones((8, 4)), w, 1)                # all mass and all pairs on one expert
    assert f["counts"].tolist() == [0, 0, 8, 0, 8] and np.isclose(f["losses"][0], 4.0)


def test_oracle_left_out_tokens():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((9, 8)), rng.standard_normal((5, 8))
    mask = np.array([1, 0, 1, 1, 0, 1, 1, 1, 0])
    full, part = RB.forward(x[mask > 0], w, 3), RB.forward(np.where(mask[:, None], x, np.nan), w, 3, mask)
    assert (part["ids"][mask == 0] == -1).all() and np.array_equal(part["ids"][mask > 0], full["ids"])
    assert np.array_equal(part["counts"], full["counts"]) and np.allclose(part["losses"], full["losses"])
    none = RB.forward(x, w, 3, np.zeros(9))
    assert not none["counts"].any() and not none["losses"].any()


@pytest.mark.parametrize("T,E,k,H", [(6, 5, 2, 7), (4, 1, 1, 3), (3, 4, 4, 5)])
def test_oracle_gradients_against_differences(T, E, k, H):
    rng = np.random.default_rng(T + E)
    x, w = rng.standard_normal((T, H)), rng.standard_normal((E, H))
    mask = np.ones(T)
    mask[1] = 0
    g, ab = rng.standard_normal((T, k)), (0.7, -0.3)
    f = RB.forward(x, w, k, mask)

    def loss(x, w):
        """The routed weights of the choice made, and the two losses with their counts as they are."""
        on = mask > 0
        z = x @ w.T
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        lse = np.log(np.exp(z).sum(1))
        n = on.sum()
        chosen = (g[on] * np.take_along_axis(p[on], f["ids"][on], 1)).sum()
        return chosen + ab[0] * E / (k * n) * (f["counts"][:E] * p[on].mean(0)).sum() + ab[1] * (lse[on] ** 2).mean()

    dx, dw = RB.backward(x, w, RB.dlogits(f["probs"], f["lse"], f["ids"], f["counts"], g, ab, mask), mask)
    h = 1e-5
    for arr, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss(x, w)
            arr[i] = keep - h
            down = loss(x, w)
            arr[i] = keep
            # h^2 / 6 times a third derivative of order one, and rounding / h
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-8


# ---------------------------------------------------------------- refusals
A16, ODD8, ODD2 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 2)
SIZES = [dict(T=-1), dict(H=0), dict(H=-64), dict(E=0), dict(k=0), dict(k=-1), dict(E=4, k=5)]
SHAPES = [dict(E=257), dict(E=64, k=33), dict(H=96), dict(H=(1 << 20) + 64), dict(T=1 << 31), dict(T=(1 << 31) // 2)]


def test_forward_refusals():
    f = R.lib().rmoe_router_train_f16
    names = ["ids", "vals", "probs", "lse", "counts", "losses", "scratch"]

    def call(x=A16, w=A16, mask=None, T=4, H=128, E=8, k=2, **ptr):
        return f(x, w, mask, T, H, E, k, *[ptr.get(n, A16) for n in names], None)

    for bad in SIZES:
        assert call(**bad) == INVALID, bad
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    for n in ["x", "w"] + names:
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD8 if n in ("x", "w") else ODD2}) == MISALIGNED, n


def test_backward_refusals():
    f = R.lib().rmoe_router_backward_f16
    names = ["x", "w", "mask", "ids", "probs", "lse", "counts", "drw", "cpos", "dlosses", "add", "dx", "dw", "scratch"]

    def call(T=4, H=128, E=8, k=2, **ptr):
        return f(*[ptr.get(n, A16) for n in names], T, H, E, k, None)

    for bad in SIZES:
        assert call(**bad) == INVALID, bad
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    for n in names:
        if n == "mask":
            continue
        if n not in ("cpos", "dlosses", "add"):
            assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD8 if n in ("x", "w", "add", "dx", "dw", "scratch") else ODD2}) == MISALIGNED, n


def test_scratch_bytes():
    f, b = R.lib().rmoe_router_train_scratch_bytes, R.router_backward_scratch_bytes
    assert f(0, 8) == 0 and f(-1, 8) == 0 and f(5, 0) == 0 and f(5, 257) == 0
    assert f(33, 8) == 2 * 18 * 4
    for bad in ((-1, 128, 8), (4, 100, 8), (4, 0, 8), (4, 128, 0), (4, 128, 257)):
        assert b(*bad) == 0
    last = 0
    for T in (1, 63, 64, 65, 1000, 100000):
        assert b(T, 128, 8) >= max(last, 256) and b(T, 128, 8) % 256 == 0
        last = b(T, 128, 8)
    # two copies of dl as two fp16 values for 64-token blocks of 32-expert tiles, and more
    assert b(16384, 7168, 128) > 2 * 16384 * 128 * 4


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        R.router_train(torch.zeros(4, 128, dtype=torch.float16), torch.zeros(8, 128, dtype=torch.float16), 2)

"""The training entry points without a GPU: the gradient oracle against
autograd and against differences, the scratch size and every refusal (checked
before any HIP call)."""
import ctypes

import pytest
import torch

import mixture_experts_routed_grouped_amd as R
from oracle import train as TR

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
P = ctypes.c_void_p
A16, ODD8, ODD2 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 2)


def _inputs(n=5, H=12, I=7, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(n, H), r(n, H), r(I, H), r(I, H), r(H, I), torch.rand(n, generator=g, dtype=torch.float64)


def test_oracle_against_autograd():
    x, dy, wg, wu, wd, w = _inputs()
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, w)]
    (TR.forward(*leaves) * dy).sum().backward()
    for got, leaf in zip(TR.backward(x, dy, wg, wu, wd, w), leaves):
        assert torch.allclose(got, leaf.grad, rtol=1e-12, atol=1e-12)


def test_oracle_against_differences():
    x, dy, wg, wu, wd, w = _inputs(seed=1)
    base = [x, wg, wu, wd, w]
    grads = TR.backward(x, dy, wg, wu, wd, w)
    eps = 1e-5
    for i in range(5):
        v = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - eps * v, base[i] + eps * v
        d = ((TR.forward(*hi) - TR.forward(*lo)) * dy).sum() / (2 * eps)
        # central differences: third derivatives times eps^2, and 2^-52 / eps of the sums
        assert abs(d - (grads[i] * v).sum()) <= 1e-7 * (1 + (grads[i] * v).abs().sum())


def test_scratch_bytes():
    assert R.backward_scratch_bytes(10, 128) == 40
    assert R.backward_scratch_bytes(10, 1408) == 10 * 11 * 4
    assert R.backward_scratch_bytes(0, 128) == 0 and R.backward_scratch_bytes(3, 0) == 0
    assert R.backward_scratch_bytes(-1, 128) == 0


CALLS = {
    "rmoe_gate_up_train_f16": "x gw uw gs gpo gidx gate up hidden",
    "rmoe_backward_f16": "x dout gw uw dw rw gate up gs go gpo gidx dgate dup whidden scratch dx dgw duw ddw drw",
    "rmoe_down_backward_f16": "dout dw rw gate up gs go gpo gidx dgate dup whidden scratch drw",
    "rmoe_gate_up_backward_f16": "dgate dup gw uw gs gpo gidx dx",
    "rmoe_weight_grad_f16": "x dout dgate dup whidden gs gpo dgw duw ddw",
}
WORDS = {"gs", "go", "gpo", "gidx", "rw", "drw", "scratch"}   # 4-byte aligned


@pytest.mark.parametrize("fn", list(CALLS))
def test_refusals(fn):
    f, names = getattr(R.lib(), fn), CALLS[fn].split()
    grad = fn == "rmoe_weight_grad_f16"

    def call(H=256, I=384, E=2, Tp=512, pairs=5, M=3, **ptr):
        args = [ptr.get(n, A16) for n in names]
        return f(*args, H, I, E, Tp, None) if grad else f(*args, H, I, E, Tp, pairs, M, None)

    for bad in (dict(H=0), dict(I=-128), dict(E=0), dict(Tp=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=192), dict(I=100), dict(H=(1 << 20) + 128), dict(I=(1 << 20) + 128)):
        assert call(**bad) == SHAPE, bad
    if not grad:
        for bad in (dict(pairs=-1), dict(M=-1), dict(Tp=383)):
            assert call(**bad) == INVALID, bad
        assert call(M=65536, Tp=65536 * 128) == SHAPE
    if fn in ("rmoe_backward_f16", "rmoe_weight_grad_f16"):    # 3 * 4096 * 4096 tiles
        assert call(H=1 << 20, I=1 << 20) == SHAPE
    for n in names:
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD2 if n in WORDS else ODD8}) == MISALIGNED, n


def test_nothing_to_do():
    """No block: nothing is launched (the weight gradients alone write zeros
    for every expert, so they have no such call)."""
    L = R.lib()
    assert L.rmoe_gate_up_train_f16(*[A16] * 9, 256, 384, 2, 512, 0, 0, None) == OK
    assert L.rmoe_down_backward_f16(*[A16] * 14, 256, 384, 2, 512, 0, 0, None) == OK
    assert L.rmoe_gate_up_backward_f16(*[A16] * 8, 256, 384, 2, 512, 0, 0, None) == OK


def test_binding_refuses_cpu_tensors():
    z = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        R.gate_up_train(z(256, 128), z(2, 128, 128), z(2, 128, 128), i(2), i(3), i(2), z(256, 128), z(256, 128),
                        z(256, 128))
    with pytest.raises(ValueError):
        R.gate_up_backward(z(256, 128), z(256, 128), z(2, 128, 128), z(2, 128, 128), i(2), i(3), i(2), z(256, 128))
    with pytest.raises(ValueError):
        R.weight_grad(z(256, 128), z(256, 128), z(256, 128), z(256, 128), z(256, 128), i(2), i(3), z(2, 128, 128),
                      z(2, 128, 128), z(2, 128, 128))
    with pytest.raises(TypeError):
        R.gate_up_train(None, z(2, 128, 128), z(2, 128, 128), i(2), i(3), i(2), z(256, 128), z(256, 128), z(256, 128))

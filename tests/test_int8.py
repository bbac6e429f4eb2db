"""8-bit integer rows without a GPU: the oracle against hand-worked rows, the
library's sizes, and every refusal of the entry points (checked before any HIP
call, so bad sizes never reach a kernel)."""
import ctypes

import numpy as np
import pytest

import mixture_experts_routed_grouped_amd as R
from oracle import int8 as Q

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
P = ctypes.c_void_p


# ------------------------------------------------------------------ oracle
def test_oracle_handworked_rows():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -126.5, 126.5, 3.4999, 3.5001],      # scale 1: ties to even
                  [0.0] * 8,
                  [254.0, 1.0, -1.0, 3.0, -3.0, 253.0, -253.0, 2.0],           # scale 2
                  [1.0, np.inf, 0, 0, 0, 0, 0, 0], [1.0, np.nan, 0, 0, 0, 0, 0, 0]])
    codes, scales = Q.quantize(x)
    assert scales[:3].tolist() == [1.0, 0.0, 2.0] and np.isnan(scales[3:]).all()
    assert codes[0].tolist() == [127, 0, 2, -2, -126, 126, 3, 4]
    assert codes[1].tolist() == [0] * 8
    assert codes[2].tolist() == [127, 0, 0, 2, -2, 126, -126, 1]
    assert not codes[3:].any()
    assert Q.values(codes, scales)[2].tolist() == [254, 0, 0, 4, -4, 252, -252, 2]


def test_oracle_rows_below_the_normal_numbers():
    tiny = 2.0 ** -149
    codes, scales = Q.quantize(np.array([[127 * tiny, tiny, -tiny, 0], [60 * tiny, tiny, 0, 0], [200 * tiny, 3 * tiny, 0, 0]]))
    assert scales.tolist() == [tiny, 0.0, 2 * tiny]
    assert codes[0].tolist() == [127, 1, -1, 0] and not codes[1].any() and codes[2].tolist() == [100, 2, 0, 0]


def test_rounding_by_a_fused_add_and_the_remainder():
    """The kernels' rounding in fp32, step by step in numpy: x inv rounded by
    adding 1.5 2^23, and where it lies near a border the sign of x - n s minus
    half of s, against the oracle on values next to every border."""
    rng = np.random.default_rng(0)
    f = np.float32
    for s in rng.uniform(1, 2, 40).astype(f):
        n = np.arange(-127, 127)
        mid = ((n + 0.5) * float(s)).astype(f)
        x = np.concatenate([mid, np.nextafter(mid, f(np.inf)), np.nextafter(mid, f(-np.inf)), rng.uniform(-127, 127, 999).astype(f) * s])
        x = np.concatenate([x, [f(127) * s]]).astype(f)
        top = f(np.abs(x).max())
        s2 = f(top / f(127))
        inv = f(f(1) / s2)
        r = (x.astype(np.float64) * float(inv)).astype(f)          # rounded once, as a product is
        t = (x.astype(np.float64) * float(inv) + 12582912.0).astype(f)
        q = t - f(12582912.0)
        near = np.abs(r - q) > f(0.4999)
        e = x.astype(np.float64) - q.astype(np.float64) * float(s2)
        assert (e[near] == e[near].astype(f)).all()                # the remainder is exact in 32 bits there
        odd = q.astype(int) % 2 != 0
        h = float(s2) / 2
        fixed = q + (near & ((e > h) | ((e == h) & odd))) - (near & ((e < -h) | ((e == -h) & odd)))
        want, scale = Q.quantize(x[None].astype(np.float64))
        assert scale[0] == s2 and fixed.astype(int).tolist() == want[0].tolist()


def test_workspace_bytes():
    assert R.int8_workspace_bytes(256, 384) == 256 * (384 * 5 + 4)
    for tp, i in ((0, 128), (-1, 128), (128, 0), (128, -128)):
        assert R.int8_workspace_bytes(tp, i) == 0


# ---------------------------------------------------------------- refusals
A16, ODD8, ODD2 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 2)


@pytest.mark.parametrize("fn", ["rmoe_quantize_int8", "rmoe_dequantize_int8"])
def test_quantize_refusals(fn):
    f = getattr(R.lib(), fn)

    def call(x=A16, codes=A16, scales=A16, ty=0, rows=4, cols=256):
        if fn == "rmoe_quantize_int8":
            return f(x, ty, rows, cols, codes, scales, None)
        return f(codes, scales, ty, rows, cols, x, None)

    assert call(rows=0) == OK and call(rows=0, x=None, codes=None, scales=None) == OK
    assert call(ty=3) == INVALID and call(ty=-1) == INVALID
    assert call(rows=-1) == INVALID and call(cols=0) == INVALID and call(cols=-8) == INVALID
    assert call(cols=12) == SHAPE and call(cols=1) == SHAPE
    assert call(rows=1 << 40, cols=1 << 40) == SHAPE and call(rows=1 << 57, cols=8) == SHAPE
    for cols in ((1 << 63) - 8, 1 << 62):
        assert call(cols=cols, rows=1) == SHAPE and call(cols=cols, rows=4) == SHAPE
    assert call(x=None) == INVALID and call(codes=None) == INVALID and call(scales=None) == INVALID
    assert call(x=ODD8) == MISALIGNED and call(codes=ODD8) == MISALIGNED and call(scales=ODD2) == MISALIGNED


def test_pack_refusals():
    f = R.lib().rmoe_pack_int8_f16

    def call(x=A16, w=A16, prow=A16, cpos=A16, T=4, k=2, H=256, codes=A16, scales=A16, wc=A16, Tp=512):
        return f(x, w, prow, cpos, T, k, H, codes, scales, wc, Tp, None)

    assert call(T=0) == OK and call(k=0) == OK
    assert call(T=-1) == INVALID and call(k=-1) == INVALID and call(Tp=-1) == INVALID and call(H=0) == INVALID
    assert call(H=260) == SHAPE and call(T=1 << 31) == SHAPE and call(H=(1 << 63) - 8) == SHAPE
    for name in ("x", "w", "prow", "cpos", "codes", "scales", "wc"):
        assert call(**{name: None}) == INVALID, name
    for name in ("x", "codes"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    for name in ("w", "prow", "cpos", "wc", "scales"):
        assert call(**{name: ODD2}) == MISALIGNED, name


GU = ["xc", "xs", "gc", "gsc", "uc", "us", "gs", "gpo", "gidx", "rows", "hc", "hs"]
DN = ["hc", "hs", "dc", "ds", "rw", "gs", "go", "gpo", "gidx", "out"]
FW = ["xc", "xs", "gc", "gsc", "uc", "us", "dc", "ds", "rw", "gs", "go", "gpo", "gidx", "ws", "out"]
FOUR = {"gs", "go", "gpo", "gidx", "rw", "xs", "hs"}      # aligned to 4 bytes, the others to 16


@pytest.mark.parametrize("fn,names", [("rmoe_gate_up_int8", GU), ("rmoe_down_int8", DN), ("rmoe_forward_int8", FW)])
def test_product_refusals(fn, names):
    f = getattr(R.lib(), fn)

    def call(H=256, I=384, E=2, Tp=512, pairs=5, M=3, variant=0, **ptr):
        return f(*[ptr.get(n, A16) for n in names], H, I, E, Tp, pairs, M, variant, None)

    assert call(M=0) == OK and call(M=0, Tp=513) == OK        # no block, nothing launched
    for bad in (dict(H=0), dict(I=-128), dict(E=0), dict(Tp=-1), dict(pairs=-1), dict(M=-1), dict(variant=3),
                dict(variant=-1), dict(Tp=383)):
        assert call(**bad) == INVALID, bad
    # the largest sums of products of codes: 127^2 133120 < 2^31 <= 127^2 133248
    for bad in (dict(H=192), dict(I=100), dict(H=133248), dict(I=133248), dict(M=65536, Tp=65536 * 128)):
        assert call(**bad) == SHAPE, bad
    assert call(M=0, H=133120, I=133120) == OK
    for n in names:
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD2 if n in FOUR else ODD8}) == MISALIGNED, n


def test_pick_variant():
    assert R.pick_variant_int8(0, 1) == "stream"
    assert R.pick_variant_int8(1 << 20, 8) == "tile"
    assert R.pick_variant_int8(5, 8, "tile") == "tile"
    f = R.lib().rmoe_pick_variant_int8
    assert f(0, -1, 1) == INVALID and f(0, 1, 0) == INVALID and f(3, 1, 1) == INVALID


def test_binding_refuses_cpu_tensors_and_types():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        R.quantize_int8(torch.zeros(4, 256, dtype=torch.float16))
    with pytest.raises(ValueError):
        R.dequantize_int8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError):
        R.dequantize_int8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4), dtype=torch.float64)

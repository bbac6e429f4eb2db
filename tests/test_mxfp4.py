"""MXFP4 without a GPU: the oracle against hand-worked blocks, the library's
sizes, and every refusal of the MXFP4 entry points (checked before any HIP
call, so bad pages and sizes never reach a kernel)."""
import ctypes
import math

import numpy as np
import pytest

import mixture_experts_routed_grouped_amd as R
from oracle import mxfp4 as MX

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
P = ctypes.c_void_p


# ------------------------------------------------------------------ oracle
def test_oracle_every_tie_goes_to_the_even_code():
    #            tie:   0.25 0.75 1.25 1.75 2.5 3.5 5    neighbours -> even code
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert MX.nearest_code(ties).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert MX.nearest_code(np.nextafter(ties, 9)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert MX.nearest_code(np.nextafter(ties, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert MX.nearest_code(np.array([6.0, 7.0, 7.99])).tolist() == [7, 7, 7]


def test_oracle_handworked_row():
    x = np.zeros((1, 40))
    x[0, :4] = [8.0, -3.0, 0.4, 15.9]          # amax 15.9: scale 2^(3-2) = 2
    x[0, 32:35] = [2.0 ** -126, -2.0 ** -127, 2.0 ** -128]
    codes, exps = MX.quantize(x)
    assert exps[0, :3].tolist() == [1, -127, -127]
    # 4 -> 4 (code 6), -1.5 -> code 3 with sign, 0.2 -> 0, 7.95 -> 6 (code 7)
    assert codes[0, :4].tolist() == [6, 3 | 8, 0, 7]
    # units of 2^-127: 2, -1, 0.5
    assert codes[0, 32:35].tolist() == [4, 2 | 8, 1]
    cb, sb = MX.stored(codes, exps)
    assert cb.shape == (1, 128) and sb.shape == (1, 1, 8)
    assert cb[0, :2].tolist() == [6 | (11 << 4), 0 | (7 << 4)]
    assert sb[0, 0].tolist() == [128, 0, 0, 0, 0, 0, 0, 0]
    v = MX.values(cb, sb, 40)
    assert v[0, :4].tolist() == [8.0, -3.0, 0.0, 12.0]
    assert v[0, 32] == 2.0 ** -126


def test_oracle_scale_byte_order():
    x = np.zeros((2, 512))
    for b in range(16):
        x[1, 32 * b] = 2.0 ** b
    _, sb = MX.stored(*MX.quantize(x))
    assert sb.shape == (2, 2, 8)
    assert (sb[0, 1].astype(int) - 125).tolist() == [0, 2, 4, 6, 1, 3, 5, 7]
    assert (sb[1, 1].astype(int) - 125).tolist() == [8, 10, 12, 14, 9, 11, 13, 15]


# ------------------------------------------------------------------- sizes
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 256), (5, 264), (128, 4096), (7, 1408)])
def test_sizes(rows, cols):
    ch = math.ceil(cols / 256)
    L = R.lib()
    assert L.rmoe_mxfp4_chunks(cols) == ch
    assert R.mxfp4_row_bytes(cols) == 128 * ch
    assert L.rmoe_mxfp4_code_bytes(rows, cols) == rows * 128 * ch
    assert L.rmoe_mxfp4_scale_bytes(rows, cols) == rows * 8 * ch
    assert R.mxfp4_workspace_bytes(rows, cols) == rows * 136 * ch
    assert R.mxfp4_shapes((rows, cols)) == ((rows, 128 * ch), (ch, rows, 8))
    assert R.mxfp4_shapes((2, rows, cols)) == ((2, rows, 128 * ch), (2, ch, rows, 8))


def test_sizes_of_nothing():
    L = R.lib()
    for rows, cols in ((0, 256), (-1, 256), (4, 0), (4, -8)):
        assert L.rmoe_mxfp4_code_bytes(rows, cols) == 0
        assert L.rmoe_mxfp4_scale_bytes(rows, cols) == 0
    assert L.rmoe_mxfp4_row_bytes(0) == 0 and L.rmoe_mxfp4_chunks(-1) == 0
    with pytest.raises(ValueError):
        R.mxfp4_shapes((4,))


# ---------------------------------------------------------------- refusals
A16, ODD8, ODD4, ODD2 = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 4), P((1 << 20) + 2)


@pytest.mark.parametrize("fn", ["rmoe_quantize_mxfp4", "rmoe_dequantize_mxfp4"])
def test_quantize_refusals(fn):
    f = getattr(R.lib(), fn)

    def call(x=A16, codes=A16, scales=A16, ty=0, batch=1, rows=4, cols=256):
        if fn == "rmoe_quantize_mxfp4":
            return f(x, ty, batch, rows, cols, codes, scales, None)
        return f(codes, scales, ty, batch, rows, cols, x, None)

    assert call(rows=0) == OK and call(batch=0) == OK       # nothing to do, nothing launched
    assert call(rows=0, x=None, codes=None, scales=None) == OK
    assert call(ty=3) == INVALID and call(ty=-1) == INVALID
    assert call(rows=-1) == INVALID and call(batch=-1) == INVALID
    assert call(cols=0) == INVALID and call(cols=-256) == INVALID
    assert call(cols=12) == SHAPE and call(cols=1) == SHAPE
    assert call(rows=1 << 31, cols=8) == SHAPE               # 2^31 chunks
    assert call(batch=1 << 40, rows=1 << 40) == SHAPE        # the count itself overflows
    assert call(x=None) == INVALID and call(codes=None) == INVALID and call(scales=None) == INVALID
    assert call(x=ODD8) == MISALIGNED and call(codes=ODD8) == MISALIGNED
    assert call(scales=ODD4) == MISALIGNED


def test_pack_refusals():
    f = R.lib().rmoe_pack_mxfp4_f16

    def call(x=A16, w=A16, prow=A16, cpos=A16, T=4, k=2, H=256, codes=A16, scales=A16, wc=A16, Tp=512):
        return f(x, w, prow, cpos, T, k, H, codes, scales, wc, Tp, None)

    assert call(T=0) == OK and call(k=0) == OK
    assert call(T=-1) == INVALID and call(k=-1) == INVALID and call(Tp=-1) == INVALID and call(H=0) == INVALID
    assert call(H=260) == SHAPE and call(T=1 << 31) == SHAPE
    for name in ("x", "w", "prow", "cpos", "codes", "scales", "wc"):
        assert call(**{name: None}) == INVALID, name
    for name in ("x", "codes"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    assert call(scales=ODD4) == MISALIGNED
    for name in ("w", "prow", "cpos", "wc"):
        assert call(**{name: ODD2}) == MISALIGNED, name


GU = ["xc", "xs", "gc", "gsc", "uc", "us", "gs", "gpo", "gidx", "hc", "hs"]
DN = ["hc", "hs", "dc", "ds", "rw", "gs", "go", "gpo", "gidx", "out"]
FW = ["xc", "xs", "gc", "gsc", "uc", "us", "dc", "ds", "rw", "gs", "go", "gpo", "gidx", "ws", "out"]
TABLES = {"gs", "go", "gpo", "gidx", "rw"}


@pytest.mark.parametrize("fn,names", [("rmoe_gate_up_mxfp4", GU), ("rmoe_down_mxfp4", DN),
                                      ("rmoe_forward_mxfp4", FW)])
def test_product_refusals(fn, names):
    f = getattr(R.lib(), fn)

    def call(H=256, I=384, E=2, Tp=512, pairs=5, M=3, variant=0, **ptr):
        return f(*[ptr.get(n, A16) for n in names], H, I, E, Tp, pairs, M, variant, None)

    assert call(M=0) == OK                                   # no block, nothing launched
    for bad in (dict(H=0), dict(I=-128), dict(E=0), dict(Tp=-1), dict(pairs=-1), dict(M=-1), dict(variant=3),
                dict(variant=-1), dict(Tp=383)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=192), dict(I=100), dict(H=(1 << 20) + 128), dict(M=65536, Tp=65536 * 128)):
        assert call(**bad) == SHAPE, bad
    for n in names:
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD2 if n in TABLES else ODD8}) == MISALIGNED, n


def test_pick_variant():
    assert R.pick_variant_mxfp4(0, 1) == "stream"
    assert R.pick_variant_mxfp4(1 << 20, 8) == "tile"
    assert R.pick_variant_mxfp4(5, 8, "tile") == "tile"
    f = R.lib().rmoe_pick_variant_mxfp4
    assert f(0, -1, 1) == INVALID and f(0, 1, 0) == INVALID and f(3, 1, 1) == INVALID


def test_binding_refuses_cpu_tensors_and_types():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        R.quantize_mxfp4(torch.zeros(4, 256, dtype=torch.float16))
    with pytest.raises(ValueError):
        R.dequantize_mxfp4(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 8, dtype=torch.uint8), 512)
    with pytest.raises(TypeError):
        R.dequantize_mxfp4(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 8, dtype=torch.uint8), 256,
                           dtype=torch.float64)


# the longest row lengths that 64 bits hold, a multiple of 8: the chunk count must not wrap around
HUGE = [(1 << 63) - 8, (1 << 63) - 256, 1 << 62]


@pytest.mark.parametrize("cols", HUGE)
def test_row_lengths_next_to_the_end_of_64_bits(cols):
    L = R.lib()
    assert L.rmoe_mxfp4_chunks(cols) == -(-cols // 256)
    for rows in (1, 4):
        assert L.rmoe_quantize_mxfp4(A16, 0, 1, rows, cols, A16, A16, None) == SHAPE
        assert L.rmoe_dequantize_mxfp4(A16, A16, 0, 1, rows, cols, A16, None) == SHAPE
        assert L.rmoe_pack_mxfp4_f16(A16, A16, A16, A16, rows, 2, cols, A16, A16, A16, 512, None) == SHAPE


@pytest.mark.parametrize("fn,names", [("rmoe_gate_up_mxfp4", GU), ("rmoe_down_mxfp4", DN), ("rmoe_forward_mxfp4", FW)])
@pytest.mark.parametrize("variant", [0, 1, 2])
def test_odd_padded_row_counts(fn, names, variant):
    """The scales of a chunk lie 8 Tp bytes after the chunk's before, and are
    16-byte aligned only for an even Tp."""
    f = getattr(R.lib(), fn)
    for Tp in (385, 511, 513):
        assert f(*[A16] * len(names), 512, 512, 2, Tp, 5, 3, variant, None) == SHAPE
    assert f(*[A16] * len(names), 512, 512, 2, 514, 0, 0, variant, None) == OK

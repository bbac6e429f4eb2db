"""GPU tests of the MXFP4 stages at sizes that small cases do not reach:
every number of waves per workgroup of the streaming family with passes of
every width, and tiled launches with more items than workgroups, whose next
item is fetched while the one before is written.  Checked as the small cases
are (bounds there), with the operands' values read through the library's
dequantisation, which is exact in fp32."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import test_gpu_mxfp4 as M
from oracle import mxfp4 as MX

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def values_on_the_gpu(monkeypatch):
    monkeypatch.setattr(M, "_val", lambda c, s, cols: R.dequantize_mxfp4(
        c.contiguous(), s.contiguous(), cols, dtype=torch.float32).double())


def _stages(counts, H, I, variant, seed):
    print(f"[mx] {variant} counts={counts} H={H} I={I}", flush=True)
    d = M._case(counts, H, I, seed=seed)
    M._gate_up(d, variant)
    M._down(d, variant)
    torch.cuda.synchronize()
    M._check(d)


# Passes of 8, 16, 32, 48 and 64 token rows, and two of them, in one, two and
# four waves per workgroup: one wave from I / 32 * experts (gate/up) or H / 64
# * experts (down) of 512 on, two from 256 on.  K in whole chunks of 256, in
# half ones, and in fewer chunks than waves.
@pytest.mark.parametrize("counts", [[9, 16, 17, 33, 47, 64, 65, 128], [8, 1, 40, 56, 72, 96, 113, 127]])
@pytest.mark.parametrize("H,I", [(4096, 2048), (4224, 2176), (2048, 1024), (2176, 1152), (2048, 128), (256, 1024),
                                 (512, 384)])
def test_streaming_passes(counts, H, I):
    _stages(counts, H, I, "stream", seed=H + I + counts[0])


# More than 256 items per stage, whole blocks of 128 rows, lone last blocks;
# K loops of one step, of a few and of many
@pytest.mark.parametrize("counts,H,I", [([5000, 3000, 0, 2000], 2048, 2048), ([1100, 900, 0, 700], 256, 8192),
                                        ([1100, 900, 0, 700], 8192, 256), ([256, 1024, 640, 131], 384, 8320)])
def test_tiled_items_one_after_another(counts, H, I):
    _stages(counts, H, I, "tile", seed=H + I)


@pytest.mark.parametrize("variant", ["stream", "tile"])
@pytest.mark.parametrize("which", ["wg", "wu", "wd"])
def test_nan_block_of_a_weight(which, variant):
    """An infinity in a weight makes its block NaN (codes 0, scale byte 255):
    NaN wherever that weight takes part, also against zeros, and nowhere
    else."""
    d = M._case([3, 70, 5], 256, 384, seed=10)
    n, k = (256, 384) if which == "wd" else (384, 256)
    w = torch.randn((3, n, k), generator=torch.Generator().manual_seed(1)) / k ** 0.5
    w[1, 77, 40] = float("inf")
    d[which] = R.quantize_mxfp4(w.cuda())
    start = int(d["c"]["group_padded_offsets"][1])
    d["codes"][start + 69].zero_(), d["scales"][:, start + 69].zero_()   # a token row of zeros
    M._gate_up(d, variant)
    M._down(d, variant)
    torch.cuda.synchronize()
    rows = torch.from_numpy(np.sort(d["c"]["padded_row_of_pair"])).long().cuda()
    nan = torch.isnan(d["out"][rows])
    mine = (rows >= start) & (rows < start + 70)
    want = torch.zeros_like(nan)
    if which == "wd":
        want[mine, 77] = True                          # one column of the output
    else:
        want[mine] = True                              # a hidden block, and every output with it
    assert torch.equal(nan, want)


def test_calls_on_given_memory_and_streams():
    """Outputs in memory of the caller, of the default type, on a stream that
    is not the current one, given as an object and as a handle; rows of none."""
    x = torch.randn(40, 1416, generator=torch.Generator().manual_seed(2)).half()
    want = MX.quantized_values(x.double().numpy())
    xd, side = x.cuda(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        codes, scales = R.quantize_mxfp4(xd, stream=stream)
        out = torch.full((40, 1416), 7.0, device="cuda")
        torch.cuda.synchronize()
        back = R.dequantize_mxfp4(codes, scales, 1416, stream=stream)
        assert R.dequantize_mxfp4(codes, scales, 1416, out=out, stream=stream) is out
        torch.cuda.synchronize()
        assert back.dtype == torch.float16 and np.array_equal(back.double().cpu().numpy(), want)
        assert np.array_equal(out.double().cpu().numpy(), want)
    for shape in ((0, 256), (0, 3, 256), (2, 0, 256)):
        codes, scales = R.quantize_mxfp4(torch.empty(shape, device="cuda"))
        assert (codes.shape, scales.shape) == R.mxfp4_shapes(shape)
        assert R.dequantize_mxfp4(codes, scales, 256).shape == shape
    i32 = torch.empty(0, dtype=torch.int32, device="cuda")
    f32 = torch.empty(0, device="cuda")
    codes, scales = (torch.full(s, 0x5A, dtype=torch.uint8, device="cuda") for s in R.mxfp4_shapes((128, 256)))
    R.pack_mxfp4(torch.empty((0, 256), dtype=torch.float16, device="cuda"), f32, i32, i32, codes, scales, f32)
    torch.cuda.synchronize()
    assert (codes == 0x5A).all() and (scales == 0x5A).all()


BASE = 4096  # rows that repeat


@pytest.mark.parametrize("variant", ["stream", "tile"])
def test_largest_block_table(variant):
    """65535 blocks of one expert, rows of 640 code bytes: offsets past 2^32
    bytes in the tokens, the hidden rows and the output.  The rows repeat after
    4096, and so must the results, bit for bit; the first 4096 against 64 bits."""
    M_, H, I = 65535, 1152, 1152
    pairs, Tp = (M_ - 1) * 128, M_ * 128
    print(f"[mx] {variant} {M_} blocks H={H} I={I}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    u8 = lambda s, v: torch.full(s, v, dtype=torch.uint8, device="cuda")  # noqa: E731
    qc, qs = R.quantize_mxfp4(rnd(BASE, H))
    (cs, ss), (hcs, hss) = R.mxfp4_shapes((Tp, H)), R.mxfp4_shapes((Tp, I))
    d = {"E": 1, "H": H, "I": I, "Tp": Tp, "pairs": pairs, "codes": u8(cs, 0xFF), "scales": u8(ss, 0xFF),
         "hc": u8(hcs, 0x5A), "hs": u8(hss, 0xA5), "gs": i32(pairs), "go": i32(0, pairs), "gpo": i32(0, Tp),
         "gidx": torch.zeros(M_, dtype=torch.int32, device="cuda"),
         "wg": R.quantize_mxfp4(rnd(1, I, H) / H ** 0.5), "wu": R.quantize_mxfp4(rnd(1, I, H) / H ** 0.5),
         "wd": R.quantize_mxfp4(rnd(1, H, I) / I ** 0.5)}
    whole = pairs // BASE * BASE
    d["codes"][:whole].view(-1, BASE, cs[1]).copy_(qc)
    d["codes"][whole:pairs].copy_(qc[:pairs - whole])
    d["scales"][:, :whole].view(ss[0], -1, BASE, 8).copy_(qs[:, None])
    d["scales"][:, whole:pairs].copy_(qs[:, :pairs - whole])
    d["rw"] = torch.rand(BASE, generator=g, device="cuda").repeat(whole // BASE + 1)[:pairs].contiguous()
    d["out"] = torch.full((Tp, H), 0x7E5A, dtype=torch.int16, device="cuda").view(torch.float16)
    M._gate_up(d, variant)
    M._down(d, variant)
    torch.cuda.synchronize()
    bits = d["out"].view(torch.int16)
    for t, rows in ((d["hc"], 0), (bits, 0), (d["hs"], 1)):
        first = t.narrow(rows, 0, BASE)
        for p in range(BASE, pairs, BASE):
            n = min(BASE, pairs - p)
            assert torch.equal(t.narrow(rows, p, n), first.narrow(rows, 0, n)), p
    assert (d["hc"][pairs:] == 0x5A).all() and (d["hs"][:, pairs:] == 0xA5).all() and (bits[pairs:] == 0x7E5A).all()
    f = {**d, "Tp": BASE, "counts": [BASE], "c": {"group_padded_offsets": [0], "group_offsets": [0]}}
    for n in ("codes", "hc", "out"):
        f[n] = d[n][:BASE]
    for n in ("scales", "hs"):
        f[n] = d[n][:, :BASE].contiguous()
    M._check(f)

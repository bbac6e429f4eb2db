"""GPU tests of the training pass at sizes that small cases do not reach:
launches with more items than workgroups, whose next item is fetched while
the one before is written, in every stage.  Checked against 64 bits as the
small cases are (bounds there)."""
import pytest
import torch

import test_gpu_train as T

pytestmark = pytest.mark.gpu


# More than 256 items in every row product and weight-gradient tiles of many
# steps; K loops of two steps in the first products, and of four in dx; and
# weight gradients of a single step each
@pytest.mark.parametrize("counts,H,I", [([5000, 3000, 0, 2000], 2048, 2048), ([1100, 900, 0, 700], 128, 8192),
                                        ([1100, 900, 0, 700], 8192, 128), ([256, 1024, 640, 131], 8320, 384),
                                        ([40, 64, 1, 63, 33] * 4, 1024, 1152)])
def test_items_one_after_another(counts, H, I):
    print(f"[train] counts={counts} H={H} I={I}", flush=True)
    d = T._case(counts, H, I, seed=H + I)
    T._forward(d)
    torch.cuda.synchronize()
    T._check_forward(d)
    print("[train] backward", flush=True)
    T._backward(d)
    torch.cuda.synchronize()
    T._check_backward(d)
    T._untouched(d, ["dgate", "dup", "whidden", "dx"])


def test_few_large_experts():
    """8 uneven experts of 4096 x 14336, 8192 rows: K loops of 64 and 448
    steps, a last, partly free round of dx items."""
    counts, H, I = [1000, 1048, 900, 1148, 1024, 1024, 800, 1248], 4096, 14336
    print(f"[train] counts={counts} H={H} I={I}", flush=True)
    d = T._case(counts, H, I, seed=1)
    T._forward(d)
    torch.cuda.synchronize()
    T._check_forward(d)
    print("[train] backward", flush=True)
    T._backward(d)
    torch.cuda.synchronize()
    T._check_backward(d)
    T._untouched(d, ["dgate", "dup", "whidden", "dx"])


def test_largest_block_table():
    """65535 blocks of one expert, more than 2^32 elements per tensor of I
    columns.  A few rows, on both sides of the 32-bit borders, hold an output
    gradient; every other row's is zero, so each gradient is theirs alone."""
    M, H, I = 65535, 512, 640
    pairs, Tp = (M - 1) * 128, M * 128
    print(f"[train] {M} blocks H={H} I={I}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bits = lambda *s: torch.full(s, T.BITS, dtype=torch.int16, device="cuda").view(torch.float16)  # noqa: E731
    some = [0, 127, 128, (1 << 31) // I - 1, (1 << 31) // I + 1, (1 << 31) // H, (1 << 32) // I, (1 << 32) // I + 1,
            pairs - 129, pairs - 1]
    at = torch.tensor(some, device="cuda")
    d = {"E": 1, "H": H, "I": I, "Tp": Tp, "pairs": pairs, "gs": i32(pairs), "go": i32(0, pairs), "gpo": i32(0, Tp),
         "gidx": torch.zeros(M, dtype=torch.int32, device="cuda"), "wg": rnd(1, I, H) / H ** 0.5,
         "wu": rnd(1, I, H) / H ** 0.5, "wd": rnd(1, H, I) / I ** 0.5,
         "rw": torch.rand(pairs, generator=g, device="cuda"),
         "scratch": torch.full((pairs * 5,), float("nan"), device="cuda"),
         "drw": torch.full((pairs,), float("nan"), device="cuda")}
    base = rnd(4096, H)
    d["x"], d["dout"] = bits(Tp, H), bits(Tp, H)
    for p in range(0, pairs, 4096):
        d["x"][p:min(p + 4096, pairs)] = base[:min(4096, pairs - p)]
    d["x"][at], d["dout"][:pairs] = rnd(len(some), H), 0.0
    d["dout"][at] = rnd(len(some), H)
    for n in ("gate", "up", "hidden", "dgate", "dup", "whidden"):
        d[n] = bits(Tp, I)
    d["dx"], d["dgw"], d["duw"], d["ddw"] = bits(Tp, H), bits(1, I, H), bits(1, I, H), bits(1, H, I)
    T._forward(d)
    T._backward(d)
    torch.cuda.synchronize()
    for n in ("gate", "up", "hidden", "dgate", "dup", "whidden", "dx"):
        assert (d[n][pairs:].view(torch.int16) == T.BITS).all(), n
    rest = torch.ones(pairs, dtype=torch.bool, device="cuda")
    rest[at] = False
    for n in ("dgate", "dup", "dx", "drw"):
        assert not (d[n][:pairs] != 0).view(pairs, -1).any(1)[rest].any(), n
    # the picked rows by themselves, as a group of their own
    k = len(some)
    f = {**d, "Tp": k, "counts": [k], "c": {"group_padded_offsets": [0], "group_offsets": [0]}}
    for n in ("x", "dout", "gate", "up", "hidden", "dgate", "dup", "whidden", "dx", "rw", "drw"):
        f[n] = d[n][at]
    T._check_forward(f)
    T._check_backward(f)

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

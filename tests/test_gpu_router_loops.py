"""GPU tests of the training router where its loops go round: several tiles of
tokens per workgroup of dx and several parts of the gate matrix's gradient for
every count of expert tiles, and 64 tokens per workgroup, as one block and as
two lagging halves, with every form of the expert tiles.  Bounds as in
test_gpu_router_train.py."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
from oracle import router_train as RB
from test_gpu_router_train import _backward, _check_backward, _check_forward, _inputs, _np

pytestmark = pytest.mark.gpu


def _regime(T, E, H):
    """(tiles of 32 tokens per dx workgroup, parts of the gate matrix's
    gradient), as the launcher cuts them."""
    tiles, blocks = -(-T // 32), -(-T // 64)
    slices, groups = -(-H // 256), -(-(-(-E // 32)) // 4)
    parts = max(1, min(256 // (slices * groups), blocks // 4))
    wgs = 512 - -(-slices * parts // 8) * 8 if E <= 128 else 512 + slices - 1
    return tiles / max(1, min(tiles, wgs // slices)), parts


@pytest.mark.parametrize("T,E,k,H,left_out", [(20001, 96, 4, 320, 0.1), (20001, 128, 8, 320, 0.3), (20001, 64, 6, 576, 0),
                                              (40001, 160, 3, 192, 0.2), (40001, 192, 4, 64, 0), (40001, 224, 5, 192, 0.5),
                                              (40001, 256, 8, 192, 0.1), (20001, 1, 1, 320, 0.2)])
def test_backward_of_many_tiles_and_parts(T, E, k, H, left_out):
    per_wg, parts = _regime(T, E, H)
    assert per_wg > 2 and parts > 8, (per_wg, parts)
    print(f"[router_backward loops] T={T} E={E} k={k} H={H}", flush=True)
    x, w, mask, xg, wg, mg = _inputs(T, E, H, T + E, left_out)
    f = RB.forward(x, w, k, mask)
    rng = np.random.default_rng(T)
    g, ab = rng.standard_normal((T, k)), (0.02 * T, -0.003 * T)
    add = torch.from_numpy(rng.standard_normal((T, H)) * 1e-2).half()
    dx, dw = _backward(f, xg, wg, mg, g, ab)
    _check_backward(dx, dw, f, x, w, mask, g, ab)
    dx2, dw2 = _backward(f, xg, wg, mg, g, ab, add=add.cuda(), compact=True)
    _check_backward(dx2, dw2, f, x, w, mask, g, ab, _np(add))
    assert torch.equal(dw, dw2)
    dx3, dw3 = _backward(f, xg, wg, mg, g, ab, add=add.cuda(), compact=True, alias=True)
    assert torch.equal(dx2, dx3) and torch.equal(dw, dw3)


@pytest.mark.parametrize("H", [64, 576])
@pytest.mark.parametrize("E", [96, 130, 160, 224])
@pytest.mark.parametrize("per_cu", [64, 128])
def test_forward_of_64_tokens_per_workgroup(per_cu, E, H):
    """From 64 tokens per compute unit on two lagging halves, from 128 on one
    block; the last pair of waves has no tile of its own with an odd count."""
    T = per_cu * torch.cuda.get_device_properties(0).multi_processor_count + 5
    print(f"[router_train loops] T={T} E={E} H={H}", flush=True)
    x, w, mask, xg, wg, mg = _inputs(T, E, H, T + E, 0.2)
    got = R.router_train(xg, wg, 5, token_mask=mg)
    torch.cuda.synchronize()
    _check_forward(got, x, w, 5, mask)
    ids, vals = R.router(torch.where(mg[:, None] > 0, xg, 0), wg, 5)
    torch.cuda.synchronize()
    on = mg > 0
    assert torch.equal(ids[on], got["topk_ids"][on]) and torch.equal(vals[on], got["topk_weights"][on])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_forward_of_a_token_without_a_choice(value):
    """A NaN or +infinite logit: no expert, the weight -1, NaN probabilities;
    the other tokens as without it."""
    _, _, _, xg, wg, _ = _inputs(70, 12, 128, 3)
    wg[:, 3] = 0.5
    plain = R.router_train(xg, wg, 3)
    bad = xg.clone()
    bad[5, 3] = value
    got = R.router_train(bad, wg, 3)
    torch.cuda.synchronize()
    rest = [t for t in range(70) if t != 5]
    assert (got["topk_ids"][5] == 2 ** 31 - 1).all() and (got["topk_weights"][5] == -1).all()
    assert torch.isnan(got["probs"][5]).all() and torch.isnan(got["losses"]).all()
    for n in ("topk_ids", "topk_weights", "probs", "lse"):
        assert torch.equal(got[n][rest], plain[n][rest]), n

"""GPU tests of the MXFP4 stages on row counts of the padded layout that are
no multiple of a block: a chunk's token scales then start at other offsets."""
import numpy as np
import pytest
import torch

import mixture_experts_routed_grouped_amd as R
import test_gpu_mxfp4 as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", ["stream", "tile"])
@pytest.mark.parametrize("more", [2, 66, 130])
def test_more_rows_than_blocks(more, variant):
    """Rows behind the last block belong to nobody and stay as they were."""
    print(f"[mx] {variant} {more} rows behind the last block", flush=True)
    d = M._case([130, 0, 40, 3], 640, 768, seed=12)
    d["Tp"] += more
    grown = lambda t, dim: torch.cat([t, t.narrow(dim, 0, 1).expand(  # noqa: E731
        *[more if i == dim else -1 for i in range(t.dim())])], dim).contiguous()
    for name, dim in (("codes", 0), ("scales", 1), ("hc", 0), ("hs", 1)):
        d[name] = grown(d[name], dim)
    d["out"] = grown(d["out"].view(torch.int16), 0).view(torch.float16)
    M._gate_up(d, variant)
    M._down(d, variant)
    torch.cuda.synchronize()
    M._check(d)


def test_pack_of_many_experts_per_token():
    """More experts per token than a half-wave has lanes, one of them twice."""
    T, k, E, H = 5, 40, 64, 520
    rng = np.random.default_rng(0)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[2, 7] = ids[2, 3]
    c = R.build_contract(ids, E)
    Tp, prow, cpos = c["total_padded_tokens"], c["padded_row_of_pair"], c["compact_pos_of_pair"]
    x, w = torch.from_numpy(rng.standard_normal((T, H))).half().cuda(), torch.rand(T * k, device="cuda")
    codes, scales = (torch.full(s, 0x5A, dtype=torch.uint8, device="cuda") for s in R.mxfp4_shapes((Tp, H)))
    wc = torch.full((T * k,), -7.0, device="cuda")
    R.pack_mxfp4(x, w, torch.from_numpy(prow).cuda(), torch.from_numpy(cpos).cuda(), codes, scales, wc)
    qc, qs = R.quantize_mxfp4(x)
    torch.cuda.synchronize()
    rows, tok = torch.from_numpy(prow).long().cuda(), torch.arange(T * k, device="cuda") // k
    assert torch.equal(codes[rows], qc[tok]) and torch.equal(scales[:, rows], qs[:, tok])
    assert torch.equal(wc[torch.from_numpy(cpos).long().cuda()], w)
    rest = torch.ones(Tp, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert (codes[rest] == 0x5A).all() and (scales[:, rest] == 0x5A).all()

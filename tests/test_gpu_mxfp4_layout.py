"""GPU tests of the MXFP4 stages on row counts of the padded layout that are
no multiple of a block: a chunk's token scales then start at other offsets."""
import pytest
import torch

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

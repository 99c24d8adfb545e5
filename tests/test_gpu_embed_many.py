"""qmv_embed of more rows than one launch's work-items reach at one row a workgroup (2^24 x 256 work-items are 2^32)."""
import pytest
import torch

from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, Weights, say

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_grid_of_workgroups():
    rows, cols, n = 61, 65 * 32, (1 << 24) + 77  # 130 sixteens of columns: a row a workgroup
    say(f"embed {n} rows of {cols}")
    w = Weights("q8_0", rows, cols, seed=8)
    dense = torch.zeros(rows + 1, cols, dtype=torch.float16, device=DEV)  # (the last: ids outside the table)
    qmv.qmv_dequant(w.desc, dense[:rows], "f16")
    ids = (torch.arange(n, device=DEV) * 7919 % (rows + 1)).to(torch.int32)
    out = torch.full((n + 1, cols), 7.0, dtype=torch.float16, device=DEV)
    qmv.qmv_embed(w.desc, ids, n, out, "f16")
    for at in range(0, n, 1 << 20):
        end = min(n, at + (1 << 20))
        assert torch.equal(out[at:end], dense[ids[at:end].long()]), at
    assert bool((out[n] == 7.0).all())
    del out
    torch.cuda.empty_cache()

"""qmv_verify where sequences have more than max_rows rows: as if they ended there, whole numbers, equal to the oracle's."""
import numpy as np
import pytest
import torch

from oracle.step import verify64
from gpu_util import say
from test_gpu_verify import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("u", [0.0, None, 1.0 - 2.0**-24])  # every draft accepted, some, few
@pytest.mark.parametrize("max_rows", [1, 2, 3, 4])
def test_rows_past_max_rows_are_as_if_not_there(max_rows, u, probs):
    rows, temp = [5, 2, 7, 4, 1], [1.0, 0.7, 0.0, 0.0, 1.3]
    for seed in range(3):
        say(f"verify max_rows {max_rows} u {u} probs {probs} seed {seed}")
        s = make(700, rows, "f32", probs, temp, seed=20 + seed)
        if u is not None:
            s["u_accept"][:] = u
        got, acc = run(s, max_rows=max_rows)
        start = s["row_start"].numpy()
        kept = [min(n, max_rows) for n in rows]
        keep = np.concatenate([np.arange(a, a + n) for a, n in zip(start[:-1], kept)])
        cut = np.concatenate([[0], np.cumsum(kept)]).astype(np.int32)
        f = lambda x: None if x is None else x.double().numpy()[keep]  # noqa: E731
        want, wacc, margin = verify64(f(s["logits"]), s["tokens"].numpy()[keep], cut, s["u_accept"].numpy()[keep],
                                      s["u_sample"].numpy(), None if not probs else s["draft_probs"].numpy()[keep],
                                      s["temperature"].numpy())
        assert margin.min() > 1e-10
        whole = np.full(sum(rows), -1, np.int32)
        whole[keep] = want
        assert np.array_equal(acc, wacc) and np.array_equal(got, whole), (acc, wacc, got, whole)

"""qmv_attn with infinities among the keys that rows see: the same by every tile and at every head width.

A key whose score is -inf weighs nothing: the output is, bit for bit, that of a finite key whose weight is 0."""
import pytest
import torch

from gpu_util import say
from test_gpu_attn import Step

pytestmark = pytest.mark.gpu

INF = float("inf")
# rows of each sequence, heads: at most 16 rows of a key head, at most 64, more
SHAPES = {"few": ([1, 2], 4), "some": ([5, 4], 6), "many": ([8] * 9, 4)}


def places(s, where):
    """(k, v) views of one key [kv, D] that every row (suffix, draft: every row of sequence 0) sees."""
    if where == "first":
        return s.kp[0], s.vp[0]
    if where == "prefix":
        return s.kp[len(s.kp) - 7], s.vp[len(s.kp) - 7]
    j = 3 if where == "suffix" else s.suffix[0] - s.rows[0]  # draft: the first row's own token
    page = int(s.table[0, j // s.page])
    return s.k_pages[page, j % s.page], s.v_pages[page, j % s.page]


@pytest.mark.parametrize("dim", [8, 64, 72, 80, 96, 128, 200, 256])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_key_of_minus_infinity_weighs_nothing(dtype, shape, dim):
    rows, heads = SHAPES[shape]
    for where in ("first", "prefix", "suffix", "draft"):
        for col in (3, dim - 1):
            say(f"attn key -inf {dtype} {shape} dim {dim} {where} column {col}")
            s = Step(dtype, heads, 2, dim, 150, rows, [40 + n for n in rows], seed=dim)
            s.q[..., col] = s.q[..., col].abs() + 1.0
            k, _ = places(s, where)
            k[:, col] = -60000.0  # a score below -160 whatever the other columns are
            want, lse = s.run().clone(), s.lse.clone()
            k[:, col] = -INF
            s.run()
            assert torch.equal(s.out, want) and torch.equal(s.lse, lse)
            assert bool(s.out.isfinite().all())


def test_a_key_of_infinity_is_nan_for_the_heads_that_read_it():
    for rows, heads in SHAPES.values():
        s = Step("f16", heads, 2, 72, 100, rows, [20 + n for n in rows], seed=4)
        s.q[..., 2] = 1.0
        clean = s.run().clone()
        s.kp[50, 1, 2] = INF
        s.run()
        half = heads // 2
        assert torch.equal(s.out[:, :half], clean[:, :half]) and bool(s.out[:, half:].isnan().all())

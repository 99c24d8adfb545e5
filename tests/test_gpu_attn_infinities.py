"""qmv_attn with infinities among the keys and values that rows see: the same by every tile and at every head width.

A key whose score is -inf weighs nothing: the output is, bit for bit, that of a finite key whose weight is 0.  An infinite
value that a row sees gives that infinity in its column (NaN where both signs meet), and the other columns stay
within the tolerance of test_gpu_attn.py."""
import numpy as np
import pytest
import torch

from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say
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


def check_but(s, col):
    """The finite columns against the oracle; returns the column."""
    got = s.out[..., col].clone()
    for x in [x for x in (s.vp, s.v_pages) if x is not None]:
        x[..., col] = torch.where(x[..., col].isinf(), 0.0, x[..., col])
    b, _, _, _ = s.oracle()
    s.out[..., col] = torch.from_numpy(b[..., col]).to(s.out.dtype).to(DEV)
    s.check()
    return got


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_an_infinite_value_is_infinite_in_its_column(dtype, shape, dim):
    rows, heads = SHAPES[shape]
    for where in ("first", "prefix", "suffix", "draft"):
        for value in (INF, -INF):
            say(f"attn value {value} {dtype} {shape} dim {dim} {where}")
            s = Step(dtype, heads, 2, dim, 150, rows, [40 + n for n in rows], seed=dim)
            _, v = places(s, where)
            v[:, 5] = value
            s.run()
            got = check_but(s, 5)
            mine = got[:rows[0]] if where in ("suffix", "draft") else got
            assert bool((mine == value).all())
            if where in ("suffix", "draft"):
                assert bool(got[rows[0]:].isfinite().all())


def test_one_token():
    # its weight is 1 exactly
    for shape, (rows, heads) in SHAPES.items():
        s = Step("f16", heads, 2, 64, 1, rows, [0] * len(rows), seed=1)
        s.vp[0, :, 7] = -INF
        s.run()
        assert bool((check_but(s, 7) == -INF).all())


def test_rising_maxima():
    # many tiles of one range, each with a larger maximum than the last, and an infinity in an early one
    for dtype in ("bf16", "f16"):
        for rows, heads in SHAPES.values():
            s = Step(dtype, heads, 2, 64, 2048, rows, rows, seed=2)
            s.q[..., 0] = 8.0
            s.kp[..., 0] = (torch.arange(2048, device=DEV) * (60.0 / 2048))[:, None].to(s.q.dtype)
            for j in (1800, 2040):
                s.vp[j, :, 9] = INF
            s.run()
            assert bool((check_but(s, 9) == INF).all())


def test_both_signs_meet():
    for rows, heads in SHAPES.values():
        s = Step("bf16", heads, 2, 80, 100, rows, [20 + n for n in rows], seed=3)
        s.vp[4, :, 0], s.vp[70, :, 0] = INF, -INF
        s.run()
        assert bool(check_but(s, 0).isnan().all())


def test_a_key_of_infinity_is_nan_for_the_heads_that_read_it():
    for rows, heads in SHAPES.values():
        s = Step("f16", heads, 2, 72, 100, rows, [20 + n for n in rows], seed=4)
        s.q[..., 2] = 1.0
        clean = s.run().clone()
        s.kp[50, 1, 2] = INF
        s.run()
        half = heads // 2
        assert torch.equal(s.out[:, :half], clean[:, :half]) and bool(s.out[:, half:].isnan().all())


def test_infinities_with_pages_outside_the_pool_and_trees():
    for rows, heads in SHAPES.values():
        s = Step("bf16", heads, 2, 64, 90, rows, [50 + n for n in rows], page=8, paged_prefix=True, tree=True, seed=5,
                 bad=[(0, 1, -1)])
        s.prefix_pages[3] = 1 << 20
        s.v_pages[int(s.prefix_pages[5]), 2, :, 11] = INF
        s.run()
        assert bool((check_but(s, 11) == INF).all())


def test_large_finite_values_stay_finite():
    # unnormalized sums of them pass fp32's range, their means do not
    for rows, heads in SHAPES.values():
        for dim in (64, 72):
            s = Step("bf16", heads, 2, dim, 300, rows, [20 + n for n in rows], seed=6)
            for x in (s.vp, s.v_pages):
                x[x.isfinite()] = 1.5e38
            s.run()
            s.check()


def test_infinities_where_rows_and_sequences_are_few_many_or_none():
    for seqs in (5, 70):  # (fewer than 64 sequences are looked up at once)
        rows = [(0, 2, 1, 3)[i % 4] for i in range(seqs)]
        s = Step("f16", 4, 2, 72, 40, rows, [(0, 9, 1, 3)[i % 4] for i in range(seqs)], page=8, outside=2, seed=seqs)
        s.vp[11, :, 4] = -INF
        s.run()
        assert bool((check_but(s, 4) == -INF).all())


def test_infinities_without_a_prefix():
    # three rows, two of their tokens cached: the first row sees nothing
    s = Step("bf16", 4, 2, 64, 0, [3, 4], [2, 30], page=8, seed=7)
    s.v_pages[int(s.table[0, 0]), 0, :, 6] = INF
    s.v_pages[int(s.table[1, 3]), 5, :, 6] = -INF  # its last row's own
    s.run()
    got = check_but(s, 6)
    assert bool((got[0] == 0).all()) and bool((got[1:3] == INF).all())
    assert bool(got[3:6].isfinite().all()) and bool((got[6] == -INF).all())


def test_infinities_in_a_captured_call():
    s = Step("bf16", 14, 2, 128, 2000, [8] * 12, [38] * 12, seed=8)
    s.vp[1000, :, 3] = INF
    want, lse = s.run().clone(), s.lse.clone()
    assert bool((want[..., 3] == INF).all())
    a = s.args()
    nws = qmv.qmv_attn_workspace_size(a)
    ws, st, g = torch.empty(nws, dtype=torch.uint8, device=DEV), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        qmv.qmv_attn(a, ws, nws, st)
    for _ in range(4):
        s.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, want) and torch.equal(s.lse, lse)
        assert torch.equal(s.run(), want)

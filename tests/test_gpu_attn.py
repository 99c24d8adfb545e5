"""qmv_attn against the float64 oracle.

Tolerances.  A score is a product sum of D terms in fp32: off by at most (D + 8) 2^-24 smax, smax the sum of its
terms' magnitudes (with the scale and the exponent's argument); twice that (itself and the maximum) is the relative
error of a probability, plus 2^-22 of the exponential.  A probability enters the second product within 2^-16 of
itself -- or, for the prefix's keys where a key head has more than 64 rows, rounded once to the type (half its
epsilon, both in the sum and in the weights) -- and n of them are added in fp32 (n 2^-24).  Numerator and denominator
both carry these, so an output is off by at most mag (4 smax (D + 8) 2^-24 + 2^-15 + 2^-21 + 4 n 2^-24, and the
epsilon), mag the probabilities' mean of |v|, plus its own rounding: half the type's epsilon (fp16: at least 2^-25,
its subnormal step)."""
import numpy as np
import pytest
import torch

from oracle.step import attn64
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Step:
    """One call's tensors, seeded.  rows: rows of each sequence; suffix: tokens of each; poison: what no row sees is NaN."""

    def __init__(self, dtype, heads, kv, dim, prefix, rows, suffix, page=16, tree=False, seed=0, paged_prefix=False,
                 poison=True, bad=(), outside=0, scale=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        t = TYPES[dtype]
        self.dtype, self.kv, self.page, self.prefix, self.rows, self.suffix = dtype, kv, page, prefix, rows, suffix
        n = sum(rows) + outside
        self.scale = scale or dim ** -0.5

        def normal(*shape):
            return (torch.randn(*shape, generator=g) * spread).to(t).to(DEV)

        self.q = normal(n, heads, dim)
        per = [-(-s // page) for s in suffix]
        ppre = -(-prefix // page) if paged_prefix else 0
        pages = sum(per) + ppre + 1
        order = torch.randperm(pages, generator=g)[:pages - 1].tolist()  # one page stays unused
        self.k_pages, self.v_pages = normal(pages, page, kv, dim), normal(pages, page, kv, dim)
        self.kp = self.vp = self.prefix_pages = None
        if paged_prefix:
            self.prefix_pages = torch.tensor(order[:ppre], dtype=torch.int32, device=DEV)
        elif prefix:
            self.kp, self.vp = normal(prefix, kv, dim), normal(prefix, kv, dim)
        table = torch.full((len(rows), max(per + [1]) + 1), 1 << 30, dtype=torch.int32)
        at = ppre
        for b, k in enumerate(per):
            table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        if poison:
            used = torch.zeros(pages, page, dtype=torch.bool)
            for j in range(prefix if paged_prefix else 0):
                used[order[j // page], j % page] = True
            for b, s in enumerate(suffix):
                for j in range(s):
                    used[table[b, j // page], j % page] = True
            self.k_pages[~used.to(DEV)] = float("nan")
            self.v_pages[~used.to(DEV)] = float("nan")
        for b, entry, number in bad:
            table[b, entry] = number
        self.table = table.to(DEV)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.row_start = torch.from_numpy(self.start).to(DEV)
        self.suffix_len = torch.tensor(suffix, dtype=torch.int32, device=DEV)
        self.mask = None
        if tree:
            m = torch.randint(0, 1 << 62, (n,), generator=g)
            m[0] = 0  # this row sees no row, not even itself
            self.mask = m.to(DEV)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((n, heads), 7.0, device=DEV)

    def args(self, out=None, **over):
        k = dict(scale=self.scale, k_prefix=self.kp, v_prefix=self.vp, prefix_pages=self.prefix_pages,
                 k_pages=self.k_pages, v_pages=self.v_pages, block_table=self.table, suffix_len=self.suffix_len,
                 max_suffix=max(self.suffix), tree_mask=self.mask, lse=self.lse)
        if self.prefix_pages is not None:
            k["prefix_len"] = self.prefix
        k.update(over)
        return qmv.qmv_create_attn(self.q, self.out if out is None else out, self.row_start, max(max(self.rows), 1), **k)

    def run(self, stream=None, **over):
        a = self.args(**over)
        nws = qmv.qmv_attn_workspace_size(a)
        ws = torch.full((nws,), 255, dtype=torch.uint8, device=DEV)  # NaN patterns: nothing may rely on its contents
        qmv.qmv_attn(a, ws, nws, stream)
        return self.out

    def oracle(self):
        f = lambda x: None if x is None else x.cpu().double().numpy()  # noqa: E731
        i = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
        return attn64(f(self.q), self.start, self.scale, f(self.kp), f(self.vp), i(self.prefix_pages), self.prefix,
                      f(self.k_pages), f(self.v_pages), i(self.table), self.suffix, i(self.mask))

    def check(self):
        out, lse = self.out.cpu().double().numpy(), self.lse.cpu().double().numpy()
        want, wlse, mag, smax = self.oracle()
        d, n = self.q.shape[2], self.prefix + max(self.suffix)
        rel = 4 * smax * (d + 8) * 2.0**-24 + 2.0**-15 + 2.0**-21 + 4 * n * 2.0**-24
        half = torch.finfo(TYPES[self.dtype]).eps / 2
        eps = torch.finfo(TYPES[self.dtype]).eps
        once = eps if self.q.shape[0] * (self.q.shape[1] // self.kv) > 64 and self.prefix else 0.0
        rel = rel + once
        tol = mag * rel[..., None] * (1 + half) + np.abs(want) * half + (2.0**-25 if self.dtype == "f16" else 0)
        worst = np.max(np.abs(out - want) / np.maximum(tol, 1e-30))
        say(f"  worst error / tolerance {worst:.3f}")
        assert np.all(np.abs(out - want) <= tol)
        none = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(lse), none)
        wlse[none] = lse[none] = 0.0
        tl = np.abs(wlse) * 2.0**-22 + 2 * smax * (d + 8) * 2.0**-24 + 2 * n * 2.0**-24 + 2.0**-21 + once / 2
        assert np.all(np.abs(lse - wlse)[~none] <= tl[~none])


HEADS = [(1, 1, 64), (28, 4, 128), (8, 8, 80), (6, 3, 8), (10, 2, 256), (7, 1, 72), (16, 2, 96), (3, 3, 200)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv,dim", HEADS)
def test_head_shapes(heads, kv, dim, dtype):
    say(f"attn heads {heads}/{kv} dim {dim} {dtype}")
    s = Step(dtype, heads, kv, dim, 67, [1, 3, 2], [5, 3, 41], seed=dim)
    s.run()
    s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,suffix", [([1], [40]), ([2], [2]), ([1, 1], [100, 33])])
@pytest.mark.parametrize("heads,kv,dim", HEADS)
def test_few_rows(heads, kv, dim, rows, suffix, dtype):
    # at most 16 rows of a key head
    say(f"attn heads {heads}/{kv} dim {dim} rows {rows} {dtype}")
    s = Step(dtype, heads, kv, dim, 171, rows, suffix, page=8, tree=rows == [2], seed=dim + 1)
    s.run()
    s.check()


def test_few_rows_beside_many():
    # the prefix's rows are many, each sequence's few
    for seqs in (9, 40):
        s = Step("f16", 14, 2, 128, 300, [1] * seqs, [1 + 13 * i % 70 for i in range(seqs)], page=8, seed=seqs)
        s.run()
        s.check()


@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 63, 64, 65, 127, 257, 1030])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefix_lengths(prefix, dtype):
    say(f"attn prefix {prefix} {dtype}")
    s = Step(dtype, 6, 2, 64, prefix, [1, 2], [1, 9], page=8, seed=prefix)
    s.run()
    s.check()


@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
@pytest.mark.parametrize("suffix", [[0, 1], [2, 31], [33, 32], [64, 65], [129, 300], [511, 5]])
def test_suffix_lengths_and_pages(suffix, page):
    say(f"attn suffix {suffix} page {page}")
    s = Step("bf16", 8, 2, 64, 40, [1, 1], suffix, page=page, seed=page)
    s.run()
    s.check()


# rows of a key head together: few, past one wave's tile, past one workgroup's, several workgroups'
@pytest.mark.parametrize("rows,heads,kv", [([1] * 5, 7, 1), ([3] * 11, 4, 4), ([5, 1, 7, 2, 8], 8, 2),
                                           ([8] * 10, 7, 1), ([4] * 40, 6, 2), ([33, 1, 60], 4, 1)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows(rows, heads, kv, tree, dim):
    say(f"attn rows {rows} heads {heads}/{kv} dim {dim} tree {tree}")
    s = Step("bf16", heads, kv, dim, 200, rows, [n + 11 * (i % 5) for i, n in enumerate(rows)], tree=tree, seed=len(rows))
    s.run()
    s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [[2], [6] * 24])
def test_long_prefix_is_split(rows, dtype):
    s = Step(dtype, 4, 2, 64, 9001, rows, [10] * len(rows), seed=3)
    s.run()
    s.check()


def test_many_rows_of_wide_heads():
    s = Step("bf16", 8, 1, 256, 700, [6] * 25, [40] * 25, seed=4)
    s.run()
    s.check()


def test_prefix_in_pages():
    for prefix, page, rows in [(100, 16, [2, 1]), (517, 32, [8] * 9), (3, 64, [1, 1])]:
        s = Step("f16", 8, 2, 64, prefix, rows, [n + 20 for n in rows], page=page, paged_prefix=True, seed=prefix)
        s.run()
        s.check()


def test_pages_outside_the_pool_are_not_seen():
    for rows, heads in (([1, 2, 1], 8), ([8, 5, 8], 8), ([1, 1, 1], 4)):
        s = Step("bf16", heads, 2, 64, 33, rows, [50, 37, 48], page=16, seed=8,
                 bad=[(0, 1, -1), (1, 0, 1 << 30), (2, 0, -(1 << 31)), (2, 1, 9999), (2, 2, 77)])
        s.run()
        s.check()
    s = Step("bf16", 4, 2, 64, 40, [3, 2], [9, 9], page=8, seed=9, paged_prefix=True)
    s.prefix_pages[1] = -5
    s.prefix_pages[4] = 1 << 20
    s.run()
    s.check()


def test_rows_that_see_nothing():
    s = Step("f16", 4, 2, 64, 0, [2, 1, 3], [2, 0, 3], page=8, tree=True, seed=10)
    s.mask[:] = 0
    s.mask[3] = 0b100
    s.run()
    s.check()
    assert not s.out[:3].any() and s.out[3].any()


def test_sequences_without_rows_and_rows_without_sequence():
    s = Step("bf16", 4, 2, 64, 50, [0, 2, 0, 0, 1, 0], [7, 9, 0, 3, 1, 0], page=8, outside=2, seed=11)
    s.run()
    s.check()


def test_suffix_shorter_than_the_rows():
    # three rows, two of their tokens cached: the first row sees no suffix token
    s = Step("bf16", 4, 2, 64, 20, [3, 4], [2, 0], page=8, seed=12)
    s.run()
    s.check()


def test_unseen_drafts_may_hold_anything():
    # tree: rows see only themselves; the other drafts' keys and values are NaN and infinity for them
    for rows, dim, heads in [([4, 3], 64, 6), ([5, 4], 128, 6), ([3, 2], 64, 6), ([4, 3], 72, 4)]:
        s = Step("bf16", heads, 2, dim, 30, rows, [12, 9], page=8, tree=True, seed=13, poison=True)
        s.mask[:] = 1  # everyone sees the first row's token alone
        for b, (n, length) in enumerate(zip(rows, [12, 9])):
            for i, x in zip(range(1, n), [float("nan"), float("inf"), float("-inf"), float("nan")]):
                j = length - n + i
                s.k_pages[s.table[b, j // 8], j % 8] = x
                s.v_pages[s.table[b, j // 8], j % 8] = x
        s.run()
        s.check()


def test_a_later_draft_of_nan_stays_with_the_rows_that_see_it():
    for heads in (4, 6):
        later_draft_of_nan(heads)


def later_draft_of_nan(heads):
    s = Step("f16", heads, 2, 64, 30, [4, 2], [12, 6], page=8, seed=14)
    j = 12 - 1  # the last row's own key and value
    clean = s.run().clone()
    s.v_pages[s.table[0, j // 8], j % 8] = float("inf")
    s.run()
    assert torch.equal(s.out[:3], clean[:3]) and torch.equal(s.out[4:], clean[4:])
    assert bool((s.out[3] == float("inf")).all())
    s.k_pages[s.table[0, j // 8], j % 8] = float("nan")
    s.run()
    assert torch.equal(s.out[:3], clean[:3]) and bool(s.out[3].isnan().all())


def test_large_scores_and_a_late_maximum():
    # scores of hundreds, the largest key last: earlier sums are rescaled to nothing or kept exactly
    for dtype in TYPES:
        s = Step(dtype, 4, 2, 64, 3000, [2, 1], [5, 4], seed=15, spread=4.0, scale=0.5)
        s.kp[2999] = s.kp[2999] * 3
        s.run()
        s.check()


def test_strides():
    # q and out as slices of a wider projection, k and v interleaved, head-major prefix, a table of wider rows
    s = Step("bf16", 8, 2, 64, 75, [2, 3], [20, 17], page=8, seed=16)
    rows = s.q.shape[0]
    want = s.run().clone()
    wide = torch.zeros(rows, 16, 128, dtype=s.q.dtype, device=DEV)
    wide[:, ::2, 64:] = s.q
    s.q = wide[:, ::2, 64:]
    target = torch.full((rows, 9, 80), 5.0, dtype=want.dtype, device=DEV)
    kv = torch.stack([s.kp.transpose(0, 1), s.vp.transpose(0, 1)], 1).contiguous()  # [kv head][k, v][token][D]
    s.kp, s.vp = kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)
    both = torch.stack([s.k_pages, s.v_pages], 2).contiguous()
    s.k_pages, s.v_pages = both[:, :, 0], both[:, :, 1]
    s.table = torch.nn.functional.pad(s.table, (0, 5), value=3)[:, :-5]
    s.run(out=target[:, 1:, 8:72])
    assert torch.equal(target[:, 1:, 8:72], want)
    target[:, 1:, 8:72] = 5.0
    assert bool((target == 5.0).all())  # nothing outside the view


def test_offsets_past_32_bits():
    # tokens, then pages, then query rows, each more than 2^31 elements apart
    s = Step("bf16", 4, 2, 64, 5, [1, 2], [10, 3], page=8, seed=17)
    want = s.run().clone()
    far = 1 << 30
    buf = torch.empty(4 * far + 1024, dtype=torch.bfloat16, device=DEV)
    kp = buf.as_strided((5, 2, 64), (far, 64, 1))
    vp = buf.as_strided((5, 2, 64), (far, 64, 1), 128)
    kp.copy_(s.kp), vp.copy_(s.vp)
    s.kp, s.vp = kp, vp
    s.run()
    assert torch.equal(s.out, want)
    pages = s.k_pages.shape[0]
    pool = torch.empty((pages - 1) * far + 4096, dtype=torch.bfloat16, device=DEV)
    kq = pool.as_strided((pages, 8, 2, 64), (far, 128, 64, 1))
    vq = pool.as_strided((pages, 8, 2, 64), (far, 128, 64, 1), 2048)
    kq.copy_(s.k_pages), vq.copy_(s.v_pages)
    s.k_pages, s.v_pages = kq, vq
    s.run()
    assert torch.equal(s.out, want)
    qq = buf.as_strided((3, 4, 64), (2 * far - 64, 64, 1), 512)
    qq.copy_(s.q)
    s.q = qq
    s.run()
    assert torch.equal(s.out, want)


def test_two_runs_another_stream_and_a_graph_agree():
    for rows in ([1, 1], [8] * 12):
        s = Step("bf16", 14, 2, 128, 2000, rows, [n + 30 for n in rows], seed=18)
        want, lse = s.run().clone(), s.lse.clone()
        s.out.zero_()
        assert torch.equal(s.run(), want) and torch.equal(s.lse, lse)
        a = s.args()
        nws = qmv.qmv_attn_workspace_size(a)
        ws = torch.empty(nws, dtype=torch.uint8, device=DEV)
        st = torch.cuda.Stream()
        s.out.zero_()
        st.wait_stream(torch.cuda.current_stream())
        qmv.qmv_attn(a, ws, nws, st)
        st.synchronize()
        assert torch.equal(s.out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            qmv.qmv_attn(a, ws, nws, st)
        for i in range(4):
            s.out.zero_()
            s.q.mul_(1.0 if i % 2 else -1.0)  # new inputs between the replays
            g.replay()
            got = s.out.clone()
            assert torch.equal(s.run(), got)
            assert torch.equal(got, want) == (i >= 2)  # the sign is back
            torch.cuda.synchronize()


def test_a_row_past_max_rows_is_nan_and_a_suffix_past_max_suffix_is_cut():
    s = Step("bf16", 4, 2, 64, 20, [3, 1], [12, 9], page=8, seed=19)
    a = s.args(max_suffix=7)
    a.max_rows = 2
    nws = qmv.qmv_attn_workspace_size(a)
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV)
    qmv.qmv_attn(a, ws, nws)
    assert bool(s.out[2].isnan().all()) and not bool(s.out[:2].isnan().any())
    s.suffix = [7, 7]
    want, _, _, _ = s.oracle()
    got = s.out.cpu().double().numpy()
    assert np.allclose(got[[0, 1, 3]], want[[0, 1, 3]], atol=0.03, rtol=0.02)


def test_wild_device_integers_stay_in_bounds():
    # row_start and suffix_len that make no sense: any finite result or NaN, but no fault and nothing outside out
    s = Step("bf16", 4, 2, 64, 20, [3, 1, 2], [12, 9, 4], page=8, seed=20)
    s.row_start.copy_(torch.tensor([-7, 900, 2, 1 << 30], dtype=torch.int32))
    s.suffix_len.copy_(torch.tensor([1 << 30, -3, 12], dtype=torch.int32))
    buf = torch.full((8, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    s.run(out=buf[1:7])
    torch.cuda.synchronize()
    assert bool((buf[0] == 5.0).all()) and bool((buf[7] == 5.0).all())

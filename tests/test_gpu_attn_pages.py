"""qmv_attn over a prefix in pages, where a key head has many rows: pages outside the pool in the first, a middle and the
last tile; and page lists of more pages than one workgroup stages."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_attn import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("rows,heads", [([8] * 9, 4), ([40, 3, 60], 2), ([1, 2], 4)])
def test_prefix_pages_outside_the_pool(rows, heads, page, dim):
    tokens = 700
    pages = -(-tokens // page)
    for bad in ([0], [pages // 2], [pages - 1], [0, pages // 2, pages - 1], list(range(pages))):
        say(f"attn prefix pages {bad} of {pages} outside the pool, dim {dim}, {sum(rows)} rows")
        s = Step("bf16", heads, 2, dim, tokens, rows, [n + 9 for n in rows], page=page, paged_prefix=True, seed=dim + page)
        # page 0, which the kernels copy in the place of one that is not there, is out of use and NaN
        taken = int((s.prefix_pages == 0).any() or (s.table == 0).any())
        if taken:
            free = [p for p in range(s.k_pages.shape[0]) if not bool((s.prefix_pages == p).any() or (s.table == p).any())][0]
            s.k_pages[free], s.v_pages[free] = s.k_pages[0].clone(), s.v_pages[0].clone()
            s.prefix_pages[s.prefix_pages == 0] = free
            s.table[s.table == 0] = free
        s.k_pages[0], s.v_pages[0] = float("nan"), float("inf")
        for i, b in enumerate(bad):
            s.prefix_pages[b] = (-1, 1 << 30, s.k_pages.shape[0], -(1 << 31))[i % 4]
        s.run()
        s.check()


@pytest.mark.parametrize("page,tokens", [(1, 2300), (1, 4097), (2, 5000), (8, 17001)])
@pytest.mark.parametrize("rows,heads", [([1], 2), ([3, 2], 4), ([8] * 9, 4)])
def test_more_prefix_pages_than_a_workgroup_stages(rows, heads, page, tokens):
    say(f"attn prefix of {tokens} tokens in pages of {page}, {sum(rows)} rows")
    s = Step("f16", heads, 1, 64, tokens, rows, rows, page=page, paged_prefix=True, seed=page)
    s.prefix_pages[tokens // page // 2] = -1
    s.run()
    s.check()


@pytest.mark.parametrize("page,tokens", [(1, 4500), (8, 17000)])
@pytest.mark.parametrize("seqs", [1, 70])
def test_more_suffix_pages_than_a_workgroup_stages(seqs, page, tokens):
    # many sequences: long key ranges
    suffix = [tokens] + [5 + i % 7 for i in range(seqs - 1)]
    say(f"attn suffix of {tokens} tokens in pages of {page}, {seqs} sequences")
    s = Step("bf16", 16, 16, 64, 33, [1] * seqs, suffix, page=page, seed=seqs)
    s.table[0, tokens // page - 3] = -1
    s.run()
    s.check()

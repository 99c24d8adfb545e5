"""Sizes past a launch's 2^32 work-items are refused on the host (fake pointers, never dereferenced)."""
import pytest

from block_quantized_weight_qmv_amd import qmv
from test_step_checks import _attn, _expect


def wide_batch(nseq, kv_heads):
    # a workgroup of 256 for each sequence and key head
    return _attn(nseq=nseq, rows=nseq, heads=kv_heads, kv_heads=kv_heads, head_dim=8, q_row=8 * kv_heads, q_head=8,
                 out_row=8 * kv_heads, out_head=8, page_row=8 * kv_heads, page_head=8, page_stride=128 * kv_heads,
                 max_rows=1, prefix_len=0, k_prefix=None, v_prefix=None, max_suffix=16, table_stride=1)


@pytest.mark.parametrize("nseq,kv_heads", [(1 << 17, 128), (1 << 20, 16)])
def test_attn_of_too_many_workgroups_is_refused(nseq, kv_heads):
    _expect(-6, qmv.qmv_attn_workspace_size, wide_batch(nseq, kv_heads))  # 2^24 workgroups
    assert qmv.qmv_attn_workspace_size(wide_batch(nseq - 1, kv_heads)) > 0

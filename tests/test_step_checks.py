"""qmv_embed, qmv_attn and qmv_verify without a GPU: every refusal, from the C ABI's checks (fake pointers, never
dereferenced) and from the binding's checks of tensors (stand-ins)."""
import ctypes

import pytest
import torch

from block_quantized_weight_qmv_amd import qmv

FAKE = 0x7F0000000000


def _expect(status, fn, *a, **k):
    with pytest.raises(qmv.QmvError) as e:
        fn(*a, **k)
    assert e.value.status == status, str(e.value)


def _w(fmt="q4_k", rows=8, cols=512):
    return qmv.qmv_create_weights(fmt, rows, cols, FAKE, qmv.qmv_packed_size(fmt, rows, cols))


def test_embed_refusals():
    w = _w()
    e = qmv.qmv_embed
    _expect(-3, e, w, FAKE, -1, FAKE, "f32")
    _expect(-1, e, w, None, 4, FAKE, "f32")
    _expect(-1, e, w, FAKE, 4, None, "f32")
    _expect(-6, e, w, FAKE, 4, FAKE, 7)
    _expect(-4, e, w, FAKE + 2, 4, FAKE, "f32")
    _expect(-4, e, w, FAKE, 4, FAKE + 8, "f16")
    _expect(-6, e, w, FAKE, 1 << 31, FAKE, "f16")
    bad = _w()
    bad.nbytes += 1
    _expect(-5, e, bad, FAKE, 4, FAKE, "f32")
    e(w, None, 0, None, "f32")  # nothing to look up


def _attn(**over):
    a = qmv.QmvAttnArgs()
    base = dict(dtype=2, head_dim=128, heads=28, kv_heads=4, nseq=2, max_rows=3, page_size=16, scale=0.1, rows=5,
                prefix_len=100, max_suffix=40, num_pages=9, table_stride=3, q_row=3584, q_head=128, out_row=3584,
                out_head=128, prefix_row=512, prefix_head=128, page_stride=8192, page_row=512, page_head=128, q=FAKE,
                k_prefix=FAKE, v_prefix=FAKE, k_pages=FAKE, v_pages=FAKE, block_table=FAKE, row_start=FAKE,
                suffix_len=FAKE, out=FAKE)
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    return a


def test_attn_arguments():
    size = qmv.qmv_attn_workspace_size
    size(_attn())
    assert qmv.lib().qmv_attn_workspace_size(None, ctypes.byref(ctypes.c_uint64())) == -1
    assert qmv.lib().qmv_attn_workspace_size(ctypes.byref(_attn()), None) == -1
    for status, over in [
            (-6, dict(dtype=0)), (-6, dict(dtype=3)), (-6, dict(head_dim=0)), (-6, dict(head_dim=100)),
            (-6, dict(head_dim=264)), (-3, dict(heads=27)), (-3, dict(kv_heads=0)), (-3, dict(rows=-1)),
            (-3, dict(nseq=0)), (-3, dict(nseq=-1)), (-3, dict(prefix_len=-1)), (-3, dict(max_suffix=-1)),
            (-3, dict(max_rows=0)), (-3, dict(page_size=24)), (-3, dict(page_size=0)), (-3, dict(page_size=1 << 17)),
            (-7, dict(scale=0.0)), (-7, dict(scale=-1.0)), (-7, dict(scale=float("nan"))),
            (-7, dict(scale=float("inf"))), (-1, dict(q=None)), (-1, dict(out=None)), (-1, dict(row_start=None)),
            (-1, dict(k_prefix=None)), (-1, dict(v_prefix=None)), (-1, dict(k_pages=None)), (-1, dict(v_pages=None)),
            (-1, dict(block_table=None)), (-1, dict(suffix_len=None)), (-5, dict(table_stride=2)),
            (-3, dict(q_row=3580)), (-3, dict(page_head=-8)), (-3, dict(prefix_row=1 << 40)),
            (-4, dict(q=FAKE + 8)), (-4, dict(out=FAKE + 2)), (-4, dict(k_pages=FAKE + 4)),
            (-4, dict(row_start=FAKE + 2)), (-4, dict(lse=FAKE + 1)), (-4, dict(tree_mask=FAKE + 4)),
            (-6, dict(tree_mask=FAKE, max_rows=65)), (-6, dict(rows=1 << 21)), (-6, dict(prefix_len=1 << 31)),
            (-6, dict(num_pages=1 << 31))]:
        _expect(status, size, _attn(**over))
    size(_attn(max_suffix=0, k_pages=None, v_pages=None, block_table=None, suffix_len=None, page_size=0))
    size(_attn(prefix_len=0, k_prefix=None, v_prefix=None))
    size(_attn(num_pages=0, k_pages=None, v_pages=None))  # an empty pool: every page number is outside it
    size(_attn(prefix_pages=FAKE, k_prefix=None, v_prefix=None))
    size(_attn(tree_mask=FAKE, max_rows=64))
    assert size(_attn(rows=0, q=None, out=None, row_start=None)) == 0
    qmv.qmv_attn(_attn(rows=0), None, 0, 0)  # nothing to do


def test_attn_workspace_refusals():
    a = _attn()
    n = qmv.qmv_attn_workspace_size(a)
    if n:
        _expect(-1, qmv.qmv_attn, a, None, 0, 0)
        _expect(-5, qmv.qmv_attn, a, FAKE, n - 1, 0)
    _expect(-4, qmv.qmv_attn, a, FAKE + 16, n, 0)


def _verify(**over):
    a = qmv.QmvVerifyArgs()
    base = dict(logits_dtype=0, nseq=2, max_rows=3, rows=5, vocab=1000, logits_row=1000, draft_row=1000, logits=FAKE,
                draft_probs=FAKE, tokens=FAKE, row_start=FAKE, temperature=FAKE, u_accept=FAKE, u_sample=FAKE,
                out_tokens=FAKE, accepted=FAKE)
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    return a


def test_verify_arguments():
    size = qmv.qmv_verify_workspace_size
    size(_verify())
    assert qmv.lib().qmv_verify_workspace_size(None, ctypes.byref(ctypes.c_uint64())) == -1
    assert qmv.lib().qmv_verify_workspace_size(ctypes.byref(_verify()), None) == -1
    for status, over in [
            (-6, dict(logits_dtype=3)), (-3, dict(rows=-1)), (-3, dict(nseq=-1)), (-3, dict(nseq=0)),
            (-3, dict(vocab=0)), (-3, dict(max_rows=0)), (-6, dict(vocab=(1 << 24) + 1, logits_row=1 << 25,
                                                                   draft_row=1 << 25)),
            (-6, dict(rows=65536)), (-6, dict(nseq=65536)), (-3, dict(logits_row=999)), (-3, dict(draft_row=999)),
            (-1, dict(logits=None)), (-1, dict(tokens=None)), (-1, dict(row_start=None)), (-1, dict(u_accept=None)),
            (-1, dict(u_sample=None)), (-1, dict(out_tokens=None)), (-1, dict(accepted=None)),
            (-4, dict(logits=FAKE + 2)), (-4, dict(draft_probs=FAKE + 2)), (-4, dict(tokens=FAKE + 2)),
            (-4, dict(accepted=FAKE + 1))]:
        _expect(status, size, _verify(**over))
    size(_verify(draft_probs=None, draft_row=0, temperature=None))
    size(_verify(logits_dtype=1, logits=FAKE + 2))
    assert size(_verify(rows=0, nseq=0, row_start=None)) == 0
    qmv.qmv_verify(_verify(rows=0, nseq=0), None, 0, 0)
    a = _verify()
    n = qmv.qmv_verify_workspace_size(a)
    if n:
        _expect(-1, qmv.qmv_verify, a, None, 0, 0)
        _expect(-5, qmv.qmv_verify, a, FAKE, n - 1, 0)
    _expect(-4, qmv.qmv_verify, a, FAKE + 16, n, 0)


class Dev:
    """Stand-in for a device tensor: what the binding's checks look at, on a meta tensor."""

    def __init__(self, t, device="cuda:0"):
        self._t, self.is_cuda, self.device = t, True, device
        self.dtype, self.shape = t.dtype, t.shape

    def __getattr__(self, name):
        return getattr(self._t, name)

    def data_ptr(self):
        return FAKE


def dev(*shape, dtype=torch.bfloat16):
    return Dev(torch.empty(*shape, dtype=dtype, device="meta"))


def test_binding_refuses_embed_tensors():
    w = _w()
    ids, out = dev(4, dtype=torch.int32), dev(4, 512, dtype=torch.float32)
    _expect(-2, qmv.qmv_embed, w, dev(4, dtype=torch.int64), 4, out, "f32", 1.0, 0)
    _expect(-5, qmv.qmv_embed, w, ids, 5, dev(5, 512, dtype=torch.float32), "f32", 1.0, 0)
    _expect(-5, qmv.qmv_embed, w, ids, 4, dev(3, 512, dtype=torch.float32), "f32", 1.0, 0)
    _expect(-2, qmv.qmv_embed, w, ids, 4, out, "bf16", 1.0, 0)
    _expect(-6, qmv.qmv_embed, w, torch.zeros(4, dtype=torch.int32), 4, out, "f32", 1.0, 0)


def _tensors(**over):
    i32 = torch.int32
    t = dict(q=dev(5, 28, 128), out=dev(5, 28, 128), row_start=dev(3, dtype=i32), k_prefix=dev(100, 4, 128),
             v_prefix=dev(100, 4, 128), k_pages=dev(9, 16, 4, 128), v_pages=dev(9, 16, 4, 128),
             block_table=dev(2, 3, dtype=i32), suffix_len=dev(2, dtype=i32))
    t.update(over)
    q, out, rs = t.pop("q"), t.pop("out"), t.pop("row_start")
    kw = dict(scale=0.1, max_suffix=40)
    kw.update(t)
    return (q, out, rs, 3), kw


def _create(**over):
    a, k = _tensors(**over)
    return qmv.qmv_create_attn(*a, **k)


def test_binding_checks_attn_tensors():
    a = _create()
    assert (a.rows, a.heads, a.kv_heads, a.head_dim, a.nseq, a.prefix_len, a.num_pages, a.page_size) == \
        (5, 28, 4, 128, 2, 100, 9, 16)
    assert (a.q_row, a.q_head, a.prefix_row, a.page_stride, a.page_row, a.page_head, a.table_stride) == \
        (3584, 128, 512, 8192, 512, 128, 3)
    i32 = torch.int32
    for status, over in [
            (-6, dict(q=dev(5, 28, 128, dtype=torch.float32))), (-3, dict(q=dev(5, 3584))),
            (-2, dict(out=dev(5, 28, 128, dtype=torch.float16))), (-3, dict(out=dev(4, 28, 128))),
            (-2, dict(row_start=dev(3, dtype=torch.int64))), (-2, dict(k_prefix=dev(100, 4, 128, dtype=torch.float16))),
            (-3, dict(k_prefix=dev(99, 4, 128))), (-3, dict(k_prefix=dev(100, 4, 64), v_prefix=dev(100, 4, 64))),
            (-3, dict(k_pages=dev(9, 16, 2, 128), v_pages=dev(9, 16, 2, 128))),
            (-1, dict(v_prefix=None)), (-1, dict(v_pages=None)), (-1, dict(k_pages=None, v_pages=None)),
            (-1, dict(block_table=None)), (-5, dict(block_table=dev(1, 3, dtype=i32))),
            (-5, dict(block_table=dev(2, 2, dtype=i32))), (-1, dict(suffix_len=None)),
            (-5, dict(suffix_len=dev(1, dtype=i32))), (-5, dict(tree_mask=dev(4, dtype=torch.int64))),
            (-2, dict(tree_mask=dev(5, dtype=i32))), (-5, dict(lse=dev(5, 27, dtype=torch.float32))),
            (-5, dict(prefix_len=101)), (-3, dict(k_prefix=None, v_prefix=None, prefix_pages=dev(7, dtype=i32))),
            (-3, dict(prefix_pages=dev(7, dtype=i32), prefix_len=100)),
            (-5, dict(k_prefix=None, v_prefix=None, prefix_pages=dev(6, dtype=i32), prefix_len=100)),
            (-6, dict(k_pages=Dev(torch.empty(9, 16, 4, 128, dtype=torch.bfloat16, device="meta"), "cuda:1"))),
            (-6, dict(q=Dev(torch.empty(5, 28, 256, dtype=torch.bfloat16, device="meta")[..., ::2]))),
            (-3, dict(q=Dev(torch.empty(5, 28, 129, dtype=torch.bfloat16, device="meta")[..., :128]))),
            (-6, dict(q=torch.zeros(5, 28, 128, dtype=torch.bfloat16)))]:
        _expect(status, _create, **over)
    a = _create(k_prefix=None, v_prefix=None, prefix_pages=dev(7, dtype=i32), prefix_len=100)
    assert a.prefix_len == 100
    kv = torch.empty(100, 2, 4, 128, dtype=torch.bfloat16, device="meta")  # k and v of a token side by side
    a = _create(k_prefix=Dev(kv[:, 0]), v_prefix=Dev(kv[:, 1]))
    assert a.prefix_row == 1024
    _expect(-3, _create, k_prefix=Dev(kv[:, 0]))


def test_binding_checks_verify_tensors():
    i32, f32 = torch.int32, torch.float32

    def create(**over):
        t = dict(logits=dev(5, 1000, dtype=f32), tokens=dev(5, dtype=i32), row_start=dev(3, dtype=i32),
                 u_accept=dev(5, dtype=f32), u_sample=dev(2, dtype=f32), out_tokens=dev(5, dtype=i32),
                 accepted=dev(2, dtype=i32), draft_probs=dev(5, 1000, dtype=f32), temperature=dev(2, dtype=f32))
        t.update(over)
        return qmv.qmv_create_verify(max_rows=3, **t)

    a = create()
    assert (a.rows, a.vocab, a.nseq, a.logits_row, a.draft_row, a.logits_dtype) == (5, 1000, 2, 1000, 1000, 0)
    for status, over in [
            (-6, dict(logits=dev(5, 1000, dtype=torch.float64))), (-3, dict(logits=dev(5000, dtype=f32))),
            (-5, dict(tokens=dev(4, dtype=i32))), (-2, dict(tokens=dev(5, dtype=torch.int64))),
            (-5, dict(u_sample=dev(1, dtype=f32))), (-5, dict(accepted=dev(1, dtype=i32))),
            (-2, dict(draft_probs=dev(5, 1000))), (-3, dict(draft_probs=dev(4, 1000, dtype=f32))),
            (-2, dict(temperature=dev(2))), (-1, dict(u_accept=None)),
            (-6, dict(u_accept=torch.zeros(5)))]:
        _expect(status, create, **over)
    assert create(draft_probs=None, temperature=None).draft_probs is None
    a = create(logits=Dev(torch.empty(5, 1024, dtype=torch.float16, device="meta")[:, :1000]))
    assert a.logits_row == 1024 and a.logits_dtype == 1

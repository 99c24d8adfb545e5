"""Tensors of one call on different GPUs are refused by the binding (stand-ins, never dereferenced)."""
import torch

from block_quantized_weight_qmv_amd import qmv
from test_step_checks import Dev, _create, _expect, _w, dev


def other(*shape, dtype):
    return Dev(torch.empty(*shape, dtype=dtype, device="meta"), "cuda:1")


def test_embed_ids_and_out():
    out = dev(4, 512, dtype=torch.float32)
    _expect(-6, qmv.qmv_embed, _w(), other(4, dtype=torch.int32), 4, out, "f32", 1.0, 0)


def test_attn_workspace():
    a = _create()
    n = qmv.qmv_attn_workspace_size(a)
    assert n > 0
    _expect(-6, qmv.qmv_attn, a, other(n, dtype=torch.uint8), n, 0)


def test_verify_workspace():
    i32, f32 = torch.int32, torch.float32
    a = qmv.qmv_create_verify(dev(5, 1000, dtype=f32), dev(5, dtype=i32), dev(3, dtype=i32), 3, dev(5, dtype=f32),
                              dev(2, dtype=f32), dev(5, dtype=i32), dev(2, dtype=i32))
    n = qmv.qmv_verify_workspace_size(a)
    assert n > 0
    _expect(-6, qmv.qmv_verify, a, other(n, dtype=torch.uint8), n, 0)

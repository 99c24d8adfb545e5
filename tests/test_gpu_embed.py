"""qmv_embed against the float64 oracle: every format, layout and output type.

The weight is its fp32 value (bit-exact in qmv_dequant), times the scale rounded once to fp32 (2^-24 relative), then
rounded once to the output type (half its epsilon; fp16 below its normal range: half of 2^-24 absolute)."""
import numpy as np
import pytest
import torch

import oracle
from oracle.step import embed64
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, Weights, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CASES = [("q8_0", "blocks"), ("q4_k", "blocks"), ("q4_k", "planes"), ("q5_k", "blocks"), ("q5_k", "planes"),
         ("q6_k", "blocks"), ("q6_k", "planes"), ("int4_g128", "blocks")]


def _desc(w, layout):
    if layout == "blocks":
        return w.desc
    buf = torch.empty(qmv.qmv_planes_size(w.fmt, w.rows, w.cols), dtype=torch.uint8, device=DEV)
    return qmv.qmv_repack_planes(w.desc, buf)


@pytest.mark.parametrize("out_dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,blocks,n,scale", [(1, 1, 1, 1.0), (37, 3, 5, 0.5), (130, 14, 300, 59.866),
                                                 (5, 1, 1000, -3.0), (3, 33, 7, 1.0)])
@pytest.mark.parametrize("fmt,layout", CASES)
def test_embed(fmt, layout, rows, blocks, n, scale, out_dtype):
    cols = blocks * oracle.QK[fmt]
    say(f"embed {fmt} {layout} {rows}x{cols} n {n} {out_dtype}")
    w = Weights(fmt, rows, cols, seed=900 + rows)
    ids = np.random.default_rng(n).integers(-2, rows + 2, n).astype(np.int32)
    ids[0] = rows - 1
    ids[-1] = 0 if n > 1 else rows - 1
    if n > 5:
        ids[1:5] = [-1, rows, 2**31 - 1, -2**31]
    out = torch.full((n + 1, cols), 7.0, dtype=TYPES[out_dtype], device=DEV)
    qmv.qmv_embed(_desc(w, layout), torch.from_numpy(ids).to(DEV), n, out, out_dtype, scale)
    assert bool((out[n] == 7.0).all())  # nothing past the last row
    got = out[:n].cpu().double().numpy()
    want = embed64(oracle.dequant32(fmt, w.oracle_bytes(), rows, cols), ids, scale)
    tol = np.abs(want) * 2.0**-24
    if out_dtype != "f32":
        tol += np.abs(want) * torch.finfo(TYPES[out_dtype]).eps / 2 * (1 + 2.0**-20)
    if out_dtype == "f16":
        tol += 2.0**-25
        over = np.abs(want) >= 65520
        assert np.array_equal(np.isinf(got), over)
        got, want = np.where(over, 0, got), np.where(over, 0, want)
    assert np.all(np.abs(got - want) <= tol)


def test_embed_scale_one_is_dequant_bit_for_bit():
    w = Weights("q4_k", 64, 512, seed=5)
    for dt in TYPES:
        dense = torch.empty(64, 512, dtype=TYPES[dt], device=DEV)
        qmv.qmv_dequant(w.desc, dense, dt)
        ids = torch.randperm(64, device=DEV).to(torch.int32)
        out = torch.empty_like(dense)
        qmv.qmv_embed(w.desc, ids, 64, out, dt)
        assert torch.equal(out, dense[ids.long()])


def test_embed_far_rows():
    # a table of more than 2^32 bytes: the last row's blocks lie past 32-bit offsets
    fmt, cols = "q8_0", 32 * 1024
    rows = (1 << 32) // (cols // 32 * 34) + 3
    table = torch.zeros(qmv.qmv_packed_size(fmt, rows, cols), dtype=torch.uint8, device=DEV)
    w = Weights(fmt, 2, cols, seed=6)
    per = cols // 32 * 34
    table[:per] = w.dev[:per]
    table[-per:] = w.dev[per:]
    big = qmv.qmv_create_weights(fmt, rows, cols, table)
    out = torch.empty(2, cols, dtype=torch.float32, device=DEV)
    qmv.qmv_embed(big, torch.tensor([0, rows - 1], dtype=torch.int32, device=DEV), 2, out, "f32")
    assert np.array_equal(out.cpu().numpy(), oracle.dequant32(fmt, w.oracle_bytes(), 2, cols))


def test_embed_other_stream_and_graph():
    w = Weights("q6_k", 50, 768, seed=7)
    ids = torch.arange(49, -1, -1, dtype=torch.int32, device=DEV)
    want = torch.empty(50, 768, dtype=torch.bfloat16, device=DEV)
    qmv.qmv_embed(w.desc, ids, 50, want, "bf16", 2.0)
    torch.cuda.synchronize()
    s, out = torch.cuda.Stream(), torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    qmv.qmv_embed(w.desc, ids, 50, out, "bf16", 2.0, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qmv.qmv_embed(w.desc, ids, 50, out, "bf16", 2.0, stream=s)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

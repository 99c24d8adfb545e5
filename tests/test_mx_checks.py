"""qmv_quantize, qmv_mx4_gemm, qmv_norm and the mxfp4 format without a GPU: refusals of the C ABI (fake pointers, never
dereferenced) and of the binding (stand-ins)."""
import ctypes

import pytest
import torch

from block_quantized_weight_qmv_amd import qmv
from test_step_checks import FAKE, Dev, _expect, dev
from test_step_devices import other

F32, F16, BF16, I32 = torch.float32, torch.float16, torch.bfloat16, torch.int32


def _w(rows=8, cols=64, fmt="mxfp4", at=FAKE):
    return qmv.qmv_create_weights(fmt, rows, cols, at, qmv.qmv_packed_size(fmt, rows, cols))


def test_descriptor():
    w = _w()
    assert (w.fmt, w.nbytes, w.scales_offset) == (8, 8 * 2 * 17, 256)
    _expect(-3, qmv.qmv_create_weights, "mxfp4", 8, 48, FAKE, 8 * 17)
    _expect(-5, qmv.qmv_create_weights, "mxfp4", 8, 64, FAKE, 8 * 2 * 17 + 1)
    _expect(-4, qmv.qmv_create_weights, "mxfp4", 8, 64, FAKE + 8, 8 * 2 * 17)
    _expect(-6, qmv.qmv_create_weights_planes, "mxfp4", 8, 256, FAKE, 100)
    assert qmv.qmv_planes_size("mxfp4", 8, 256) == 0
    _expect(-6, qmv.qmv_repack_planes, w, FAKE + (1 << 20), 1 << 20)
    w.scales_offset = 0
    _expect(-2, qmv.qmv_dequant, w, FAKE, "f32")
    _expect(-6, qmv.qmv_gemv, "mxfp4", _w(4, 65536 + 32), FAKE, "f32", FAKE, 4, 65536 + 32, 1)
    _expect(-6, qmv.qmv_gemv_swiglu, "mxfp4", _w(4, 4128), _w(4, 4128), FAKE, "f32", FAKE, 4, 4128, 1)


def _quantize(w, x, dtype, row):
    return qmv.lib().qmv_quantize(None if w is None else ctypes.byref(w), x, dtype, row, None)


def test_quantize_refusals():
    x = FAKE + (1 << 20)
    assert _quantize(None, x, 0, 64) == -1
    assert _quantize(_w(), None, 0, 64) == -1
    assert _quantize(_w(fmt="int4_g128", cols=128), x, 0, 128) == -6
    assert _quantize(_w(), x, 3, 64) == -6
    assert _quantize(_w(), x + 8, 0, 64) == -4
    for row in (63, 56, 68, -64, 1 << 32):
        assert _quantize(_w(), x, 0, row) == -3, row
    assert _quantize(_w(), FAKE + 256, 0, 64) == -3  # on the scales
    assert _quantize(_w(), FAKE - 8 * 64 * 2 + 16, 1, 64) == -3
    bad = _w()
    bad.nbytes -= 1
    assert _quantize(bad, x, 0, 64) == -5


def test_quantize_binding():
    q = qmv.qmv_quantize
    _expect(-6, q, _w(), dev(8, 64, dtype=torch.float64), 0)
    _expect(-6, q, _w(), torch.zeros(8, 64), 0)
    _expect(-3, q, _w(), dev(8, 96), 0)
    _expect(-3, q, _w(), dev(7, 64), 0)
    _expect(-3, q, _w(), dev(8 * 64), 0)
    _expect(-6, q, _w(), Dev(torch.empty(8, 128, dtype=BF16, device="meta")[:, ::2]), 0)
    _expect(-3, q, _w(), Dev(torch.empty(8, 68, dtype=BF16, device="meta")[:, :64]), 0)
    w = _w()
    w.owner = other(8 * 34, dtype=torch.uint8)
    _expect(-6, q, w, dev(8, 64), 0)


Y, XAT = FAKE + (1 << 30), FAKE + (1 << 28)


def _mx4(W=None, X=None, **over):
    a = qmv.QmvMx4Args()
    a.keep = (W or _w(96, 64), X or _w(10, 64, at=XAT))
    base = dict(y_dtype=2, epilogue=0, experts=0, rows=10, y_row=96, y=Y)
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    a.W, a.X = ctypes.pointer(a.keep[0]), ctypes.pointer(a.keep[1])
    return a


def _gemm(a):
    return qmv.lib().qmv_mx4_gemm(ctypes.byref(a), None)


def test_mx4_gemm_refusals():
    assert qmv.lib().qmv_mx4_gemm(None, None) == -1
    grouped = dict(experts=3, expert_start=FAKE, y_row=32)
    for status, over in [
            (-6, dict(y_dtype=3)), (-6, dict(epilogue=2)), (-3, dict(rows=-1)), (-3, dict(experts=-1)),
            (-6, dict(rows=(1 << 22) + 1)), (-6, dict(experts=(1 << 16) + 1)), (-1, dict(y=None)),
            (-3, dict(y_row=95)), (-3, dict(y_row=1 << 32)), (-4, dict(y=Y + 1)), (-4, dict(y=Y + 2, y_dtype=0)),
            (-1, dict(experts=3, y_row=32)), (-3, dict(expert_start=FAKE)), (-3, dict(grouped, experts=5)),
            (-3, dict(grouped, epilogue=1, experts=32)), (-4, dict(grouped, expert_start=FAKE + 2)),
            (-4, dict(x_index=FAKE + 1)), (-3, dict(rows=11)), (-3, dict(y=XAT + 64)), (-3, dict(y=FAKE + 96 * 34 - 2)),
            (-3, dict(X=_w(10, 96, at=XAT))), (-2, dict(X=_w(10, 128, "int4_g128", XAT))),
            (-2, dict(W=_w(96, 64, "q8_0"))), (-3, dict(W=_w(95, 64), epilogue=1, y_row=47))]:
        assert _gemm(_mx4(**over)) == status, over
    a = _mx4()
    a.W = None
    assert _gemm(a) == -1
    a = _mx4()
    a.keep[1].nbytes += 1
    assert _gemm(a) == -5
    # (too many outputs; more bytes of codes than 32 bits count)
    assert _gemm(_mx4(W=_w((1 << 27) + 64, 64), y_row=(1 << 27) + 64, y=FAKE + (1 << 43))) == -6
    assert _gemm(_mx4(W=_w(1 << 21, 8192), X=_w(10, 8192, at=FAKE + (1 << 42)), y_row=1 << 21, y=FAKE + (1 << 43))) == -6
    assert _gemm(_mx4(W=_w(96, 8192), X=_w(1 << 21, 8192, at=FAKE + (1 << 42)), x_index=FAKE, y=FAKE + (1 << 43))) == -6
    assert _gemm(_mx4(W=_w((1 << 31) - 1, 32), X=_w(1 << 22, 32, at=FAKE + (1 << 42)), rows=1 << 22,
                      y_row=(1 << 31) - 1, y=FAKE + (1 << 43))) == -6
    a = _mx4(rows=0, y=None)
    a.W = None
    assert _gemm(a) == 0  # nothing to do


def test_mx4_binding():
    def create(W=None, X=None, y=None, **k):
        return qmv.qmv_create_mx4(W or _w(96, 64), X or _w(10, 64, at=XAT), dev(10, 96) if y is None else y, **k)

    a = create()
    assert (a.experts, a.rows, a.y_row, a.y_dtype, a.epilogue) == (0, 10, 96, 2, 0)
    a = create(y=dev(20, 16, dtype=F16), swiglu=True, expert_start=dev(4, dtype=I32), x_index=dev(20, dtype=I32))
    assert (a.experts, a.rows, a.y_row, a.y_dtype, a.epilogue) == (3, 20, 16, 1, 1)
    a = create(y=Dev(torch.empty(10, 128, dtype=F32, device="meta")[:, :96]))
    assert (a.y_row, a.y_dtype) == (128, 0)
    idx = dev(10, dtype=I32)
    for status, k in [
            (-6, dict(y=dev(10, 96, dtype=torch.int32))), (-6, dict(y=torch.zeros(10, 96))), (-3, dict(y=dev(960))),
            (-3, dict(y=dev(10, 95))), (-3, dict(swiglu=True)), (-3, dict(expert_start=dev(4, dtype=I32))),
            (-2, dict(x_index=dev(10, dtype=torch.int64))), (-5, dict(x_index=dev(9, dtype=I32))),
            (-5, dict(expert_start=dev(1, dtype=I32))), (-6, dict(x_index=torch.zeros(10, dtype=I32))),
            (-6, dict(x_index=other(10, dtype=I32))), (-6, dict(y=other(10, 96, dtype=BF16), x_index=idx)),
            (-6, dict(y=Dev(torch.empty(10, 192, dtype=BF16, device="meta")[:, ::2])))]:
        _expect(status, create, **k)
    _expect(-3, qmv.qmv_mx4_gemm, create(y=Dev(torch.empty(1, 96, dtype=BF16, device="meta").expand(10, 96))), 0)


def _norm(**over):
    a = qmv.QmvNormArgs()
    base = dict(dtype=2, weight_dtype=2, y_dtype=2, pre=1, post=2, eps=1e-6, scale=0.5, rows=4, cols=100,
                residual_row=100, block_row=100, sum_row=100, y_row=100, gate_row=0, residual=FAKE, block=FAKE + 1000,
                gate=FAKE + 2000, pre_weight=FAKE, pre_bias=FAKE, post_weight=FAKE, post_bias=FAKE, sum=FAKE + 3000,
                y=FAKE + 4000)
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    return a


def _call(a):
    return qmv.lib().qmv_norm(ctypes.byref(a), None)


def test_norm_refusals():
    assert qmv.lib().qmv_norm(None, None) == -1
    nan, inf = float("nan"), float("inf")
    for status, over in [
            (-6, dict(dtype=3)), (-6, dict(weight_dtype=-1)), (-6, dict(y_dtype=7)), (-6, dict(pre=3)),
            (-6, dict(post=-1)), (-3, dict(rows=-1)), (-3, dict(cols=0)), (-6, dict(cols=32769)),
            (-6, dict(rows=1 << 31)), (-7, dict(eps=-1.0)), (-7, dict(eps=nan)), (-7, dict(eps=inf)),
            (-7, dict(scale=nan)), (-7, dict(scale=-inf)), (-1, dict(residual=None)), (-1, dict(sum=None, y=None)),
            (-3, dict(block=None)), (-3, dict(block=None, gate=None)), (-3, dict(block=None, post=0)),
            (-3, dict(post=0)), (-3, dict(pre=0)), (-3, dict(y=None)), (-3, dict(residual_row=99)),
            (-3, dict(block_row=0)), (-3, dict(gate_row=99)), (-3, dict(sum_row=1 << 32)), (-3, dict(y_row=-100)),
            (-4, dict(residual=FAKE + 1)), (-4, dict(y=FAKE + 4001)), (-4, dict(y=FAKE + 4002, y_dtype=0)),
            (-4, dict(pre_weight=FAKE + 1)), (-4, dict(post_bias=FAKE + 2, weight_dtype=0)),
            (-3, dict(sum=FAKE + 2)), (-3, dict(y=FAKE + 1000, y_dtype=0)), (-3, dict(y=FAKE + 3400)),
            (-3, dict(y=FAKE + 1000, y_row=104)), (-3, dict(y=FAKE + 3000))]:
        assert _call(_norm(**over)) == status, over
    for side in (2, 198, 202, 398):  # columns of one buffer that meet
        far = dict(residual_row=200, sum_row=200, block=FAKE + 9000, y=FAKE + 20000)
        assert _call(_norm(sum=FAKE + side, **far)) == -3, side
    assert _call(_norm(rows=0, residual=None, y=None, sum=None)) == 0  # nothing to do


def test_norm_binding():
    def create(residual=None, y=None, **k):
        return qmv.qmv_create_norm(dev(4, 100) if residual is None else residual, y, **k)

    x, v = dev(4, 100), dev(100)
    a = create(y=dev(4, 100, dtype=F32), pre="rms", pre_weight=v, block=x, post="layer", gate=x, sum_out=x, scale=0.5)
    assert (a.dtype, a.weight_dtype, a.y_dtype, a.pre, a.post, a.rows, a.cols, a.gate_row) == (2, 2, 0, 1, 2, 4, 100, 100)
    a = create(y=x, block=Dev(torch.empty(4, 128, dtype=BF16, device="meta")[:, :100]), gate=v)
    assert (a.block_row, a.gate_row, a.pre) == (128, 0, 0)
    for status, k in [
            (-6, dict(residual=dev(4, 100, dtype=torch.float64))), (-3, dict(residual=dev(400))),
            (-2, dict(block=dev(4, 100, dtype=F32))), (-3, dict(block=dev(3, 100))), (-3, dict(sum_out=dev(4, 99))),
            (-6, dict(y=dev(4, 100, dtype=torch.int8))), (-3, dict(y=dev(4, 96))), (-2, dict(gate=dev(100, dtype=F16))),
            (-3, dict(gate=dev(99))), (-3, dict(gate=dev(1, 4, 100))), (-6, dict(pre="rms_norm")),
            (-6, dict(pre="rms", pre_weight=dev(100, dtype=torch.int32))),
            (-6, dict(pre="rms", pre_weight=v, pre_bias=dev(100, dtype=F32))), (-5, dict(pre="rms", pre_weight=dev(99))),
            (-6, dict(block=other(4, 100, dtype=BF16))), (-6, dict(residual=torch.zeros(4, 100)))]:
        _expect(status, create, **k)
    with pytest.raises(qmv.QmvError):
        qmv.qmv_norm(create(), 0)  # neither sum nor y


def test_gemm_sizes_past_32_bits():
    """Rows of X and columns that would be others when cut to 32 bits."""
    far = FAKE + (1 << 43)
    assert _gemm(_mx4(W=_w(96, 32), X=_w((1 << 32) + 5, 32, at=FAKE + (1 << 42)), x_index=FAKE, y=far)) == -6
    assert _gemm(_mx4(W=_w(96, (1 << 32) + 32), X=_w(10, (1 << 32) + 32, at=FAKE + (1 << 42)), x_index=FAKE, y=far)) == -6
    assert _gemm(_mx4(W=_w(2, 1 << 31), X=_w(2, 1 << 31, at=FAKE + (1 << 42)), rows=2, y=far)) == -6

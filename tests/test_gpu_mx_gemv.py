"""MXFP4 as a format of the decode GEMV: exact activations in fp32, fp16 and bf16, one and several rows, rows of every
length within and past a wave's slice, the paired and the SwiGLU launch.

Decoded weights times activations are exact in fp32 up to one rounding a product; a sum of K of them is off by at most
K 2^-24 of sum |w x| in any order, twice that with the products' roundings and the scales' (powers of two: exact)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import mx
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Mx:
    """Random codes with powers 2^lo .. 2^hi, on the GPU and in 64 bits."""

    def __init__(self, rows, cols, seed, lo=-9, hi=-3):
        r = np.random.default_rng(seed)
        self.rows, self.cols = rows, cols
        self.bytes = mx.mx4_pack(r.integers(127 + lo, 128 + hi, (rows, cols // 32)), r.integers(0, 16, (rows, cols)))
        self.dev = torch.from_numpy(self.bytes).to(DEV)
        self.desc = qmv.qmv_create_weights("mxfp4", rows, cols, self.dev)
        self.w = mx.mx4_decode64(self.bytes, rows, cols)


def x_of(batch, cols, dt, seed, scale=1.0):
    return (torch.randn(batch, cols, generator=torch.Generator().manual_seed(seed)) * scale).to(TYPES[dt]).to(DEV)


def gemv(m, x, dt):
    y = torch.full((len(x) + 1, m.rows), 7.0, device=DEV)
    qmv.qmv_gemv("mxfp4", m.desc, x, dt, y, m.rows, m.cols, len(x))
    assert bool((y[-1] == 7.0).all())
    return y[:-1]


def close(y, x, w):
    x = x.cpu().double().numpy()
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    assert np.all(np.abs(y.cpu().double().numpy() - want) <= 2 * w.shape[1] * 2.0**-24 * mag)


SHAPES = [(1, 32), (5, 96), (67, 3584), (33, 4096), (130, 4128), (9, 18944), (4, 65536), (700, 64), (19, 8224)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gemv(rows, cols, dt):
    m = Mx(rows, cols, rows + cols)
    for batch in (1, 2, 3, 4, 7, 16, 33):
        say(f"gemv {rows}x{cols} {dt} batch {batch}")
        x = x_of(batch, cols, dt, batch)
        y = gemv(m, x, dt)
        close(y, x, m.w)
        one = torch.cat([gemv(m, x[b:b + 1].clone(), dt) for b in range(batch)])
        if batch < (5 if cols <= 4096 else 3) or dt == "f32":
            assert torch.equal(one, y)  # rows of a batch equal the calls of one row, up to where the matrix cores begin


@pytest.mark.parametrize("scale,lo,hi", [(1e-30, -20, -10), (1e30, -40, -30), (1.0, -127, -120), (1e-3, 100, 110),
                                         (1e10, -60, 60)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gemv_far_powers(dt, scale, lo, hi):
    m = Mx(40, 1024, 3, lo, hi)
    for batch in (3, 9):
        x = x_of(batch, 1024, dt, 1, scale)
        y = gemv(m, x, dt).cpu().double().numpy()
        xd = x.cpu().double().numpy()
        want, mag = xd @ m.w.T, np.abs(xd) @ np.abs(m.w).T
        # (products and sums below fp32's normal range may be flushed: 2^-126 each)
        assert np.all(np.abs(y - want) <= 2 * 1024 * 2.0**-24 * mag + 1024 * (2.0**-149 if batch < 5 else 2.0**-126))


def test_a_nan_block_makes_its_row_nan():
    m = Mx(6, 256, 2)
    m.dev[6 * 128 + 8 * 3 + 5] = 255
    for dt in TYPES:
        for batch in (1, 2, 6):
            y = gemv(m, x_of(batch, 256, dt, 5), dt).cpu()
            assert torch.isnan(y[:, 3]).all() and not torch.isnan(y[:, [0, 1, 2, 4, 5]]).any()


@pytest.mark.parametrize("dt", list(TYPES))
def test_pairs_and_swiglu(dt):
    a, b = Mx(130, 2592, 7), Mx(130, 2592, 8)
    for batch in (1, 3):
        x = x_of(batch, 2592, dt, 9)
        ya, yb = torch.empty(batch, 130, device=DEV), torch.empty(batch, 130, device=DEV)
        qmv.qmv_gemv_multi("mxfp4", dt, batch, [(a.desc, x, ya), (b.desc, x, yb)])
        close(ya, x, a.w)
        close(yb, x, b.w)
        h = torch.empty(batch, 130, device=DEV)
        qmv.qmv_gemv_swiglu("mxfp4", a.desc, b.desc, x, dt, h, 130, 2592, batch)
        xd = x.cpu().double().numpy()
        want = oracle.silu64(xd @ a.w.T) * (xd @ b.w.T)
        assert np.all(oracle.normwise_rel_err(h.cpu().numpy(), want) <= 2e-3)


def test_several_matrices_and_no_workspace():
    ms = [Mx(67, 1024, 1), Mx(5, 4096, 2), Mx(130, 8192, 3)]
    items = []
    for m in ms:
        x = x_of(2, m.cols, "f16", m.rows)
        items.append((m.desc, x, torch.empty(2, m.rows, device=DEV)))
    assert qmv.qmv_workspace_size("mxfp4", "f16", 2, items) == 0
    qmv.qmv_gemv_multi_ws("mxfp4", "f16", 2, items, None, 0)
    for m, (_, x, y) in zip(ms, items):
        close(y, x, m.w)
    y = torch.empty(2, 67, device=DEV)
    qmv.qmv_gemv_noalloc("mxfp4", ms[0].desc, items[0][1], "f16", y, 67, 1024, 2)
    assert torch.equal(y, items[0][2])


def test_fp16_rows_of_every_size_on_the_matrix_cores():
    """Numbers of all of fp16's magnitudes, its subnormals among them: each is the sum of two bf16 numbers."""
    bits = torch.arange(65536, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.float16)
    x = x[torch.isfinite(x)].view(8, -1)[:, :7936].contiguous().to(DEV)
    m = Mx(33, 7936, 5)
    close(gemv(m, x, "f16"), x, m.w)
    one = torch.eye(16, 256, dtype=torch.float16, device=DEV) * 3.140625  # products stand alone: exact
    m = Mx(70, 256, 6)
    assert np.array_equal(gemv(m, one, "f16").cpu().double().numpy(), 3.140625 * m.w[:, :16].T)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("cols", [256, 4128])
def test_infinities_and_nan_of_activations(cols, dt):
    """An infinite activation makes its row's outputs infinite (NaN where the weight is zero), a NaN its row NaN."""
    m = Mx(40, cols, 4)
    column = m.w[:, 100]
    assert (column == 0).any() and (column > 0).any() and (column < 0).any()
    for batch in (1, 6, 18):
        say(f"gemv infinities 40x{cols} {dt} batch {batch}")
        x = x_of(batch, cols, dt, 6)
        x[0, 100] = float("inf")
        if batch > 1:
            x[2, 100], x[5, 100] = float("-inf"), float("nan")
        y = gemv(m, x, dt).cpu().double().numpy()
        with np.errstate(invalid="ignore"):
            for row, v in ((0, np.inf), (2, -np.inf))[:batch]:
                np.testing.assert_array_equal(y[row], v * column)
        if batch > 1:
            assert np.isnan(y[5]).all() and np.isfinite(y[[1, 3, 4]]).all()

"""qmv_quantize and qmv_dequant of MXFP4 on the GPU against the 64-bit definition: codes, powers and values are exact."""
import numpy as np
import pytest
import torch

from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say
from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def quantized(x):
    """x on the GPU to MXFP4: (descriptor, bytes on the host), with a guard behind the bytes."""
    rows, cols = x.shape
    n = qmv.qmv_packed_size("mxfp4", rows, cols)
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    w = qmv.qmv_create_weights("mxfp4", rows, cols, buf[:n])
    qmv.qmv_quantize(w, x)
    host = buf.cpu().numpy()
    assert (host[n:] == 0xA5).all()
    return w, host[:n]


def check(x):
    rows, cols = x.shape
    _, got = quantized(x)
    p, code = mx.mx4_encode64(x.cpu().double().numpy())
    gp, gc = mx.mx4_unpack(got, rows, cols)
    assert np.array_equal(gp, p)
    assert np.array_equal(gc, code)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 3584), (3, 96), (77, 2880), (256, 64), (5, 18944), (1000, 32)])
def test_quantize(rows, cols, dt):
    say(f"quantize {rows}x{cols} {dt}")
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)
    check(x.to(TYPES[dt]).to(DEV))


@pytest.mark.parametrize("dt", list(TYPES))
def test_quantize_ties_signs_and_extremes(dt):
    t = TYPES[dt]
    f = torch.finfo(t)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0])
    both = torch.cat([ties, -ties])
    rows = [both.clone() for _ in range(6)]
    near = both.to(t)
    up = torch.where(near != 0, (near.double() * (1 + 2 * f.eps)), 0.0).to(t).float()
    down = torch.where(near != 0, (near.double() * (1 - f.eps)), 0.0).to(t).float()
    rows += [up, down]
    x = torch.stack(rows)
    powers = torch.tensor([1.0, 2.0**-10, 2.0**10, 2.0**12, 2.0**-6, 2.0**-13, 1.0, 1.0])[:, None]
    x = (x * powers).to(t)
    special = torch.zeros(7, 32, dtype=t)
    special[0] = f.max
    special[1] = f.tiny
    special[2, 5] = f.smallest_normal * f.eps  # the smallest subnormal alone
    special[3] = -f.max
    special[3, 1:] = f.tiny
    special[4] = torch.linspace(0, 1, 32).to(t) * f.smallest_normal
    special[5, 0] = -0.0
    special[6, 31] = f.smallest_normal * 3
    check(torch.cat([x, special]).to(DEV))


def test_quantize_far_powers():
    e = torch.arange(-149, 128).float()
    x = torch.randn(len(e), 32, generator=torch.Generator().manual_seed(3)).clamp(-1.99, 1.99)
    check(torch.ldexp(x.double(), e[:, None].double()).float().to(DEV))


@pytest.mark.parametrize("dt", list(TYPES))
def test_blocks_with_nan_and_infinity_read_back_as_nan(dt):
    x = torch.ones(2, 128, dtype=TYPES[dt])
    x[0, 3], x[0, 64], x[1, 127] = float("inf"), float("nan"), -float("inf")
    check(x.to(DEV))
    w, _ = quantized(x.to(DEV))
    for out in TYPES:
        y = torch.empty(2, 128, dtype=TYPES[out], device=DEV)
        qmv.qmv_dequant(w, y, out)
        y = y.cpu()
        bad = torch.zeros(2, 4, dtype=torch.bool)
        bad[0, 0] = bad[0, 2] = bad[1, 3] = True
        assert torch.equal(torch.isnan(y).view(2, 4, 32).all(-1), bad)
        assert bool((y.view(2, 4, 32)[~bad] == 1).all())


@pytest.mark.parametrize("dt", list(TYPES))
def test_rows_of_any_stride(dt):
    t = torch.randn(9, 5, 96, generator=torch.Generator().manual_seed(1)).to(TYPES[dt]).to(DEV)
    check(t[:, 2])
    check(t[:, 0, 32:])
    check(t.view(9, 480)[:1, 64:128])
    check(t.view(9, 480)[1:8:3, :320])


@pytest.mark.parametrize("out", list(TYPES))
def test_dequant_of_every_power_and_code(out):
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    p = np.arange(256, dtype=np.uint8)[:, None]
    buf = torch.from_numpy(mx.mx4_pack(p, code)).to(DEV)
    w = qmv.qmv_create_weights("mxfp4", 256, 32, buf)
    y = torch.empty(256, 32, dtype=TYPES[out], device=DEV)
    qmv.qmv_dequant(w, y, out)
    want = torch.from_numpy(mx.mx4_decode64(buf.cpu().numpy(), 256, 32)).float().to(TYPES[out])
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])
    ids = torch.tensor([5, 300, 254, 0, 255, -1, 127], dtype=torch.int32, device=DEV)
    e = torch.empty(7, 32, dtype=TYPES[out], device=DEV)
    qmv.qmv_embed(w, ids, 7, e, out, 0.5)
    full = torch.from_numpy(mx.mx4_decode64(buf.cpu().numpy(), 256, 32)).float()
    for i, r in enumerate(ids.tolist()):
        want = (full[r] * 0.5 if 0 <= r < 256 else torch.zeros(32)).to(TYPES[out])
        assert torch.equal(torch.isnan(e[i].cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(e[i].cpu(), nan=0.0), torch.nan_to_num(want, nan=0.0))


def test_on_another_stream_and_replayed():
    x = torch.randn(33, 256, device=DEV)
    n = qmv.qmv_packed_size("mxfp4", 33, 256)
    buf = torch.zeros(n, dtype=torch.uint8, device=DEV)
    w = qmv.qmv_create_weights("mxfp4", 33, 256, buf)
    out = torch.empty(33, 256, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qmv.qmv_quantize(w, x)
        qmv.qmv_dequant(w, out, "f32")
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmv.qmv_quantize(w, x)
        qmv.qmv_dequant(w, out, "f32")
    for seed in range(3):
        x.copy_(torch.randn(33, 256, generator=torch.Generator().manual_seed(seed)) * 10.0**seed)
        g.replay()
        torch.cuda.synchronize()
        p, code = mx.mx4_encode64(x.cpu().double().numpy())
        want = mx.mx4_decode64(mx.mx4_pack(p, code), 33, 256)
        assert np.array_equal(out.cpu().double().numpy(), want)

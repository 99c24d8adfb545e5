"""qmv_norm against the 64-bit definition.

A row's sums take at most 32 additions in a thread, 6 in a wave and 16 over waves, so they are off by at most 54 2^-24 of
the sum of magnitudes; with the handful of roundings around them a normed value is off by less than 2^-18 of itself, of
the row's centre (layer norms) and of the number before centring, over the root.  An error d of the sum that the second
norm takes comes out as (d + mean d + |z| rms d) / root.  Outputs round once more, by half an epsilon."""
import numpy as np
import pytest
import torch

from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say
from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0**-18


def host(t):
    return None if t is None else t.cpu().double().numpy()


def normed(x, d, kind, w, b, eps):
    """(value, bound of its error) for an input off by at most d."""
    if kind is None:
        return x, d
    c = x.mean(-1, keepdims=True) if kind == "layer" else np.zeros(x.shape[:-1] + (1,))
    root = np.sqrt(((x - c)**2).mean(-1, keepdims=True) + eps)
    z = (x - c) / root
    y = mx.norm64(x, kind, w, b, eps)
    t = E * np.abs(z) + (d + np.abs(z) * np.sqrt((d * d).mean(-1, keepdims=True))) / root
    if kind == "layer":
        t = t + (E * (np.abs(x).mean(-1, keepdims=True) + np.abs(x)) + d.mean(-1, keepdims=True)) / root
    t = t if w is None else t * np.abs(w)
    return y, t + 2.0**-22 * (np.abs(y) + (0 if b is None else np.abs(b)))


def within(got, want, tol, dtype):
    f = torch.finfo(dtype)
    tol = tol + f.eps / 2 * (np.abs(want) + tol) + f.smallest_normal * f.eps
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])


def check(residual, y, **k):
    """One call, against the definition on what it was given (read before the call: outputs may be inputs)."""
    h = {n: host(k.get(n)) for n in ("block", "gate", "pre_weight", "pre_bias", "post_weight", "post_bias")}
    r, eps, scale = host(residual), k.get("eps", 1e-6), k.get("scale", 1.0)
    s, d = r, np.zeros_like(r)
    if h["block"] is not None:
        b, d = normed(h["block"], np.zeros_like(r), k.get("post"), h["post_weight"], h["post_bias"], eps)
        gate = 1.0 if h["gate"] is None else h["gate"]
        term = np.float32(scale) * np.float64(gate) * b
        s = r + term
        d = np.abs(np.float32(scale) * gate) * d + 2.0**-22 * (np.abs(term) + np.abs(s))
    qmv.qmv_norm(qmv.qmv_create_norm(residual, y, **k))
    if k.get("sum_out") is not None:
        within(k["sum_out"], s, d, k["sum_out"].dtype)
    if y is not None:
        want, t = normed(s, d, k.get("pre"), h["pre_weight"], h["pre_bias"], eps)
        within(y, want, t, y.dtype)


def data(rows, cols, dt, seed, **what):
    g = torch.Generator().manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g).to(TYPES[dt]).to(DEV)

    t = dict(residual=r(rows, cols) * 3 + 1, block=r(rows, cols) + 0.5, vector=r(cols), rows=r(rows, cols))
    t.update({n: r(cols) for n in ("pre_weight", "pre_bias", "post_weight", "post_bias")})
    return t


COLS = [1, 7, 64, 96, 511, 512, 520, 1155, 2048, 2056, 3584, 8192, 8200, 18944, 32768, 32767]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_everything_on(cols, dt):
    for rows, pre, post, gate in ((1, "rms", "layer", "vector"), (6, "layer", "rms", "rows"), (5, "rms", "rms", None)):
        say(f"norm {rows}x{cols} {dt} {pre} {post} {gate}")
        t = data(rows, cols, dt, cols + rows)
        bias = {} if rows == 5 else dict(pre_bias=t["pre_bias"], post_bias=t["post_bias"])
        for out in TYPES:
            check(t["residual"], torch.empty(rows, cols, dtype=TYPES[out], device=DEV), pre=pre, post=post,
                  pre_weight=t["pre_weight"], post_weight=t["post_weight"], block=t["block"],
                  gate=None if gate is None else t[gate], scale=0.22, sum_out=torch.empty_like(t["residual"]), **bias)


@pytest.mark.parametrize("dt", list(TYPES))
def test_parts_alone(dt):
    for cols in (96, 1001, 4096):
        t = data(4, cols, dt, cols)
        y = torch.empty(4, cols, dtype=TYPES[dt], device=DEV)
        check(t["residual"], y, pre="rms")
        check(t["residual"], y, pre="layer", pre_bias=t["pre_bias"])
        check(t["residual"], y)  # a copy
        check(t["residual"], None, sum_out=y, block=t["block"], post="rms", post_weight=t["post_weight"])
        check(t["residual"], y, block=t["block"], gate=t["vector"], scale=-2.0)


def test_weights_of_another_type():
    for dt in TYPES:
        for wt in TYPES:
            t, w = data(3, 640, dt, 1), data(1, 640, wt, 2)
            check(t["residual"], torch.empty(3, 640, device=DEV), pre="layer", pre_weight=w["pre_weight"],
                  pre_bias=w["pre_bias"], block=t["block"], post="rms", post_weight=w["post_weight"])


@pytest.mark.parametrize("cols", [72, 1155, 3584])
def test_in_place_and_strided(cols):
    big = torch.randn(3, 5, 2 * cols + 8, device=DEV).to(torch.bfloat16)
    t = data(5, cols, "bf16", 3)
    check(t["residual"], t["block"], pre="rms", pre_weight=t["pre_weight"], block=t["block"], sum_out=t["residual"])
    check(t["residual"], t["residual"], pre="layer", block=t["block"], sum_out=t["block"])
    x, b, s = big[0, :, :cols], big[1, :, 8:8 + cols], big[2, :, cols:2 * cols]
    before = big.clone()
    check(x, torch.empty(5, cols, device=DEV), pre="rms", block=b, gate=t["rows"], sum_out=s)
    before[2, :, cols:2 * cols] = s
    assert torch.equal(before, big)  # nothing beside the output
    check(big[0, :, 1:1 + cols], big[0, :, cols + 3:2 * cols + 3], pre="rms")
    one = t["vector"].expand(5, cols)
    check(t["residual"], big[0, :, :cols], block=t["block"], gate=one)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_without_spread(kind):
    for cols in (64, 5000):
        x = torch.zeros(4, cols, device=DEV)
        x[1], x[2], x[3, 0] = 1000.0, -3.0, 1e-12
        check(x, torch.empty(4, cols, device=DEV), pre=kind)
        check(x, torch.empty(4, cols, device=DEV), pre=kind, block=x.flip(0).contiguous(), post=kind, eps=1e-5)


def test_nan_and_infinity_stay_in_their_rows():
    x = torch.randn(6, 3000, device=DEV)
    x[1, 7], x[4, 2999] = float("nan"), float("inf")
    y = torch.empty_like(x)
    qmv.qmv_norm(qmv.qmv_create_norm(x, y, pre="layer"))
    assert torch.isnan(y[1]).all() and torch.isnan(y[4, 2999])
    assert torch.isfinite(y[[0, 2, 3, 5]]).all()


def test_many_rows_and_streams():
    t = data(4099, 256, "bf16", 5)
    y = torch.empty(4099, 256, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check(t["residual"], y, pre="rms", block=t["block"], post="layer")
    a = qmv.qmv_create_norm(t["residual"], y, pre="rms", block=t["block"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmv.qmv_norm(a)
    for seed in range(3):
        t["block"].copy_(torch.randn(4099, 256, generator=torch.Generator().manual_seed(seed)))
        qmv.qmv_norm(a)
        want = y.clone()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("cols", [2049, 2056, 5003, 8191, 8192])
def test_many_long_rows(cols, dt):
    """Sixteen numbers to a thread, of rows that end inside a run of eight and of rows that do not."""
    say(f"norm 1030x{cols} {dt}")
    t = data(1030, cols, dt, cols)
    check(t["residual"], torch.empty(1030, cols, dtype=TYPES["bf16"], device=DEV), pre="rms", post="layer",
          pre_weight=t["pre_weight"], post_weight=t["post_weight"], post_bias=t["post_bias"], block=t["block"],
          gate=t["rows"], sum_out=torch.empty_like(t["residual"]))

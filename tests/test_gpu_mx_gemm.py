"""qmv_mx4_gemm against the 64-bit definition, dense and by expert.

Products of two codes with their powers are exact; K additions in fp32 in any order, truncated or rounded, are off by at
most K 2^-23 of sum |x w|.  silu has a slope below 1.1, so an error dg of the gate gives 1.1 dg |u|; the epilogue itself
is good to 8 ulp.  Outputs round once more."""
import numpy as np
import pytest
import torch

import oracle
from oracle import mx
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say
from test_gpu_mx_gemv import Mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def outputs(x, w, swiglu):
    """(value, bound of the error before the output's rounding)."""
    y, d = x @ w.T, (np.abs(x) @ np.abs(w).T) * x.shape[1] * 2.0**-23
    if not swiglu:
        return y, d
    n = len(w) // 2
    g, u = y[:, :n], y[:, n:]
    h = oracle.silu64(g) * u
    return h, 1.1 * d[:, :n] * (np.abs(u) + d[:, n:]) + (np.abs(oracle.silu64(g))) * d[:, n:] + 2.0**-20 * np.abs(h)


def within(got, want, tol, dtype):
    f = torch.finfo(dtype)
    tol = tol + f.eps / 2 * (np.abs(want) + tol) + f.smallest_normal * f.eps
    bad = ~(np.abs(got.cpu().double().numpy() - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.sum(), got.cpu().double().numpy()[bad][:4], want[bad][:4])


def run(W, X, rows, n, dt, swiglu, start=None, index=None, pad=0):
    """The call, into a y with `pad` columns and a row of guards around."""
    full = torch.full((rows + 2, n + pad), 7.0, dtype=TYPES[dt], device=DEV)
    y = full[1:-1, :n]
    dev = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(W.desc, X.desc, y, swiglu=swiglu, expert_start=dev(start), x_index=dev(index)))
    assert bool((full[0] == 7.0).all()) and bool((full[-1] == 7.0).all()) and bool((full[:, n:] == 7.0).all())
    return y


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 100, 3584), (3, 17, 96), (16, 256, 1024), (17, 33, 160), (31, 48, 512),
                                   (33, 130, 2880), (64, 64, 128), (77, 1001, 544), (130, 300, 4128), (300, 70, 672),
                                   (513, 520, 288), (257, 255, 1056), (5, 40, 18944)])
def test_dense(m, n, k, dt, swiglu):
    say(f"mx4 gemm {m} x {n} x {k} {dt} swiglu {swiglu}")
    W, X = Mx(n * (2 if swiglu else 1), k, m + n + k, -9, -6), Mx(m, k, m + 1, -3, 1)
    y = run(W, X, m, n, dt, swiglu, pad=n % 5)
    within(y, *outputs(X.w, W.w, swiglu), TYPES[dt])


@pytest.mark.parametrize("start,index", [
    ([0, 4, 4, 9, 40], "random"), ([3, 3, 20, 31, 38], None), ([0, 0, 0, 0, 0], "random"), ([0, 40, 40, 40, 40], "random"),
    ([0, 10, 5, 30, 20], "random"), ([-7, -3, 12, 90, 100], None), ([0, 17, 18, 19, 40], "same"),
    ([0, 13, 14, 39, 40], "outside")])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped(start, index, swiglu):
    rows, n, k, tokens = 40, 45, 320, 40
    W, X = Mx(4 * n * (2 if swiglu else 1), k, 3, -6, -3), Mx(tokens, k, 4, -3, 1)
    r = np.random.default_rng(5)
    idx = None if index is None else np.full(rows, 7) if index == "same" else r.integers(0, tokens, rows)
    if index == "outside":
        idx[[0, 13, 20, 39]] = [-1, tokens, 2**31 - 1, -2**31]
    for dt in TYPES:
        say(f"grouped {start} {index} {swiglu} {dt}")
        y = run(W, X, rows, n, dt, swiglu, start, None if idx is None else idx.tolist(), pad=3)
        covered = np.zeros(rows, bool)
        m = n * (2 if swiglu else 1)
        for e, (a, b) in enumerate(mx.groups(start, rows)):
            covered[a:b] = True
            if a == b:
                continue
            at = np.arange(a, b) if idx is None else idx[a:b]
            known = (at >= 0) & (at < tokens)
            x = np.where(known[:, None], X.w[np.where(known, at, 0)], 0.0)
            within(y[a:b], *outputs(x, W.w[e * m:(e + 1) * m], swiglu), TYPES[dt])
            assert bool((y[a:b][torch.from_numpy(~known).to(DEV)] == 0).all())
        assert bool((y[torch.from_numpy(~covered).to(DEV)] == 7.0).all())  # rows of no expert


@pytest.mark.parametrize("experts,tokens,top,n,k", [(64, 1, 8, 96, 512), (130, 50, 3, 40, 160), (300, 17, 2, 33, 96),
                                                    (5, 700, 2, 264, 384), (2, 1000, 1, 130, 1120), (1, 37, 4, 64, 64)])
def test_many_experts_and_long_groups(experts, tokens, top, n, k):
    say(f"experts {experts} tokens {tokens} top {top}")
    r = np.random.default_rng(experts)
    rows = tokens * top
    cuts = np.sort(r.integers(0, rows + 1, experts - 1)) if experts > 1 else np.zeros(0, int)
    start = [0] + cuts.tolist() + [rows]
    idx = r.permutation(np.repeat(np.arange(tokens), top))
    for swiglu in (False, True):
        W, X = Mx(experts * n * (2 if swiglu else 1), k, 1, -6, -3), Mx(tokens, k, 2, -3, 1)
        y = run(W, X, rows, n, "bf16", swiglu, start, idx.tolist())
        m = n * (2 if swiglu else 1)
        for e in range(experts):
            a, b = start[e], start[e + 1]
            if b > a:
                within(y[a:b], *outputs(X.w[idx[a:b]], W.w[e * m:(e + 1) * m], swiglu), torch.bfloat16)


def test_integers_are_exact():
    r = np.random.default_rng(0)
    for m, n, k in ((9, 65, 1024), (200, 200, 1024), (600, 520, 2048)):
        wb = mx.mx4_pack(np.full((n, k // 32), 128), r.integers(0, 16, (n, k)))
        xb = mx.mx4_pack(np.full((m, k // 32), 128), r.integers(0, 16, (m, k)))
        W = qmv.qmv_create_weights("mxfp4", n, k, torch.from_numpy(wb).to(DEV))
        X = qmv.qmv_create_weights("mxfp4", m, k, torch.from_numpy(xb).to(DEV))
        y = torch.empty(m, n, device=DEV)
        qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(W, X, y))
        want = mx.mx4_decode64(xb, m, k) @ mx.mx4_decode64(wb, n, k).T  # integers below 2^24
        assert np.array_equal(y.cpu().double().numpy(), want)


def test_nan_blocks():
    for m in (5, 300):
        W, X = Mx(70, 256, 1), Mx(m, 256, 2, -3, 1)
        W.dev[70 * 128 + 8 * 11 + 2] = 255
        X.dev[m * 128 + 8 * 3 + 7] = 255
        y = torch.empty(m, 70, device=DEV)
        qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(W.desc, X.desc, y))
        bad = torch.zeros(m, 70, dtype=torch.bool)
        bad[:, 11] = bad[3] = True
        assert torch.equal(torch.isnan(y.cpu()), bad)


def test_far_powers():
    for m in (4, 200):
        W, X = Mx(40, 512, 1, -100, -90), Mx(m, 512, 2, 60, 70)
        within(run(W, X, m, 40, "f32", False), *outputs(X.w, W.w, False), torch.float32)


def test_swiglu_saturates():
    """Gates far from zero: silu(g) u tends to g u and to 0, without NaN."""
    k = 64
    code = np.full((2, k), 7)
    W = np.concatenate([mx.mx4_pack(np.full((2, 2), 127), code)])
    for p, lo in ((127, 0.0), (150, 0.0), (180, 0.0)):
        for sign in (0, 8):
            xb = mx.mx4_pack(np.full((1, 2), p), np.full((1, k), 7 | sign))
            w = qmv.qmv_create_weights("mxfp4", 2, k, torch.from_numpy(W).to(DEV))
            x = qmv.qmv_create_weights("mxfp4", 1, k, torch.from_numpy(xb).to(DEV))
            y = torch.empty(1, 1, device=DEV)
            qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(w, x, y, swiglu=True))
            g = 36.0 * k * 2.0**(p - 127) * (-1 if sign else 1)
            # (2304 2^53 squared is 4.3e38, above fp32's 3.4e38: rounded to y's type, an infinity)
            want = g * g if g > 0 else 0.0
            if want > torch.finfo(torch.float32).max:
                assert y.item() == float("inf")
            else:
                assert abs(y.item() - want) <= 1e-6 * abs(want), (p, sign, y.item(), want)


def test_two_streams_and_replays():
    W, X, n = Mx(3 * 96, 512, 1, -6, -3), Mx(50, 512, 2, -3, 1), 96
    start = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device=DEV)
    index = torch.arange(50, dtype=torch.int32, device=DEV)
    ys = [torch.zeros(50, n, device=DEV) for _ in range(3)]
    calls = [qmv.qmv_create_mx4(W.desc, X.desc, y, expert_start=start, x_index=index) for y in ys]
    streams = [torch.cuda.Stream() for _ in range(2)]
    qmv.qmv_mx4_gemm(calls[0])
    torch.cuda.synchronize()
    for s, c in zip(streams, calls[1:]):
        with torch.cuda.stream(s):
            qmv.qmv_mx4_gemm(c)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmv.qmv_mx4_gemm(calls[0])
    for cut in (0, 13, 50):  # the groups are read at every replay
        start.copy_(torch.tensor([0, cut, cut, 50], dtype=torch.int32))
        index.copy_(torch.randperm(50).to(torch.int32))
        g.replay()
        torch.cuda.synchronize()
        x = X.w[index.cpu().numpy()]
        for e, (a, b) in enumerate(((0, cut), (cut, cut), (cut, 50))):
            if b > a:
                within(ys[0][a:b], *outputs(x[a:b], W.w[e * n:(e + 1) * n], False), torch.float32)


def on_gpu(m, rows=None):
    """64-bit values of an Mx's rows on the GPU."""
    w = torch.from_numpy(m.w)
    return (w if rows is None else w[rows]).to(DEV)


# Shapes with more tiles than workgroups stay (each takes several in turn, the next one's first stages loaded ahead), of
# one stage, of fewer than the ring's four, of parts of a stage, and of many; and with fewer tiles, for each kernel that
# the launch chooses from.
@pytest.mark.parametrize("m,n,k", [(4100, 9000, 32), (3000, 7000, 160), (5000, 4990, 384), (4096, 5120, 512), (3001, 6007, 1440),
                                   (2500, 9000, 2048), (12, 20000, 96), (60, 20000, 256), (20, 9001, 1056), (100, 3584, 1568)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_tiles(m, n, k, swiglu):
    say(f"mx4 gemm {m} x {n} x {k} swiglu {swiglu}")
    n = n // 2 if swiglu else n
    W, X = Mx(n * (2 if swiglu else 1), k, m + n, -6, -3), Mx(m, k, m + 1, -3, 1)
    for dt in (("f32", "bf16") if m > 200 else list(TYPES)):
        y = run(W, X, m, n, dt, swiglu)
        x, w = on_gpu(X), on_gpu(W)
        want, tol = x @ w.T, (x.abs() @ w.abs().T) * k * 2.0**-23
        if swiglu:
            (g, u), (dg, du) = want.chunk(2, -1), tol.chunk(2, -1)
            s = g / (1 + torch.exp(-g))
            want, tol = s * u, 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0**-20 * (s * u).abs()
        f = torch.finfo(TYPES[dt])
        tol = tol + f.eps / 2 * (want.abs() + tol) + f.smallest_normal * f.eps
        assert bool(((y.double() - want).abs() <= tol).all())


def test_many_tiles_of_experts():
    """Enough ragged groups for several tiles to a workgroup, with indices outside and rows of no expert."""
    experts, n, k, tokens, rows = 70, 700, 288, 900, 9000
    W, X = Mx(experts * 2 * n, k, 1, -6, -3), Mx(tokens, k, 2, -3, 1)
    r = np.random.default_rng(7)
    cuts = np.sort(r.integers(20, rows - 30, experts - 1))
    start = [20] + cuts.tolist() + [rows - 30]
    idx = r.integers(-2, tokens + 2, rows)
    y = run(W, X, rows, n, "f32", True, start, idx.tolist())
    x = on_gpu(X)[torch.from_numpy(np.clip(idx, 0, tokens - 1)).to(DEV)]
    x[torch.from_numpy((idx < 0) | (idx >= tokens)).to(DEV)] = 0
    for e in range(experts):
        a, b = start[e], start[e + 1]
        w = on_gpu(W, slice(e * 2 * n, (e + 1) * 2 * n))
        g, u = (x[a:b] @ w.T).chunk(2, -1)
        mag = (x[a:b].abs() @ w.abs().T) * k * 2.0**-23
        dg, du = mag.chunk(2, -1)
        s = g / (1 + torch.exp(-g))
        tol = 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0**-20 * (s * u).abs() + 1e-38
        assert bool(((y[a:b].double() - s * u).abs() <= tol).all()), e
    assert bool((y[:20] == 7.0).all()) and bool((y[-30:] == 7.0).all())

"""qmv_attn where a few keys outweigh all others and hold values of zero (an attention sink), so that the output is the
weighted values of keys far below the maximum.

Tolerances.  As in test_gpu_attn.py, but for the probabilities.  An fp16 number below 2^-14 is a multiple of 2^-24,
so however a probability is rounded to one or two of them it can be off by half of that, 2^-25, where the largest
enters as 2^12 or more: by 2^-37 of the largest.  Above that it is within 2^-16 of itself (two numbers) or half an epsilon
(one, where a key head has more than 64 rows on the prefix).  With L the sum of the probabilities over their largest,
an output is off by at most (sum_j |v_j| + n |o|) 2^-37 / L more than before.  (The absolute term is asked of bf16
too, whose exponent has no such floor.)"""
import numpy as np
import pytest
import torch

from oracle.step import attn64
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say
from test_gpu_attn import TYPES

pytestmark = pytest.mark.gpu

NATS = [8, 10, 12, 13, 14, 15, 16, 18]


def sink(dtype, dim, heads, kv, prefix, rows, suffix, nats, at, spread, seed):
    """Sinks at every `at`-th key, `nats` above the others' scores of 0 (and a little more or less with spread)."""
    g = torch.Generator().manual_seed(seed)
    t, page, n = TYPES[dtype], 16, sum(rows)
    scale = 0.125
    q = torch.zeros(n, heads, dim)
    q[..., 0] = 8.0  # score = the key's first element
    q[..., 1] = 4.0
    per = [-(-s // page) for s in suffix]
    k = torch.zeros(prefix, kv, dim), torch.zeros(sum(per), page, kv, dim)
    v = [50.0 * (1.0 + 0.3 * torch.randn(x.shape, generator=g)) for x in k]
    for x, y, tokens in ((k[0], v[0], torch.arange(prefix)), (k[1], v[1], None)):
        x[..., 2:] = torch.randn(x[..., 2:].shape, generator=g)  # (q is zero there)
        x[..., 1] = spread * (2 * torch.rand(x[..., 1].shape, generator=g) - 1)
        where = (torch.arange(len(x)) if tokens is not None else torch.arange(len(x) * page)) % at == at // 2
        x.view(-1, kv, dim)[where, :, 0] = float(nats)
        y.view(-1, kv, dim)[where] = 0.0
    table, p = torch.zeros(len(rows), max(per + [1]), dtype=torch.int32), 0
    for b, m in enumerate(per):
        table[b, :m] = torch.arange(p, p + m)
        p += m
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q, k, v = q.to(t), [x.to(t) for x in k], [x.to(t) for x in v]
    d = lambda x: x.to(DEV)  # noqa: E731
    out, lse = torch.full(q.shape, 7.0, dtype=t, device=DEV), torch.empty(n, heads, device=DEV)
    kw = dict(k_pages=d(k[1]), v_pages=d(v[1]), block_table=d(table), max_suffix=max(suffix),
              suffix_len=torch.tensor(suffix, dtype=torch.int32, device=DEV)) if max(suffix) else {}
    if prefix:
        kw.update(k_prefix=d(k[0]), v_prefix=d(v[0]))
    a = qmv.qmv_create_attn(d(q), out, d(torch.from_numpy(start)), max(rows), scale=scale, lse=lse, **kw)
    nws = qmv.qmv_attn_workspace_size(a)
    qmv.qmv_attn(a, torch.full((nws,), 255, dtype=torch.uint8, device=DEV), nws)
    got, glse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    f = lambda x: x.double().numpy()  # noqa: E731
    want, wlse, mag, smax = attn64(f(q), start, scale, f(k[0]) if prefix else None, f(v[0]) if prefix else None, None,
                                   prefix, f(k[1]), f(v[1]), table.numpy(), suffix)
    keys = prefix + max(suffix)
    total = max(float(x.double().abs().max()) for x in v if x.numel()) * keys
    weight = np.exp(wlse - smax)[..., None]  # L, or less
    eps = torch.finfo(t).eps
    once = eps if n * heads // kv > 64 and prefix else 0.0
    rel = 4 * smax * (dim + 8) * 2.0**-24 + 2.0**-15 + 2.0**-21 + 4 * keys * 2.0**-24 + once
    tol = mag * rel[..., None] * (1 + eps / 2) + np.abs(want) * eps / 2 + (2.0**-25 if dtype == "f16" else 0)
    tol += (total + keys * np.abs(want)) * 2.0**-37 / weight
    off = np.abs(got - want)
    say(f"  {nats} nats: worst error {np.max(off / np.abs(want)):.2e} of the output, {np.max(off / tol):.3f} of the tolerance")
    assert np.all(off <= tol)
    tl = np.abs(wlse) * 2.0**-22 + 2 * smax * (dim + 8) * 2.0**-24 + 2 * keys * 2.0**-24 + 2.0**-21 + once / 2
    assert np.all(np.abs(glse - wlse) <= tl + keys * 2.0**-37 / weight[..., 0])


# (a sink in every 32 keys meets them in one tile, whatever ranges the keys are cut into; one in 128 is in one tile of four)
@pytest.mark.parametrize("at,spread", [(32, 0.0), (32, 1.0), (128, 1.0), (1000, 0.5)])
@pytest.mark.parametrize("nats", NATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["one row", "few rows", "many rows", "suffix", "suffix of one row"])
def test_values_far_below_a_sink(where, dtype, nats, at, spread):
    say(f"attn sink {where} {dtype} {nats} nats, every {at}, spread {spread}")
    prefix, rows, suffix, heads = {"one row": (1500, [1], [1], 4), "few rows": (1500, [3, 6], [3, 6], 4),
                                   "many rows": (1500, [4] * 10, [4] * 10, 8), "suffix": (0, [3, 4], [1500, 700], 8),
                                   "suffix of one row": (40, [1, 1], [1200, 300], 2)}[where]
    sink(dtype, 64, heads, 1, prefix, rows, suffix, nats, at, spread, seed=nats)


@pytest.mark.parametrize("dim", [80, 128, 256])
@pytest.mark.parametrize("rows", [[1], [5], [6] * 20])
def test_widths(rows, dim):
    for nats in (12, 16):
        sink("f16", dim, 8, 2, 900, rows, [40 + r for r in rows], nats, 32, 0.5, seed=dim)


def test_a_sink_that_comes_last():
    # the small ones are added up first, and rescaled when the sink arrives
    for rows in ([1], [4], [4] * 20):
        for nats in (12, 18):
            sink("f16", 64, 4, 1, 1999, rows, rows, nats, 3996, 1.0, seed=nats)

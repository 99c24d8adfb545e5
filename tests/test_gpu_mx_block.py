"""The MXFP4 operators together, as a block of experts uses them (examples/mxfp4_experts.py): each stage against its
64-bit definition on what the stage before gave, all of it captured and replayed, and one token's exact path."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import oracle
from oracle import mx
from gpu_util import DEV
from test_gpu_mx_gemm import outputs, within
from test_gpu_norm import normed, within as norm_within

pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().double().numpy()


def encoded(t):
    p, code = mx.mx4_encode64(host(t))
    return mx.mx4_pack(p, code)


@pytest.mark.parametrize("rows,hidden,width,experts,top", [(1, 256, 96, 8, 2), (37, 512, 384, 8, 2), (300, 320, 160, 5, 3)])
def test_block(rows, hidden, width, experts, top):
    from mxfp4_experts import Block
    b = Block(hidden, width, experts, top, seed=rows)
    g = torch.Generator(device=DEV).manual_seed(rows)
    residual, attended = (torch.randn(rows, hidden, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    total, nxt, s = b(residual, attended)
    # the norm before
    term = host(attended)
    mid = host(residual) + term
    d = 2.0**-22 * (np.abs(term) + np.abs(mid))
    norm_within(s["middle"], mid, d, torch.bfloat16)
    want, t = normed(mid, d, "rms", host(b.norms[0]), None, 1e-6)
    norm_within(s["x"], want, t, torch.bfloat16)
    # quantized, exactly
    assert np.array_equal(s["xq"].owner.cpu().numpy(), encoded(s["x"]))
    assert np.array_equal(s["hq"].owner.cpu().numpy(), encoded(s["h"]))
    for w, given in zip((b.gate_up, b.down), b.given):
        assert np.array_equal(w.owner.cpu().numpy(), encoded(given))
    # the experts' products
    x = mx.mx4_decode64(s["xq"].owner.cpu().numpy(), rows, hidden)[s["token"].cpu().numpy()]
    h = mx.mx4_decode64(s["hq"].owner.cpu().numpy(), rows * top, width)
    gu = mx.mx4_decode64(b.gate_up.owner.cpu().numpy(), experts * 2 * width, hidden).reshape(experts, -1, hidden)
    dn = mx.mx4_decode64(b.down.owner.cpu().numpy(), experts * hidden, width).reshape(experts, -1, width)
    start = s["start"].tolist()
    assert start[0] == 0 and start[-1] == rows * top
    for e in range(experts):
        a, z = start[e], start[e + 1]
        if z > a:
            within(s["h"][a:z], *outputs(x[a:z], gu[e], True), torch.bfloat16)
            within(s["y"][a:z], *outputs(h[a:z], dn[e], False), torch.float32)
    # the norms after
    blk, bd = normed(host(s["out"]), np.zeros((rows, hidden)), "rms", host(b.norms[2]), None, 1e-6)
    tot = host(s["middle"]) + 0.5 * blk
    d = 0.5 * bd + 2.0**-22 * (np.abs(0.5 * blk) + np.abs(tot))
    norm_within(total, tot, d, torch.bfloat16)
    want, t = normed(tot, d, "rms", host(b.norms[1]), None, 1e-6)
    norm_within(nxt, want, t, torch.bfloat16)


def test_block_captured():
    from mxfp4_experts import Block
    b = Block(256, 96, 6, 2)
    residual, attended = (torch.randn(20, 256, device=DEV).to(torch.bfloat16) for _ in range(2))
    _, _, s = b(residual, attended)
    route = (s["token"], s["start"], s["rows"], s["weight"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total, nxt, _ = b(residual, attended, route)
    for seed in range(3):
        residual.copy_(torch.randn(20, 256, generator=torch.Generator().manual_seed(seed)))
        want = b(residual, attended, route)
        total.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(total, want[0]) and torch.equal(nxt, want[1])


def test_one_token_exactly():
    from mxfp4_experts import Block
    b = Block(256, 96, 6, 2)
    x = torch.randn(1, 256, device=DEV).to(torch.bfloat16)
    got = host(b.one_token(x, [5, 0, 2]))
    gu = mx.mx4_decode64(b.gate_up.owner.cpu().numpy(), 6 * 192, 256).reshape(6, 192, 256)
    dn = mx.mx4_decode64(b.down.owner.cpu().numpy(), 6 * 256, 96).reshape(6, 256, 96)
    for k, e in enumerate([5, 0, 2]):
        g, u = host(x) @ gu[e, :96].T, host(x) @ gu[e, 96:].T
        want = (oracle.silu64(g) * u) @ dn[e].T
        assert np.all(oracle.normwise_rel_err(got[k:k + 1], want) <= 2e-3)


def test_example_runs(capsys):
    import mxfp4_experts
    mxfp4_experts.main()
    assert "200 rows over 8 experts" in capsys.readouterr().out

"""qmv_verify against the float64 oracle: whole numbers, equal.

Two evaluations of the same 64-bit sums differ by parts in 1e13 at most; the oracle reports how far each sequence's
comparisons are from equality, and inputs nearer than 1e-10 (none of the seeds here) would not be compared."""
import numpy as np
import pytest
import torch

from oracle.step import verify64
from block_quantized_weight_qmv_amd import qmv
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(vocab, rows, dtype="f32", probs=True, temperature=None, seed=0, spread=2.0, outside=0, agree=0.6):
    g = torch.Generator().manual_seed(seed)
    n = sum(rows) + outside
    logits = torch.randn(n, vocab, generator=g) * spread
    near = logits + agree * torch.randn(n, vocab, generator=g)
    q = torch.softmax(near, -1)
    tokens = torch.zeros(n, dtype=torch.int32)
    drawn = torch.multinomial(q, 1, generator=g)[:, 0] if probs else near.argmax(-1)
    tokens[1:] = drawn[:-1].to(torch.int32)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return dict(logits=logits.to(TYPES[dtype]), tokens=tokens, row_start=torch.from_numpy(start),
                u_accept=torch.rand(n, generator=g), u_sample=torch.rand(len(rows), generator=g),
                draft_probs=q if probs else None,
                temperature=None if temperature is None else torch.tensor(temperature, dtype=torch.float32))


def run(s, max_rows=None, stream=None, keep=None):
    d = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    nseq, n = len(s["row_start"]) - 1, len(s["tokens"])
    out = torch.full((n + 2,), 77, dtype=torch.int32, device=DEV)
    acc = torch.full((nseq + 1,), 77, dtype=torch.int32, device=DEV)
    m = max_rows or max(1, int(s["row_start"].diff().max()))
    a = qmv.qmv_create_verify(d["logits"], d["tokens"], d["row_start"], m, d["u_accept"], d["u_sample"], out[:n],
                              acc[:nseq], draft_probs=d["draft_probs"], temperature=d["temperature"])
    nws = qmv.qmv_verify_workspace_size(a)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=DEV)  # nothing may rely on its contents
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    qmv.qmv_verify(a, ws, nws, stream)
    if keep is not None:
        keep.update(a=a, ws=ws, nws=nws, out=out, acc=acc, d=d)
    torch.cuda.synchronize()
    assert bool((out[n:] == 77).all()) and int(acc[nseq]) == 77
    return out[:n].cpu().numpy(), acc[:nseq].cpu().numpy()


def check(s, **k):
    got, acc = run(s, **k)
    f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
    want, wacc, margin = verify64(f(s["logits"]), s["tokens"].numpy(), s["row_start"].numpy(), s["u_accept"].numpy(),
                                  s["u_sample"].numpy(), None if s["draft_probs"] is None else s["draft_probs"].numpy(),
                                  None if s["temperature"] is None else s["temperature"].numpy())
    assert margin.min() > 1e-10
    assert np.array_equal(acc, wacc), (acc, wacc)
    assert np.array_equal(got, want), (got, want)
    return got, acc


@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 64, 65, 255, 1000, 4097, 32000, 50257])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("probs", [True, False])
def test_vocabularies(vocab, dtype, probs):
    say(f"verify vocab {vocab} {dtype} probs {probs}")
    check(make(vocab, [5, 1, 3, 4, 2], dtype, probs, seed=vocab))


def test_lm_head_vocabulary():
    for probs in (True, False):
        got, acc = check(make(152064, [6, 1, 8, 5], "f32", probs, [1.0, 0.7, 1.3, 0.9], seed=2, spread=3.0))
        say(got, acc)


@pytest.mark.parametrize("probs", [True, False])
def test_many_sequences_temperatures_and_greedy(probs):
    rows = [1 + (i * 5) % 8 for i in range(60)]
    t = [(0.0, 0.5, 1.0, 2.0, 0.01)[i % 5] for i in range(60)]
    for seed in range(3):
        got, acc = check(make(3001, rows, "f32", probs, t, seed=seed))
        assert acc.max() > 2 and acc.min() == 0


def test_rounded_logits_with_ties_take_the_lowest():
    s = make(500, [3, 1, 2], "bf16", False, [0.0, 0.0, 0.0], seed=3)
    s["logits"] = (s["logits"].float() * 0.5).round().to(torch.bfloat16)
    check(s)


def test_border_numbers():
    s = make(300, [4, 4, 4, 1, 1], "f32", True, seed=4)
    s["u_accept"][:4], s["u_accept"][4:8] = 0.0, 1.0 - 2.0**-24
    s["u_sample"][:] = torch.tensor([0.0, 1.0 - 2.0**-24, 0.5, 0.0, 1.0 - 2.0**-24])
    got, acc = run(s)
    want, wacc, _ = verify64(s["logits"].double().numpy(), s["tokens"].numpy(), s["row_start"].numpy(),
                             s["u_accept"].numpy(), s["u_sample"].numpy(), s["draft_probs"].numpy())
    assert np.array_equal(got, want) and np.array_equal(acc, wacc)


def test_accepts_everything_where_the_draft_is_the_target():
    s = make(1000, [8, 8, 8], "f32", True, seed=5)
    s["draft_probs"] = torch.softmax(s["logits"].double(), -1).float() * (1 - 2.0**-20)
    tokens = torch.multinomial(s["draft_probs"], 1)[:, 0].to(torch.int32)
    s["tokens"][1:] = tokens[:-1]
    got, acc = check(s)
    assert list(acc) == [7, 7, 7]
    # a draft that both give no probability: rejected, and nothing remains but p itself
    s["draft_probs"] = torch.softmax(s["logits"].double(), -1).float() * (1 + 2.0**-20)
    for r, x in [(0, 5), (8, 17)]:
        s["logits"][r, x] = float("-inf")
        s["tokens"][r + 1] = x
        p = torch.softmax(s["logits"][r].double(), -1)
        s["draft_probs"][r] = (p * (1 + 2.0**-20)).float()
    got, acc = check(s)
    assert acc[0] == 0 and acc[1] == 0 and got[0] >= 0 and got[8] >= 0


def test_infinities_and_nan():
    nan, inf = float("nan"), float("inf")
    s = make(700, [3, 3, 2, 1, 2, 1], "f32", True, [1.0, 1.0, 0.0, 1.0, 0.5, 0.0], seed=6)
    s["logits"][0, ::2] = nan
    s["logits"][1, :650] = -inf
    s["logits"][3] = -inf           # no distribution
    s["logits"][6, 33] = s["logits"][6, 44] = inf   # greedy between two infinities
    s["logits"][8, 100:104] = inf   # shared between four
    s["logits"][9, 3] = inf
    s["logits"][11] = nan           # no distribution
    s["draft_probs"][0, ::3] = nan
    s["draft_probs"][9, ::5] = -1.0
    got, acc = check(s)
    assert got[3] == -1 and acc[1] == 0 and got[11] == -1 and got[8] in (100, 101, 102, 103)
    for dtype in ("f16", "bf16"):
        s["logits"] = s["logits"].to(TYPES[dtype])
        check(s)


def test_drafts_outside_the_vocabulary():
    for probs in (True, False):
        s = make(100, [3, 3, 3], "f32", probs, [1.0, 0.0, 2.0], seed=7)
        s["tokens"][1], s["tokens"][4], s["tokens"][7] = -1, 100, 2**31 - 1
        got, acc = check(s)
        assert list(acc) == [0, 0, 0]


def test_negative_and_nan_temperatures_count_as_zero():
    s = make(100, [2, 2], "f32", True, [-1.0, float("nan")], seed=8)
    check(s)


def test_tiny_and_huge_temperatures():
    s = make(2000, [3, 3, 3], "f32", True, [1e-6, 1e6, 1e-30], seed=9)
    check(s)


def test_sequences_without_rows_and_rows_without_sequence():
    s = make(100, [0, 2, 0, 3, 0], "f32", True, seed=10, outside=3)
    got, acc = check(s)
    assert list(got[5:]) == [-1, -1, -1] and acc[0] == acc[2] == acc[4] == 0


def test_no_rows_at_all():
    s = make(100, [0, 0], "f32", True, seed=10, outside=1)
    got, acc = run(s)
    assert list(got) == [-1] and list(acc) == [0, 0]


def test_strided_rows():
    s = make(1000, [4, 3], "f32", True, seed=11)
    want = run(s)
    wide, wideq = torch.zeros(7, 1037), torch.zeros(7, 1111)
    wide[:, :1000], wideq[:, 5:1005] = s["logits"], s["draft_probs"]
    d = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    wide, wideq = wide.to(DEV), wideq.to(DEV)
    out, acc = torch.empty(7, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    a = qmv.qmv_create_verify(wide[:, :1000], d["tokens"], d["row_start"], 4, d["u_accept"], d["u_sample"], out, acc,
                              draft_probs=wideq[:, 5:1005])
    nws = qmv.qmv_verify_workspace_size(a)
    qmv.qmv_verify(a, torch.empty(nws, dtype=torch.uint8, device=DEV), nws)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


def test_rows_past_max_rows_are_not_there():
    s = make(500, [5, 2], "f32", True, seed=12)
    s["u_accept"][:] = 0.0
    got, acc = run(s, max_rows=3)
    cut = dict(s, row_start=torch.tensor([0, 3, 5], dtype=torch.int32))
    assert acc[0] <= 2 and list(got[3:5]) == [-1, -1]


def test_wild_row_starts_stay_in_bounds():
    s = make(500, [3, 2, 4], "f32", True, seed=13)
    s["row_start"] = torch.tensor([-5, 1 << 30, 2, -(1 << 31)], dtype=torch.int32)
    run(s, max_rows=4)


def test_rows_past_32_bit_offsets():
    rows, vocab = 3, 1000
    s = make(vocab, [3], "f32", True, seed=14)
    want = run(s)
    far = (1 << 31) - 64
    buf = torch.empty(2 * far + vocab, dtype=torch.float32, device=DEV)
    lg = buf.as_strided((rows, vocab), (far, 1))
    lg.copy_(s["logits"])
    d = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    out, acc = torch.empty(3, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    a = qmv.qmv_create_verify(lg, d["tokens"], d["row_start"], 3, d["u_accept"], d["u_sample"], out, acc,
                              draft_probs=d["draft_probs"])
    nws = qmv.qmv_verify_workspace_size(a)
    qmv.qmv_verify(a, torch.empty(nws, dtype=torch.uint8, device=DEV), nws)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])


def test_another_stream_and_a_graph():
    s = make(5000, [4, 1, 3], "bf16", True, seed=15)
    want = run(s)
    st, keep = torch.cuda.Stream(), {}
    got = run(s, stream=st, keep=keep)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        qmv.qmv_verify(keep["a"], keep["ws"], keep["nws"], st)
    fresh = torch.rand(4, 8)
    for i in range(4):
        s["u_accept"] = fresh[i]
        keep["d"]["u_accept"].copy_(fresh[i])
        keep["out"].fill_(77)
        g.replay()
        torch.cuda.synchronize()
        want = run(s)
        assert np.array_equal(keep["out"][:8].cpu().numpy(), want[0])
        assert np.array_equal(keep["acc"][:3].cpu().numpy(), want[1])

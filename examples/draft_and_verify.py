"""Draft-and-verify decoding with block-quantized weights: the library's operators as one decode step uses them.

    python examples/draft_and_verify.py

A small decoder (random weights: INT4 projections, Q8_0 embedding table and lm-head) serves a few
sequences that share a prompt.  Every step takes all sequences' rows at once -- the last accepted token of each and the
tokens drafted after it -- through

    qmv_embed        the rows' tokens looked up in the quantized table
    qmv_gemv_multi   q, k, v; then, after attention, o, gate and up, down, and the lm-head
    qmv_attn         each row over the shared prompt and its own sequence's pages
    qmv_verify       drafts accepted or a token drawn, from given random numbers

and nothing but the step's tokens and the accepted counts returns to the host.  (Norms, SiLU and the cache's writes are torch operations
here.)  It first decodes one token a step, then verifies those very tokens as drafts, several a step, and says how many
steps that saved.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_weight_qmv_amd import qmv  # noqa: E402
from synth import gen_weights  # noqa: E402

DEV, T = "cuda:0", torch.bfloat16
HIDDEN, FFN, HEADS, KV_HEADS, DIM, VOCAB, LAYERS = 512, 1024, 8, 2, 64, 2048, 2
PAGE, PROMPT = 16, 100


class Matrix:
    """A block-quantized matrix on the GPU, and its products with a step's rows."""

    def __init__(self, fmt, rows, cols, seed, scale):
        f = gen_weights(fmt, rows, cols, seed)
        for k in ("d_bits", "s_bits"):  # the seeded scales, brought to the size of a trained matrix's
            if k in f:
                f[k] = (f[k].view("float16") * scale).astype("float16").view("uint16")
        self.fmt, self.rows, self.cols = fmt, rows, cols
        self.desc = qmv.qmv_create_weights(fmt, rows, cols, torch.from_numpy(qmv.pack_fields(fmt, f, rows, cols)).to(DEV))


def products(x, matrices):
    """x W^T for matrices of one format, in one launch where the library can."""
    out = [torch.empty(len(x), m.rows, dtype=torch.float32, device=DEV) for m in matrices]
    items = [(m.desc, x, y) for m, y in zip(matrices, out)]
    fmt, n = matrices[0].fmt, len(x)
    nws = qmv.qmv_workspace_size(fmt, "bf16", n, items)
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV) if nws else None
    qmv.qmv_gemv_multi_ws(fmt, "bf16", n, items, ws, nws)
    return out


def norm(x):
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(T).contiguous()


class Decoder:
    def __init__(self, seqs, most_tokens, seed=0):
        g = torch.Generator().manual_seed(seed)
        shapes = dict(q=(HEADS * DIM, HIDDEN), k=(KV_HEADS * DIM, HIDDEN), v=(KV_HEADS * DIM, HIDDEN),
                      o=(HIDDEN, HEADS * DIM), gate=(FFN, HIDDEN), up=(FFN, HIDDEN), down=(HIDDEN, FFN))
        self.layers = [{n: Matrix("int4_g128", r, c, 10 * i + j, 0.3) for j, (n, (r, c)) in enumerate(shapes.items())}
                       for i in range(LAYERS)]
        self.table, self.head = Matrix("q8_0", VOCAB, HIDDEN, 98, 0.15), Matrix("q8_0", VOCAB, HIDDEN, 99, 0.15)
        per = -(-most_tokens // PAGE)
        self.pages_of = torch.randperm(seqs * per, generator=g).view(seqs, per).to(DEV).to(torch.int32)
        self.k_pages = torch.zeros(LAYERS, seqs * per, PAGE, KV_HEADS, DIM, dtype=T, device=DEV)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.prompt = [torch.randn(LAYERS, PROMPT, KV_HEADS, DIM, generator=g).to(T).to(DEV) for _ in range(2)]
        self.length = torch.zeros(seqs, dtype=torch.int32, device=DEV)  # suffix tokens in the cache
        self.seqs, self.most = seqs, most_tokens

    def step(self, tokens, counts, u_accept, u_sample, temperature):
        """One step over rows of `counts` tokens a sequence: (out_tokens, accepted) as qmv_verify gives them."""
        n = len(tokens)
        starts = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
        seq = torch.repeat_interleave(torch.arange(self.seqs), torch.tensor(counts)).to(DEV)
        place = self.length[seq] + torch.arange(n, device=DEV) - starts[seq]  # the rows' places in their suffixes
        page, slot = self.pages_of[seq, (place // PAGE).long()].long(), (place % PAGE).long()
        suffix = self.length + torch.tensor(counts, dtype=torch.int32, device=DEV)
        x = torch.empty(n, HIDDEN, dtype=torch.float32, device=DEV)
        qmv.qmv_embed(self.table.desc, tokens, n, x, "f32", 8.0)
        for i, w in enumerate(self.layers):
            q, k, v = products(norm(x), [w["q"], w["k"], w["v"]])
            self.k_pages[i][page, slot] = k.view(n, KV_HEADS, DIM).to(T)
            self.v_pages[i][page, slot] = v.view(n, KV_HEADS, DIM).to(T)
            att = torch.empty(n, HEADS, DIM, dtype=T, device=DEV)
            a = qmv.qmv_create_attn(q.view(n, HEADS, DIM).to(T), att, starts, max(counts), scale=DIM ** -0.5,
                                    k_prefix=self.prompt[0][i], v_prefix=self.prompt[1][i], k_pages=self.k_pages[i],
                                    v_pages=self.v_pages[i], block_table=self.pages_of, suffix_len=suffix,
                                    max_suffix=self.most)
            nws = qmv.qmv_attn_workspace_size(a)
            qmv.qmv_attn(a, torch.empty(nws, dtype=torch.uint8, device=DEV), nws)
            x = x + products(att.view(n, HEADS * DIM), [w["o"]])[0]
            gate, up = products(norm(x), [w["gate"], w["up"]])
            x = x + products((torch.nn.functional.silu(gate) * up).to(T), [w["down"]])[0]
        logits = products(norm(x), [self.head])[0]
        out = torch.empty(n, dtype=torch.int32, device=DEV)
        accepted = torch.empty(self.seqs, dtype=torch.int32, device=DEV)
        a = qmv.qmv_create_verify(logits, tokens, starts, max(counts), u_accept, u_sample, out, accepted,
                                  temperature=temperature)
        nws = qmv.qmv_verify_workspace_size(a)
        qmv.qmv_verify(a, torch.empty(nws, dtype=torch.uint8, device=DEV), nws)
        self.length = self.length + accepted + 1  # rejected drafts' cache entries are overwritten by the next step
        return out, accepted


def decode(seqs=4, tokens=24, drafts=0, known=None, temperature=0.0, seed=0):
    """Decodes `tokens` tokens a sequence.  known: tokens [seqs][tokens] of an earlier run, proposed `drafts` at a time.
    Returns (tokens, steps, drafts accepted)."""
    d = Decoder(seqs, tokens + drafts + 2, seed)
    g = torch.Generator().manual_seed(seed + 1)
    temp = torch.full((seqs,), temperature, device=DEV)
    got = [[] for _ in range(seqs)]
    last, steps, taken = [7 + b for b in range(seqs)], 0, 0
    while min(len(x) for x in got) < tokens:
        counts, rows = [], []
        for b in range(seqs):
            ahead = [] if known is None else known[b][len(got[b]):len(got[b]) + drafts]
            counts.append(1 + len(ahead))
            rows += [last[b]] + ahead
        u = torch.rand(len(rows), generator=g).to(DEV)
        out, accepted = d.step(torch.tensor(rows, dtype=torch.int32, device=DEV), counts, u,
                               torch.rand(seqs, generator=g).to(DEV), temp)
        out, accepted, at = out.tolist(), accepted.tolist(), 0
        for b in range(seqs):
            got[b] += out[at:at + accepted[b] + 1]
            last[b] = got[b][-1]
            if len(got[b]) >= tokens:  # a finished sequence idles in place
                got[b] = got[b][:tokens]
                d.length[b] = torch.clamp(d.length[b], max=tokens)
            at += counts[b]
        steps, taken = steps + 1, taken + sum(accepted)
    return got, steps, taken


def agreeing(a, b):
    """Tokens before the sequences' first differences."""
    return sum(next((i for i, (x, y) in enumerate(zip(s, t)) if x != y), len(s)) for s, t in zip(a, b))


def main():
    plain, steps, _ = decode()
    again, fewer, taken = decode(drafts=5, known=plain)
    total = sum(len(x) for x in plain)
    # (rows taken together round differently from rows taken alone: where two tokens are nearly as likely, they may part)
    print(f"{len(plain)} sequences x {len(plain[0])} tokens: {steps} steps one token at a time, {fewer} steps with 5 drafts "
          f"({taken} accepted); the tokens agree for {agreeing(plain, again)} of {total}")
    sampled, steps, taken = decode(drafts=5, known=plain, temperature=0.3)
    print(f"at temperature 0.3 the same drafts: {steps} steps, {taken} accepted")


if __name__ == "__main__":
    main()

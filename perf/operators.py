"""The operators around the block-quantized products of one draft-and-verify decode step, as timed cases.

One step takes the rows of all sequences at once (sequence b has rows row_start[b] .. row_start[b + 1]: its last
accepted token and the tokens drafted after it):

  embed   the rows' tokens looked up in a block-quantized table, scaled;
  attn    attention of every row over a prefix that all sequences share, then over its own sequence's paged suffix
          up to and including the row (or the drafted rows that its tree mask names);
  verify  the drafted tokens checked against the target's probabilities with given uniform numbers: the accepted
          ones, and one more token from the residual (or, all accepted, the target's) distribution.

`run` computes them in plain torch operations, or, with `own`, calls the library.  `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

HIDDEN, VOCAB = 3584, 152064  # the 7B decoder layer and its lm-head, as in the benchmark


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # One sequence, one token, a short chat history: pure latency.
        dict(name="attn_one_token", op="attn", dtype="bf16", heads=28, kv_heads=4, dim=128, seqs=1, drafts=0,
             prefix=1000, suffix=37, page=16, tree=False),
        # 16 conversations on one long system prompt, one token each.
        dict(name="attn_decode_16", op="attn", dtype="bf16", heads=28, kv_heads=4, dim=128, seqs=16, drafts=0,
             prefix=8192, suffix=500, page=16, tree=False),
        # Draft trees over an odd prefix, 64-wide heads.
        dict(name="attn_tree_odd", op="attn", dtype="f16", heads=32, kv_heads=8, dim=64, seqs=5, drafts=6,
             prefix=4099, suffix=77, page=32, tree=True),
        # Short shared instructions, long answers of their own; 80-wide heads, one query head to a key head.
        dict(name="attn_long_suffix", op="attn", dtype="f16", heads=12, kv_heads=12, dim=80, seqs=32, drafts=2,
             prefix=257, suffix=2111, page=64, tree=False),
        # 64 sequences verifying 7 drafts each on a shared document.
        dict(name="attn_verify_64", op="attn", dtype="bf16", heads=28, kv_heads=4, dim=128, seqs=64, drafts=7,
             prefix=32768, suffix=1024, page=16, tree=False),
        # One sequence, four drafts: latency of the verification.
        dict(name="verify_one", op="verify", dtype="f32", vocab=VOCAB, seqs=1, drafts=4, probs=True, greedy=False),
        # Drafts without probabilities (looked up, not sampled) in half precision; some sequences greedy.
        dict(name="verify_lookup", op="verify", dtype="bf16", vocab=50257, seqs=24, drafts=5, probs=False, greedy=True),
        # A serving batch: every sequence's seven drafts with their probabilities, fp32 logits of the lm-head product.
        dict(name="verify_64", op="verify", dtype="f32", vocab=VOCAB, seqs=64, drafts=7, probs=True, greedy=False),
        # One decode token's row of a Q4_K table.
        dict(name="embed_one", op="embed", fmt="q4_k", layout="blocks", vocab=VOCAB, cols=HIDDEN, rows=1, out="f32",
             scale=1.0),
        # The rows of a verification batch from the Q6_K table that is also the lm-head.
        dict(name="embed_drafts", op="embed", fmt="q6_k", layout="blocks", vocab=VOCAB, cols=HIDDEN, rows=511,
             out="bf16", scale=1.0),
        # A prompt's rows, scaled by the root of the width.
        dict(name="embed_prompt", op="embed", fmt="q8_0", layout="blocks", vocab=VOCAB, cols=HIDDEN, rows=16384,
             out="bf16", scale=math.sqrt(HIDDEN)),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "verify", "embed"])
    if op == "attn":
        kv_heads = rng.randint(1, 8)
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), heads=kv_heads * rng.randint(1, 8), kv_heads=kv_heads,
                 dim=rng.choice([64, 80, 96, 128, 256]), seqs=_log(rng, 1, 64), drafts=rng.randint(0, 8),
                 prefix=_log(rng, 1, 32768), suffix=_log(rng, 1, 2048), page=rng.choice([8, 16, 32, 64, 256]),
                 tree=rng.random() < 0.3)
        most = 28 * 128 * 64 * 8 * 32768 // 2
        cost = c["heads"] * c["dim"] * c["seqs"] * (c["drafts"] + 1) * (c["prefix"] + c["suffix"])
        if cost > most:
            c["prefix"] = max(1, c["prefix"] * most // cost)
        return c
    if op == "verify":
        c = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), vocab=_log(rng, 1000, VOCAB),
                 seqs=_log(rng, 1, 64), drafts=rng.randint(0, 7), probs=rng.random() < 0.6, greedy=rng.random() < 0.4)
        return c
    fmt = rng.choice(["q8_0", "q4_k", "q5_k", "q6_k", "int4_g128"])
    return dict(op=op, fmt=fmt, layout=rng.choice(["blocks", "planes"]) if fmt in ("q4_k", "q5_k", "q6_k") else "blocks",
                vocab=_log(rng, 1000, VOCAB), cols=256 * rng.randint(1, 16), rows=_log(rng, 1, 16384),
                out=rng.choice(["f32", "bf16", "f16"]), scale=rng.choice([1.0, 0.5, 59.75]))


def _rows_of(case):
    """Rows of each sequence: the last accepted token and 0 .. drafts drafted ones, ragged."""
    d = case["drafts"]
    return [1 + (d if b == 0 else d - (5 * b) % (d + 1)) for b in range(case["seqs"])]


def _suffix_of(case):
    """Suffix tokens of each sequence, its rows among them, ragged."""
    return [n + max(0, case["suffix"] - n) * ((b * 7) % 10 + 1) // 10 if b else max(n, case["suffix"])
            for b, n in enumerate(_rows_of(case))]


_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = {"q8_0": (32, 34), "q4_k": (256, 144), "q5_k": (256, 176), "q6_k": (256, 210)}
_BITS = {"q8_0": 8.5, "q4_k": 4.5, "q5_k": 5.5, "q6_k": 6.5625, "int4_g128": 4.125}


def work(case):
    """Inputs read once, outputs written once, the products' multiplications and additions."""
    if case["op"] == "attn":
        rows, suffix = _rows_of(case), _suffix_of(case)
        kv = 4 * case["kv_heads"] * case["dim"]
        nbytes = (case["prefix"] + sum(suffix)) * kv + 4 * sum(rows) * case["heads"] * case["dim"]
        pairs = sum(n * (case["prefix"] + s) for n, s in zip(rows, suffix))
        return {"bytes": nbytes, "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "verify":
        n, size = sum(_rows_of(case)), {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
        probs = case["seqs"] * case["vocab"] * 4 if case["probs"] else 0
        return {"bytes": n * case["vocab"] * size + probs, "flops": 3 * n * case["vocab"]}
    elems = case["rows"] * case["cols"]
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["out"]]
    return {"bytes": elems * (_BITS[case["fmt"]] / 8 + size), "flops": 3 * elems}


# ---- inputs ------------------------------------------------------------------

def _starts(lens, dev):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"attn": _prepare_attn, "verify": _prepare_verify, "embed": _prepare_embed}[case["op"]](case, g)
    s["case"] = case
    if own:
        s["call"] = _own_call(s)  # descriptors, outputs and workspace, as a serving loop keeps them
    return s


def _prepare_attn(case, g):
    dev, t = "cuda", _TORCH[case["dtype"]]
    rows, suffix = _rows_of(case), _suffix_of(case)
    n, h, hk, d, page = sum(rows), case["heads"], case["kv_heads"], case["dim"], case["page"]
    per = [-(-x // page) for x in suffix]
    pages = sum(per)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(t)

    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)  # pages lie in the pool as they were freed
    table = torch.zeros(case["seqs"], max(per), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    s = dict(q=normal(n, h, d) * 1.5, k_prefix=normal(case["prefix"], hk, d), v_prefix=normal(case["prefix"], hk, d),
             k_pages=normal(pages, page, hk, d), v_pages=normal(pages, page, hk, d), table=table,
             row_start=_starts(rows, dev), suffix_len=torch.tensor(suffix, dtype=torch.int32, device=dev),
             mask=None, scale=1.0 / math.sqrt(d), max_rows=max(rows), max_suffix=max(suffix))
    if case["tree"]:
        # every drafted row sees itself, the first row and the ancestors of a random earlier parent
        pick = torch.randint(0, 1 << 30, (n,), generator=g, device=dev).tolist()
        mask, r = [], 0
        for k in rows:
            seen = []
            for i in range(k):
                seen.append((seen[pick[r] % i] if i else 0) | (1 << i))
                r += 1
            mask += seen
        s["mask"] = torch.tensor(mask, dtype=torch.int64, device=dev)
    return s


def _prepare_verify(case, g):
    dev, v = "cuda", case["vocab"]
    rows = _rows_of(case)
    n, b = sum(rows), case["seqs"]
    logits = torch.randn(n, v, generator=g, device=dev) * 3.0  # about 20 likely tokens of 152064
    temp = torch.tensor([(0.7, 1.0, 1.25)[i % 3] for i in range(b)], device=dev)
    if case["greedy"]:
        temp[1::2] = 0.0
    seq = torch.repeat_interleave(torch.arange(b, device=dev), torch.tensor(rows, device=dev))
    near = logits + 0.8 * torch.randn(n, v, generator=g, device=dev)  # the draft model's view of the same rows
    probs = torch.softmax(near / torch.where(temp > 0, temp, 1.0)[seq][:, None], -1)
    if case["probs"]:
        drawn = torch.multinomial(probs, 1, generator=g)[:, 0]
    else:
        drawn = near.argmax(-1)
    tokens = torch.zeros(n, dtype=torch.int32, device=dev)
    tokens[1:] = drawn[:-1].to(torch.int32)  # the token drafted after a row is the next row's
    return dict(logits=logits.to(_TORCH[case["dtype"]]), probs=probs if case["probs"] else None, tokens=tokens,
                row_start=_starts(rows, dev), temperature=temp, max_rows=max(rows),
                u_accept=torch.rand(n, generator=g, device=dev), u_sample=torch.rand(b, generator=g, device=dev))


def _half_bytes(x):
    return x.to(torch.float16).view(torch.uint8).view(*x.shape, 2)


def _prepare_embed(case, g):
    dev, fmt, v, cols = "cuda", case["fmt"], case["vocab"], case["cols"]

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=dev) * (hi - lo) + lo

    if fmt == "int4_g128":
        codes = torch.randint(0, 256, (v * cols // 2,), generator=g, device=dev, dtype=torch.uint8)
        table = torch.cat([codes, _half_bytes(uniform(0.005, 0.05, v * cols // 128)).reshape(-1)])
    else:
        qk, size = _BLOCK[fmt]
        blocks = torch.randint(0, 256, (v * cols // qk, size), generator=g, device=dev, dtype=torch.uint8)
        if fmt == "q6_k":
            blocks[:, 208:210] = _half_bytes(uniform(0.001, 0.01, len(blocks)))
        else:
            blocks[:, 0:2] = _half_bytes(uniform(0.002, 0.02, len(blocks)))
        if fmt in ("q4_k", "q5_k"):
            blocks[:, 2:4] = _half_bytes(uniform(0.002, 0.02, len(blocks)))
        table = blocks.view(-1)
    ids = torch.randint(0, v, (case["rows"],), generator=g, device=dev).to(torch.int32)
    if case["rows"] > 8:
        ids[5::9] = -1  # rows past a sequence's accepted tokens hold no token
    return dict(table=table, ids=ids)


# ---- plain forms ---------------------------------------------------------------

def _plain_attn(s):
    c, f = s["case"], torch.float32
    n, h, hk, d, b = s["q"].shape[0], c["heads"], c["kv_heads"], c["dim"], c["seqs"]
    grp, top, page, width = h // hk, s["max_rows"], c["page"], s["max_suffix"]
    start, count = s["row_start"][:-1].long(), s["row_start"].diff().long()
    q = s["q"].to(f) * s["scale"]
    # the shared prefix: all rows of a key head as one product
    qp = q.view(n, hk, grp, d).transpose(0, 1).reshape(hk, n * grp, d)
    kp = s["k_prefix"].to(f).permute(1, 2, 0).contiguous()
    sp = torch.bmm(qp, kp).view(hk, n, grp, -1)
    # each sequence's suffix, its pages gathered, its rows padded to the longest's
    at = torch.arange(width, device=q.device)
    where = s["table"].long()[:, at // page] * page + at % page
    ks = s["k_pages"].view(-1, hk, d)[where].to(f)
    vs = s["v_pages"].view(-1, hk, d)[where].to(f)
    t = torch.arange(top, device=q.device)
    row = torch.minimum(start[:, None] + t, s["row_start"][1:, None].long() - 1)
    qs = q[row].view(b, top, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(b * hk, top * grp, d)
    ss = torch.bmm(qs, ks.permute(0, 2, 3, 1).reshape(b * hk, d, width)).view(b, hk, top, grp, width)
    slot = at - (s["suffix_len"].long() - count)[:, None]  # 0 at the sequence's first row
    if s["mask"] is None:
        seen = slot[:, None, :] <= t[:, None]
    else:
        bit = (s["mask"][row][:, :, None] >> slot.clamp(0, 63)[:, None, :]) & 1
        seen = (slot < 0)[:, None, :] | ((slot < count[:, None])[:, None, :] & (bit == 1))
    seen = seen & (at < s["suffix_len"].long()[:, None])[:, None, :]
    ss = ss.masked_fill(~seen[:, None, :, None, :], -math.inf)
    # one softmax over both
    seq = torch.bucketize(torch.arange(n, device=q.device), s["row_start"][1:].long(), right=True)
    mine = (seq, torch.arange(n, device=q.device) - start[seq])
    sr = ss.permute(0, 2, 1, 3, 4)[mine].permute(1, 0, 2, 3)  # [hk, n, grp, width]
    m = torch.maximum(sp.amax(-1), sr.amax(-1))[..., None]
    ep, er = torch.exp(sp - m), torch.exp(sr - m)
    den = ep.sum(-1) + er.sum(-1)
    op = torch.bmm(ep.view(hk, n * grp, -1), s["v_prefix"].to(f).transpose(0, 1).contiguous()).view(hk, n, grp, d)
    ms = m.permute(1, 0, 2, 3)[row].permute(0, 2, 1, 3, 4)  # [b, hk, top, grp, 1]
    es = torch.exp(ss - ms).reshape(b * hk, top * grp, width)
    os_ = torch.bmm(es, vs.transpose(1, 2).reshape(b * hk, width, d)).view(b, hk, top, grp, d)
    o = op + os_.permute(0, 2, 1, 3, 4)[mine].permute(1, 0, 2, 3)
    o = o / den[..., None]
    return o.permute(1, 0, 2, 3).reshape(n, h, d).to(s["q"].dtype)


def _plain_verify(s):
    # 64 bits: a token at the border of two intervals has to fall on the same side
    lg = s["logits"].double()
    n, v = lg.shape
    dev = lg.device
    start, end = s["row_start"][:-1].long(), s["row_start"][1:].long()
    r = torch.arange(n, device=dev)
    seq = torch.bucketize(r, end, right=True)
    temp = s["temperature"].double()
    greedy = temp == 0
    x = lg / torch.where(greedy, 1.0, temp)[seq][:, None]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    total = e.sum(-1)
    index = torch.arange(v, device=dev)
    best = torch.where(lg == lg.amax(-1, keepdim=True), index, v).amin(-1)
    drafted = s["tokens"].long().roll(-1)
    px = e.gather(1, drafted[:, None])[:, 0] / total
    qx = s["probs"].gather(1, drafted[:, None])[:, 0].double() if s["probs"] is not None else 1.0
    good = torch.where(greedy[seq], best == drafted, s["u_accept"].double() * qx < px)
    good = good & (r < end[seq] - 1)
    t = torch.arange(s["max_rows"], device=dev)
    padded = good[torch.minimum(start[:, None] + t, end[:, None] - 1)] & (start[:, None] + t < end[:, None] - 1)
    accepted = padded.long().cumprod(1).sum(1)
    a = start + accepted
    rejected = accepted < end - start - 1
    p = e[a] / total[a][:, None]
    if s["probs"] is not None:
        q = torch.where(rejected[:, None], s["probs"][a].double(), 0.0)
    else:
        q = (rejected[:, None] & (index == drafted[a][:, None])).double()
    w = torch.where(p > q, p - q, 0.0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    cum = w.cumsum(-1)
    token = (cum <= s["u_sample"].double()[:, None] * w.sum(-1, keepdim=True)).sum(-1)
    token = torch.minimum(token, torch.where(w > 0, index, 0).amax(-1))
    token = torch.where(greedy, best[a], token)
    out = torch.where(r < a[seq], drafted, torch.where(r == a[seq], token[seq], -1))
    return out.to(torch.int32), accepted.to(torch.int32)


def _six_bits(sc):
    """Scales and mins [.., 8] of the twelve bytes of a Q4_K or Q5_K block."""
    lo, mid, hi = sc[..., 0:4], sc[..., 4:8], sc[..., 8:12]
    return (torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], -1), torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], -1))


def _decode(fmt, table, ids, vocab, cols, f):
    """Rows `ids` of the packed table as numbers of type f."""
    n = len(ids)

    def half(b):
        return b.contiguous().view(torch.float16).to(f)

    if fmt == "int4_g128":
        codes = table[:vocab * cols // 2].view(vocab, -1)[ids]
        scale = half(table[vocab * cols // 2:].view(vocab, -1)[ids])
        u = torch.stack([codes & 15, codes >> 4], -1).view(n, cols // 128, 128)
        return ((u.to(f) - 8) * scale[..., None]).view(n, cols)
    qk, size = _BLOCK[fmt]
    blk = table.view(vocab, cols // qk, size)[ids]
    if fmt == "q8_0":
        return (half(blk[..., 0:2]) * blk[..., 2:].contiguous().view(torch.int8).to(f)).view(n, cols)
    if fmt == "q6_k":
        ql, qh = blk[..., 0:128].view(n, -1, 2, 1, 64), blk[..., 128:192].view(n, -1, 2, 1, 32)
        lo = torch.cat([ql & 15, ql >> 4], 3).view(n, -1, 2, 4, 32)
        hi = torch.cat([qh & 3, (qh >> 2) & 3, (qh >> 4) & 3, qh >> 6], 3)
        u = (lo | (hi << 4)).view(n, -1, 16, 16).to(f) - 32
        scale = half(blk[..., 208:210]) * blk[..., 192:208].contiguous().view(torch.int8).to(f)
        return (scale[..., None] * u).view(n, cols)
    sc, mn = _six_bits(blk[..., 4:16])
    qs = blk[..., 16 if fmt == "q4_k" else 48:].reshape(n, -1, 4, 1, 32)
    u = torch.cat([qs & 15, qs >> 4], 3).view(n, -1, 8, 32)
    if fmt == "q5_k":
        bit = torch.arange(8, device=table.device, dtype=torch.uint8)
        u = u | (((blk[..., 16:48][..., None, :] >> bit[:, None]) & 1) << 4)
    scale, low = half(blk[..., 0:2]) * sc.to(f), half(blk[..., 2:4]) * mn.to(f)
    return (scale[..., None] * u.to(f) - low[..., None]).view(n, cols)


def _plain_embed(s):
    c = s["case"]
    known = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    w = _decode(c["fmt"], s["table"], torch.where(known, s["ids"], 0).long(), c["vocab"], c["cols"], torch.float32)
    return torch.where(known[:, None], w * c["scale"], 0.0).to(_TORCH[c["out"]])


# ---- the library's calls ---------------------------------------------------------

def _own_call(s):
    from block_quantized_weight_qmv_amd import qmv
    c = s["case"]
    if c["op"] == "attn":
        out = torch.empty_like(s["q"])
        a = qmv.qmv_create_attn(s["q"], out, s["row_start"], s["max_rows"], scale=s["scale"],
                                k_prefix=s["k_prefix"], v_prefix=s["v_prefix"], k_pages=s["k_pages"],
                                v_pages=s["v_pages"], block_table=s["table"], suffix_len=s["suffix_len"],
                                max_suffix=s["max_suffix"], tree_mask=s["mask"])
        nws = qmv.qmv_attn_workspace_size(a)
        ws = torch.empty(nws, dtype=torch.uint8, device="cuda")

        def call():
            qmv.qmv_attn(a, ws, nws)
            return out
        return call
    if c["op"] == "verify":
        out = torch.empty_like(s["tokens"])
        accepted = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
        a = qmv.qmv_create_verify(s["logits"], s["tokens"], s["row_start"], s["max_rows"], s["u_accept"],
                                  s["u_sample"], out, accepted, draft_probs=s["probs"], temperature=s["temperature"])
        nws = qmv.qmv_verify_workspace_size(a)
        ws = torch.empty(nws, dtype=torch.uint8, device="cuda")

        def call():
            qmv.qmv_verify(a, ws, nws)
            return out, accepted
        return call
    w = qmv.qmv_create_weights(c["fmt"], c["vocab"], c["cols"], s["table"])
    if c["layout"] == "planes":
        planes = torch.empty(qmv.qmv_planes_size(c["fmt"], c["vocab"], c["cols"]), dtype=torch.uint8, device="cuda")
        w = qmv.qmv_repack_planes(w, planes)
    out = torch.empty(c["rows"], c["cols"], dtype=_TORCH[c["out"]], device="cuda")

    def call():
        qmv.qmv_embed(w, s["ids"], c["rows"], out, c["out"], c["scale"])
        return out
    return call


def run(state):
    if own:
        return state["call"]()
    return {"attn": _plain_attn, "verify": _plain_verify, "embed": _plain_embed}[state["case"]["op"]](state)


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "attn":
        return _exact_attn(case, _prepare_attn(case, g))
    if case["op"] == "verify":
        return _exact_verify(case, _prepare_verify(case, g))
    return _exact_embed(case, _prepare_embed(case, g))


def _exact_attn(case, s):
    """Sequence by sequence, key head by key head: softmax(q . k) v over the keys that each row sees."""
    grp, page = case["heads"] // case["kv_heads"], case["page"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, length) in enumerate(zip(_rows_of(case), _suffix_of(case))):
        used = s["table"][b, :-(-length // page)].long()
        own_k = s["k_pages"][used].flatten(0, 1)[:length]
        own_v = s["v_pages"][used].flatten(0, 1)[:length]
        sees = torch.ones(n, case["prefix"] + length, dtype=torch.bool, device="cuda")
        for i in range(n):
            for j in range(n):
                ok = j <= i if s["mask"] is None else bool((int(s["mask"][first + i]) >> j) & 1)
                sees[i, case["prefix"] + length - n + j] = ok
        for hk in range(case["kv_heads"]):
            k = torch.cat([s["k_prefix"][:, hk], own_k[:, hk]]).double()
            v = torch.cat([s["v_prefix"][:, hk], own_v[:, hk]]).double()
            q = s["q"][first:first + n, hk * grp:(hk + 1) * grp].double()
            score = (q.reshape(n * grp, -1) @ k.T.contiguous() * s["scale"]).view(n, grp, -1)
            p = torch.softmax(score.masked_fill(~sees[:, None, :], -math.inf), -1)
            out[first:first + n, hk * grp:(hk + 1) * grp] = (p.view(n * grp, -1) @ v).view(n, grp, -1)
        first += n
    return out


def _exact_verify(case, s):
    """Sequence by sequence and draft by draft, on the host."""
    tokens, start = s["tokens"].cpu().numpy(), s["row_start"].cpu().numpy()
    temp, ua, us = (s[k].cpu().numpy().astype(np.float64) for k in ("temperature", "u_accept", "u_sample"))
    out, accepted = np.full(len(tokens), -1, np.int32), np.zeros(case["seqs"], np.int32)

    def target(r, t):
        row = s["logits"][r].cpu().double().numpy()
        if t == 0:
            p = np.zeros(len(row))
            p[int(np.flatnonzero(row == row.max())[0])] = 1.0
            return p
        p = np.exp((row - row.max()) / t)
        return p / p.sum()

    for b in range(case["seqs"]):
        for r in range(start[b], start[b + 1]):
            p, rest = target(r, temp[b]), None
            if r + 1 < start[b + 1]:
                x = int(tokens[r + 1])
                if temp[b] == 0 or s["probs"] is None:
                    q = np.zeros(len(p))
                    q[x] = 1.0
                else:
                    q = s["probs"][r].cpu().numpy().astype(np.float64)
                if ua[r] * q[x] < p[x]:
                    out[r] = x
                    accepted[b] += 1
                    continue
                rest = np.maximum(p - q, 0.0)
            w = p if rest is None or rest.sum() == 0 else rest
            cum = np.cumsum(w)
            out[r] = min(int(np.searchsorted(cum, us[b] * cum[-1], side="right")), int(np.flatnonzero(w)[-1]))
            break
    return torch.from_numpy(out), torch.from_numpy(accepted)


def _exact_embed(case, s):
    """Block by block from the byte maps, on the host; every distinct token once."""
    fmt, v, cols = case["fmt"], case["vocab"], case["cols"]
    ids = s["ids"].cpu().numpy()
    uniq, back = np.unique(np.where(ids >= 0, ids, 0), return_inverse=True)
    take = torch.from_numpy(uniq).to("cuda").long()
    if fmt == "int4_g128":
        codes = s["table"][:v * cols // 2].view(v, -1)[take].cpu().numpy()
        scale = s["table"][v * cols // 2:].view(v, -1)[take].cpu().numpy().view(np.float16).astype(np.float64)
        w = np.empty((len(uniq), cols))
        w[:, 0::2], w[:, 1::2] = (codes & 15).astype(np.float64) - 8, (codes >> 4).astype(np.float64) - 8
        w *= np.repeat(scale, 128, axis=1)
    else:
        qk, size = _BLOCK[fmt]
        blk = s["table"].view(v, cols // qk, size)[take].cpu().numpy()
        byte = blk.astype(np.int64)
        num = lambda a, t: np.ascontiguousarray(a).view(t).astype(np.float64)[..., 0]  # noqa: E731
        w = np.empty((len(uniq), cols // qk, qk))
        for i in range(qk):
            if fmt == "q8_0":
                w[..., i] = num(blk[..., 0:2], np.float16) * num(blk[..., 2 + i:3 + i], np.int8)
            elif fmt == "q6_k":
                hf, grp, l = i // 128, i % 128 // 32, i % 32
                u = (byte[..., 64 * hf + 32 * (grp & 1) + l] >> (4 * (grp >> 1))) & 15
                u = u | (((byte[..., 128 + 32 * hf + l] >> (2 * grp)) & 3) << 4)
                w[..., i] = num(blk[..., 208:210], np.float16) * num(blk[..., 192 + i // 16:193 + i // 16], np.int8) * (u - 32)
            else:
                j, base = i // 32, 16 if fmt == "q4_k" else 48
                u = (byte[..., base + 32 * (i // 64) + i % 32] >> (4 * (j & 1))) & 15
                if fmt == "q5_k":
                    u = u | (((byte[..., 16 + i % 32] >> j) & 1) << 4)
                if j < 4:
                    sc, mn = byte[..., 4 + j] & 63, byte[..., 8 + j] & 63
                else:
                    sc = (byte[..., 8 + j] & 15) | ((byte[..., j] >> 6) << 4)
                    mn = (byte[..., 8 + j] >> 4) | ((byte[..., 4 + j] >> 6) << 4)
                w[..., i] = num(blk[..., 0:2], np.float16) * sc * u - num(blk[..., 2:4], np.float16) * mn
        w = w.reshape(len(uniq), cols)
    return torch.from_numpy(w[back.reshape(-1)] * np.float64(case["scale"]) * (ids >= 0)[:, None])

"""The operators of a feed-forward block in microscaled 4-bit floats, dense or of experts, as timed cases.

MXFP4 holds 32 consecutive numbers of a row as 4-bit floats (sign, two exponent bits, one mantissa bit: 0, .5, 1, 1.5,
2, 3, 4, 6) and one power of two for all of them (a byte: its exponent plus 127).  One block of a model runs

  norm      s = residual + scale * gate * post(block output), y = pre(s): the norms around it, with what joins them;
  quantize  activations to MXFP4 and read back (32 share the power of two that brings their largest into [4, 8));
  product   y = x W^T, W in MXFP4, x in MXFP4 or exact (fp32, fp16, bf16: the decode GEMV);
  grouped   the same for experts: rows sorted by expert, each group against its own matrix, gathered from the tokens,
            gate and up joined to silu(g) u in the epilogue or left as they are.

`run` computes them in plain torch operations, or, with `own`, calls the library.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

HIDDEN, FFN = 3584, 18944  # the 7B decoder layer of the benchmark


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # One token between attention and the feed-forward block: pure latency.
        dict(name="norm_one", op="norm", rows=1, cols=HIDDEN, dtype="bf16", out="bf16", pre="rms", post="", gate="",
             scale=1.0),
        # A prompt's rows, the block's output normed before it is added, with a residual scale.
        dict(name="norm_prompt", op="norm", rows=16384, cols=HIDDEN, dtype="bf16", out="bf16", pre="rms", post="rms",
             gate="vector", scale=0.5),
        # The rows of a verification batch.
        dict(name="quantize_step", op="quantize", rows=64, cols=HIDDEN, dtype="f32"),
        # A prompt's rows, in front of the gate and up projections.
        dict(name="quantize_prompt", op="quantize", rows=16384, cols=HIDDEN, dtype="bf16"),
        # One token through the gate projection, its activations exact.
        dict(name="gemv_one", op="product", m=1, n=FFN, k=HIDDEN, x="f32", out="f32", swiglu=False),
        # Three drafted tokens through the down projection, which is split along its long rows.
        dict(name="gemv_drafts", op="product", m=3, n=HIDDEN, k=FFN, x="f16", out="f32", swiglu=False),
        # A decode batch of 16 tokens, gate and up in one product.
        dict(name="product_step", op="product", m=16, n=FFN, k=HIDDEN, x="mxfp4", out="bf16", swiglu=True),
        # Odd sizes: a projection of 1001 outputs for 77 rows.
        dict(name="product_odd", op="product", m=77, n=1001, k=2848, x="mxfp4", out="f16", swiglu=False),
        # A prompt through one projection: the matrix cores' rate.
        dict(name="product_prompt", op="product", m=4096, n=FFN, k=HIDDEN, x="mxfp4", out="bf16", swiglu=False),
        # Eight tokens, four experts each: the experts' matrices are read for a row or two.
        dict(name="grouped_decode", op="grouped", tokens=8, top=4, experts=32, n=2560, k=HIDDEN, out="bf16", swiglu=True),
        # A short prompt's rows over unequal experts, some of them without a row; the down projection.
        dict(name="grouped_ragged", op="grouped", tokens=333, top=3, experts=24, n=1424, k=1376, out="f32",
             swiglu=False),
        # A prompt over the experts, gate and up.
        dict(name="grouped_prompt", op="grouped", tokens=4096, top=8, experts=32, n=2560, k=2048, out="bf16",
             swiglu=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo - 0.49), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "product", "product", "grouped", "grouped"])
    if op == "norm":
        c = dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 32, 8192), dtype=rng.choice(["f32", "f16", "bf16"]),
                 out=rng.choice(["f32", "f16", "bf16"]), pre=rng.choice(["rms", "layer"]),
                 post=rng.choice(["", "rms", "layer"]), gate=rng.choice(["", "vector", "rows"]),
                 scale=rng.choice([1.0, 0.5, 0.22]))
        c["rows"] = max(1, min(c["rows"], 16384 * HIDDEN // c["cols"] // 2))
        return c
    if op == "quantize":
        c = dict(op=op, rows=_log(rng, 1, 16384), cols=32 * _log(rng, 1, FFN // 32),
                 dtype=rng.choice(["f32", "f16", "bf16"]))
        c["rows"] = max(1, min(c["rows"], 16384 * HIDDEN // c["cols"] // 2))
        return c
    if op == "product" and rng.random() < 0.4:  # the decode GEMV
        return dict(op=op, m=rng.randint(1, 4), n=_log(rng, 32, FFN), k=32 * _log(rng, 1, FFN // 32),
                    x=rng.choice(["f32", "f16", "bf16"]), out="f32", swiglu=False)
    c = dict(op=op, n=_log(rng, 32, 8192), k=32 * _log(rng, 4, 256), out=rng.choice(["f32", "f16", "bf16"]),
             swiglu=rng.random() < 0.5)
    width = c["n"] * (2 if c["swiglu"] else 1) * c["k"]
    if op == "product":
        c.update(m=min(_log(rng, 1, 4096), max(1, 4096 * FFN * HIDDEN // width)), x="mxfp4")
        return c
    c.update(tokens=_log(rng, 1, 4096), top=rng.randint(1, 8), experts=_log(rng, 2, 64))
    c["experts"] = max(2, min(c["experts"], 32 * 5120 * 2048 // width))
    c["tokens"] = max(1, min(c["tokens"], 4096 * 8 * 5120 * 2048 // (c["top"] * width)))
    return c


def _counts_of(case):
    """Rows of each expert: unequal, and none for some where there are several."""
    rows, e = case["tokens"] * case["top"], case["experts"]
    share = [0.0 if e > 4 and i % 6 == 5 else 1.0 / (2 + i * 7 % e) for i in range(e)]
    counts = [int(rows * s / sum(share)) for s in share]
    i = 0
    while sum(counts) < rows:
        counts[i % e] += 1 if share[i % e] else 0
        i += 1
    return counts


_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "mxfp4": 17 / 32}


def work(case):
    """Inputs read once, outputs written once, the products' multiplications and additions."""
    if case["op"] == "norm":
        n, a, b = case["rows"] * case["cols"], _SIZE[case["dtype"]], _SIZE[case["out"]]
        return {"bytes": n * (3 * a + b + (a if case["gate"] == "rows" else 0)), "flops": 8 * n}
    if case["op"] == "quantize":  # read, written in 4 bits, read back and written as bf16
        n = case["rows"] * case["cols"]
        return {"bytes": n * (_SIZE[case["dtype"]] + 2 * _SIZE["mxfp4"] + 2), "flops": 4 * n}
    n, k = case["n"] * (2 if case["swiglu"] else 1), case["k"]
    if case["op"] == "product":
        nbytes = n * k * _SIZE["mxfp4"] + case["m"] * (k * _SIZE[case["x"]] + case["n"] * _SIZE[case["out"]])
        return {"bytes": nbytes, "flops": 2 * case["m"] * n * k}
    rows, used = case["tokens"] * case["top"], sum(1 for c in _counts_of(case) if c)
    nbytes = (used * n + case["tokens"]) * k * _SIZE["mxfp4"] + rows * case["n"] * _SIZE[case["out"]]
    return {"bytes": nbytes, "flops": 2 * rows * n * k}


# ---- inputs ------------------------------------------------------------------

def _quantized(x):
    """MXFP4 bytes of rows x [n, k]: the codes (low nibble first), then the powers' bytes."""
    n, k = x.shape
    b = x.float().view(n, k // 32, 32)
    top = b.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 125)  # top in [4, 8) * 2^e
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(b, -e[..., None])
    mag = v.abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    for border, strict in ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)):  # ties to even
        code += (mag > border) if strict else (mag >= border)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(n, k // 2, 2)
    return torch.cat([(code[..., 0] | (code[..., 1] << 4)).reshape(-1), (e + 127).to(torch.uint8).reshape(-1)])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"norm": _prepare_norm, "quantize": _prepare_quantize, "product": _prepare_product,
         "grouped": _prepare_grouped}[case["op"]](case, g)
    s["case"] = case
    if own:
        s["call"] = _own_call(s)  # descriptors and outputs, as a serving loop keeps them
    return s


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_norm(case, g):
    t, rows, cols = _TORCH[case["dtype"]], case["rows"], case["cols"]
    channel = torch.exp(0.5 * _normal(g, cols))  # some channels of a residual stream are much larger than others
    s = dict(residual=(_normal(g, rows, cols) * channel).to(t), block=(_normal(g, rows, cols) * 0.7 + 0.1).to(t))
    for name in ("pre", "post"):
        kind = case[name]
        s[name + "_weight"] = (1.0 + 0.2 * _normal(g, cols)).to(t) if kind else None
        s[name + "_bias"] = (0.1 * _normal(g, cols)).to(t) if kind == "layer" else None
    s["gate"] = None
    if case["gate"]:
        s["gate"] = _normal(g, *((cols,) if case["gate"] == "vector" else (rows, cols))).to(t)
    return s


def _prepare_quantize(case, g):
    x = _normal(g, case["rows"], case["cols"]) * torch.exp(0.5 * _normal(g, case["cols"]))
    return dict(x=x.to(_TORCH[case["dtype"]]))


def _weights(g, rows, k):
    out = torch.empty(rows * k * 17 // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)
    for r in range(0, rows, step):
        part = _quantized(_normal(g, min(step, rows - r), k) * 0.03)
        n = min(step, rows - r)
        out[r * k // 2:(r + n) * k // 2] = part[:n * k // 2]
        out[rows * k // 2 + r * k // 32:rows * k // 2 + (r + n) * k // 32] = part[n * k // 2:]
    return out


def _activations(g, rows, k):
    return _normal(g, rows, k) * torch.exp(0.5 * _normal(g, k))


def _prepare_product(case, g):
    m, n, k = case["m"], case["n"] * (2 if case["swiglu"] else 1), case["k"]
    x = _activations(g, m, k)
    return dict(w=_weights(g, n, k), x=_quantized(x) if case["x"] == "mxfp4" else x.to(_TORCH[case["x"]]))


def _prepare_grouped(case, g):
    n, k, e, tokens = case["n"] * (2 if case["swiglu"] else 1), case["k"], case["experts"], case["tokens"]
    counts = _counts_of(case)
    order = torch.randperm(tokens * case["top"], generator=g, device="cuda")
    start = [sum(counts[:i]) for i in range(e + 1)]
    return dict(w=_weights(g, e * n, k), x=_quantized(_activations(g, tokens, k)), counts=counts,
                index=(order % tokens).to(torch.int32), start=torch.tensor(start, dtype=torch.int32, device="cuda"))


# ---- plain forms ---------------------------------------------------------------

def _plain_norm(s):
    c = s["case"]

    def norm(x, kind, weight, bias):
        if kind == "layer":
            x = x - x.mean(-1, keepdim=True)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        return x + bias.float() if bias is not None else x

    b = s["block"].float()
    if c["post"]:
        b = norm(b, c["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        b = b * s["gate"].float()
    total = s["residual"].float() + c["scale"] * b
    y = norm(total, c["pre"], s["pre_weight"], s["pre_bias"])
    return total.to(s["residual"].dtype), y.to(_TORCH[c["out"]])


def _plain_quantize(s):
    x = s["x"].float()
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 125)
    v = torch.ldexp(b, -e)
    # steps of a half below 2, of one below 4, of two above; torch.round takes halves to even
    mag = v.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / step) * step, -6.0, 6.0)
    return torch.ldexp(v, e).view(x.shape).to(torch.bfloat16)


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decoded(data, rows, k, first=0, last=None):
    """Rows first .. last of a packed tensor, in 32 bits."""
    last = rows if last is None else last
    codes = data[first * k // 2:last * k // 2]
    powers = data[rows * k // 2 + first * k // 32:rows * k // 2 + last * k // 32]
    table = torch.tensor(_VALUES, device=data.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(-1, 32)
    return (v * torch.exp2(powers.float() - 127.0)[:, None]).view(last - first, k)


def _joined(y, swiglu):
    if not swiglu:
        return y
    g, u = y.chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_product(s):
    c = s["case"]
    n = c["n"] * (2 if c["swiglu"] else 1)
    x = _decoded(s["x"], c["m"], c["k"]) if c["x"] == "mxfp4" else s["x"].float()
    return _joined(x @ _decoded(s["w"], n, c["k"]).T, c["swiglu"]).to(_TORCH[c["out"]])


def _plain_grouped(s):
    c = s["case"]
    n, k = c["n"] * (2 if c["swiglu"] else 1), c["k"]
    x = _decoded(s["x"], c["tokens"], k)[s["index"].long()]
    y = torch.empty(len(x), c["n"], dtype=_TORCH[c["out"]], device=x.device)
    r = 0
    for e, count in enumerate(s["counts"]):
        if count:
            w = _decoded(s["w"], c["experts"] * n, k, e * n, (e + 1) * n)
            y[r:r + count] = _joined(x[r:r + count] @ w.T, c["swiglu"]).to(y.dtype)
            r += count
    return y


# ---- the library's calls ---------------------------------------------------------

def _own_call(s):
    from block_quantized_weight_qmv_amd import qmv
    c = s["case"]
    if c["op"] == "norm":
        total = torch.empty_like(s["residual"])
        y = torch.empty(c["rows"], c["cols"], dtype=_TORCH[c["out"]], device="cuda")
        a = qmv.qmv_create_norm(s["residual"], y, pre=c["pre"], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"],
                                block=s["block"], post=c["post"] or None, post_weight=s["post_weight"],
                                post_bias=s["post_bias"], gate=s["gate"], scale=c["scale"], sum_out=total, eps=1e-6)

        def call():
            qmv.qmv_norm(a)
            return total, y
        return call
    if c["op"] == "quantize":
        packed = torch.empty(qmv.qmv_packed_size("mxfp4", c["rows"], c["cols"]), dtype=torch.uint8, device="cuda")
        w = qmv.qmv_create_weights("mxfp4", c["rows"], c["cols"], packed)
        out = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device="cuda")

        def call():
            qmv.qmv_quantize(w, s["x"])
            qmv.qmv_dequant(w, out, "bf16")
            return out
        return call
    n, k = c["n"] * (2 if c["swiglu"] else 1), c["k"]
    if c["op"] == "product":
        w = qmv.qmv_create_weights("mxfp4", n, k, s["w"])
        y = torch.empty(c["m"], c["n"], dtype=_TORCH[c["out"]], device="cuda")
        if c["x"] != "mxfp4":
            def call():
                qmv.qmv_gemv("mxfp4", w, s["x"], c["x"], y, n, k, c["m"])
                return y
            return call
        a = qmv.qmv_create_mx4(w, qmv.qmv_create_weights("mxfp4", c["m"], k, s["x"]), y, swiglu=c["swiglu"])
    else:
        w = qmv.qmv_create_weights("mxfp4", c["experts"] * n, k, s["w"])
        x = qmv.qmv_create_weights("mxfp4", c["tokens"], k, s["x"])
        y = torch.empty(c["tokens"] * c["top"], c["n"], dtype=_TORCH[c["out"]], device="cuda")
        a = qmv.qmv_create_mx4(w, x, y, swiglu=c["swiglu"], expert_start=s["start"], x_index=s["index"])

    def call():
        qmv.qmv_mx4_gemm(a)
        return y
    return call


def run(state):
    if own:
        return state["call"]()
    return {"norm": _plain_norm, "quantize": _plain_quantize, "product": _plain_product,
            "grouped": _plain_grouped}[state["case"]["op"]](state)


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm":
        return _exact_norm(case, _prepare_norm(case, g))
    if case["op"] == "quantize":
        return _exact_quantize(_prepare_quantize(case, g))
    if case["op"] == "product":
        return _exact_product(case, _prepare_product(case, g))
    return _exact_grouped(case, _prepare_grouped(case, g))


def _exact_norm(case, s):
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def norm(x, name):
        if case[name] == "rms":
            return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * d[name + "_weight"]
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        return (x - mean) / torch.sqrt(var + 1e-6) * d[name + "_weight"] + d[name + "_bias"]

    block = norm(d["block"], "post") if case["post"] else d["block"]
    total = d["residual"] + case["scale"] * d.get("gate", 1.0) * block
    return total, norm(total, "pre")


def _exact_quantize(s):
    """The nearest of the sixteen values, found by search: of two as near, the one with an even code."""
    x = s["x"].double()
    out = torch.empty_like(x)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    for r in range(0, len(x), 1024):
        b = x[r:r + 1024].reshape(-1, 32)
        top = b.abs().amax(-1, keepdim=True)
        power = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - 2.0, min=-127.0))
        mag = b.abs() / power
        hi = torch.searchsorted(grid, mag.contiguous()).clamp(1, 7)  # grid[hi - 1] < mag <= grid[hi], or the ends
        lo = hi - 1
        dl, dh = mag - grid[lo], grid[hi] - mag
        pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        out[r:r + 1024] = (torch.sign(b) * grid[pick] * power).view(-1, x.shape[1])
    return out


def _exact_decoded(data, rows, k, first, last):
    codes = data[first * k // 2:last * k // 2].long()
    u = torch.stack([codes % 16, codes // 16], -1).view(-1)
    e, m = (u % 8) // 2, (u % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1.0))
    power = data[rows * k // 2 + first * k // 32:rows * k // 2 + last * k // 32].double() - 127.0
    w = torch.where(u >= 8, -mag, mag).view(-1, 32) * torch.exp2(power)[:, None]
    return w.view(last - first, k)


def _exact_rows(x, data, rows, k, first, last):
    """x times rows first .. last, some of them at a time."""
    step = max(1, (1 << 26) // k)
    return torch.cat([x @ _exact_decoded(data, rows, k, r, min(last, r + step)).T for r in range(first, last, step)], -1)


def _exact_joined(y, n, swiglu):
    return y if not swiglu else y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]


def _exact_product(case, s):
    m, n, k = case["m"], case["n"] * (2 if case["swiglu"] else 1), case["k"]
    x = _exact_decoded(s["x"], m, k, 0, m) if case["x"] == "mxfp4" else s["x"].double()
    return _exact_joined(_exact_rows(x, s["w"], n, k, 0, n), case["n"], case["swiglu"])


def _exact_grouped(case, s):
    n, k = case["n"] * (2 if case["swiglu"] else 1), case["k"]
    tokens = _exact_decoded(s["x"], case["tokens"], k, 0, case["tokens"])
    start = s["start"].tolist()
    parts = []
    for e in range(case["experts"]):
        if start[e + 1] > start[e]:
            x = tokens[s["index"][start[e]:start[e + 1]].long()]
            y = _exact_rows(x, s["w"], case["experts"] * n, k, e * n, (e + 1) * n)
            parts.append(_exact_joined(y, case["n"], case["swiglu"]))
    return torch.cat(parts)

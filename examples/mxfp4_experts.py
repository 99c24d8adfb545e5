"""A feed-forward block of experts in MXFP4: the library's operators as one layer uses them.

    python examples/mxfp4_experts.py

Random weights.  The block's input (a residual stream and what attention adds to it) goes through

    qmv_norm       residual + attention's output, normed
    qmv_quantize   to MXFP4
    qmv_mx4_gemm   every row's experts: gate and up, joined to silu(g) u
    qmv_quantize   again
    qmv_mx4_gemm   down
    qmv_norm       the experts' sum normed, scaled, added to the residual, and normed for the next block

(the router's choice, the order by expert and the weighted sum are torch operations here), and nothing returns to the
host.  The same weights also serve one token exactly, without quantizing its activations: qmv_gemv over the experts that
it takes.  The program says how far the MXFP4 block is from 64-bit arithmetic on the weights as they were.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_weight_qmv_amd import qmv  # noqa: E402

DEV, T = "cuda:0", torch.bfloat16


def quantized(x):
    """x [rows, cols] on the GPU as an MXFP4 tensor."""
    buf = torch.empty(qmv.qmv_packed_size("mxfp4", *x.shape), dtype=torch.uint8, device=DEV)
    w = qmv.qmv_create_weights("mxfp4", x.shape[0], x.shape[1], buf)
    qmv.qmv_quantize(w, x)
    return w


def dense(w):
    out = torch.empty(w.rows, w.cols, device=DEV)
    qmv.qmv_dequant(w, out, "f32")
    return out


class Block:
    def __init__(self, hidden=512, width=384, experts=8, top=2, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=DEV) * scale

        self.hidden, self.width, self.experts, self.top = hidden, width, experts, top
        # each expert's gate rows, then its up rows; and its down rows
        self.given = (normal(experts * 2 * width, hidden, scale=hidden**-0.5), normal(experts * hidden, width, scale=width**-0.5))
        self.gate_up, self.down = (quantized(w) for w in self.given)
        self.router = normal(experts, hidden, scale=hidden**-0.5)
        self.norms = [1.0 + 0.1 * normal(hidden) for _ in range(3)]

    def route(self, x):
        """Rows by expert: (token of each row, expert_start, row of each token's choices, their weights)."""
        p, chosen = torch.softmax(x.float() @ self.router.T, -1).topk(self.top, -1)
        order = torch.argsort(chosen.reshape(-1), stable=True)
        back = torch.empty_like(order)
        back[order] = torch.arange(len(order), device=DEV)
        start = torch.searchsorted(chosen.reshape(-1)[order].contiguous(), torch.arange(self.experts + 1, device=DEV))
        return (order // self.top).to(torch.int32), start.to(torch.int32), back.view(-1, self.top), p / p.sum(-1, keepdim=True)

    def __call__(self, residual, attended, route=None):
        """(new residual, normed input of the next block, what went between) of rows [n, hidden] in bf16."""
        n = len(residual)
        x, middle = torch.empty_like(residual), torch.empty_like(residual)
        qmv.qmv_norm(qmv.qmv_create_norm(residual, x, pre="rms", pre_weight=self.norms[0], block=attended, sum_out=middle))
        token, start, rows, weight = self.route(x) if route is None else route
        xq = quantized(x)
        h = torch.empty(n * self.top, self.width, dtype=T, device=DEV)
        qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(self.gate_up, xq, h, swiglu=True, expert_start=start, x_index=token))
        hq = quantized(h)
        y = torch.empty(n * self.top, self.hidden, dtype=torch.float32, device=DEV)
        qmv.qmv_mx4_gemm(qmv.qmv_create_mx4(self.down, hq, y, expert_start=start))
        out = (y[rows] * weight[..., None]).sum(1).to(T)
        total, nxt = torch.empty_like(residual), torch.empty_like(residual)
        qmv.qmv_norm(qmv.qmv_create_norm(middle, nxt, pre="rms", pre_weight=self.norms[1], block=out, post="rms",
                                         post_weight=self.norms[2], scale=0.5, sum_out=total))
        return total, nxt, dict(x=x, middle=middle, xq=xq, h=h, hq=hq, y=y, out=out, token=token, start=start, rows=rows,
                                weight=weight)

    def one_token(self, x, chosen):
        """The chosen experts' outputs [len(chosen), hidden] for one row x, whose numbers enter the products exactly."""
        out = torch.empty(len(chosen), self.hidden, device=DEV)
        per, pd = self.width * self.hidden, self.hidden * self.width
        up_codes, up_scales = self.gate_up.owner[:self.gate_up.scales_offset], self.gate_up.owner[self.gate_up.scales_offset:]
        dn_codes, dn_scales = self.down.owner[:self.down.scales_offset], self.down.owner[self.down.scales_offset:]

        def part(codes, scales, i, size, rows, cols):  # matrix i of a tensor as one of its own
            data = torch.cat([codes[i * size // 2:(i + 1) * size // 2], scales[i * size // 32:(i + 1) * size // 32]])
            return qmv.qmv_create_weights("mxfp4", rows, cols, data)

        for k, e in enumerate(chosen):
            gate = part(up_codes, up_scales, 2 * e, per, self.width, self.hidden)
            up = part(up_codes, up_scales, 2 * e + 1, per, self.width, self.hidden)
            h = torch.empty(1, self.width, device=DEV)
            qmv.qmv_gemv_swiglu("mxfp4", gate, up, x, x.dtype, h, self.width, self.hidden, 1)
            qmv.qmv_gemv("mxfp4", part(dn_codes, dn_scales, e, pd, self.hidden, self.width), h, "f32", out[k:k + 1],
                         self.hidden, self.width, 1)
        return out


def main():
    b = Block()
    g = torch.Generator(device=DEV).manual_seed(1)
    residual, attended = (torch.randn(200, b.hidden, generator=g, device=DEV).to(T) for _ in range(2))
    _, _, s = b(residual, attended)
    gate_up, down = (w.double().view(b.experts, -1, w.shape[1]) for w in b.given)
    x = s["x"].double()
    want = torch.empty(len(s["token"]), b.hidden, dtype=torch.float64, device=DEV)
    for e, (first, end) in enumerate(zip(s["start"].tolist(), s["start"].tolist()[1:])):
        gt, u = (x[s["token"][first:end].long()] @ gate_up[e].T).chunk(2, -1)
        want[first:end] = (gt * torch.sigmoid(gt) * u) @ down[e].T
    err = (s["y"].double() - want).norm() / want.norm()
    print(f"{len(residual)} rows over {b.experts} experts, {b.top} each: the experts' outputs are {err.item():.3f} of their "
          f"norm from 64-bit arithmetic with the weights and activations as they were")
    chosen = [0, 3]
    y = b.one_token(s["x"][:1].contiguous(), chosen)
    for k, e in enumerate(chosen):
        gt, u = (x[:1] @ gate_up[e].T).chunk(2, -1)
        ref = (gt * torch.sigmoid(gt) * u) @ down[e].T
        print(f"one token through expert {e}, its activations exact: {((y[k] - ref[0]).norm() / ref.norm()).item():.3f}")


if __name__ == "__main__":
    main()

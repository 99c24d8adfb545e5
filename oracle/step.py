"""Float64 definitions of the operators around the products of a draft-and-verify step.

Plain loops over rows, heads and sequences, straight from the definitions in
include/qmv.h; no code shared with the GPU path.
"""
from __future__ import annotations

import numpy as np


def embed64(dense: np.ndarray, ids, scale: float) -> np.ndarray:
    """scale * W[ids] with zero rows for ids outside the table (dense: [rows][cols] float32 weights)."""
    out = np.zeros((len(ids), dense.shape[1]))
    for i, t in enumerate(ids):
        if 0 <= t < dense.shape[0]:
            out[i] = dense[t].astype(np.float64) * np.float64(np.float32(scale))
    return out


def _place(row, row_start):
    for b in range(len(row_start) - 1):
        if row_start[b] <= row < row_start[b + 1]:
            return b
    return None


def attn64(q, row_start, scale, k_prefix=None, v_prefix=None, prefix_pages=None, prefix_len=0, k_pages=None,
           v_pages=None, block_table=None, suffix_len=None, tree_mask=None):
    """Attention of every row in float64.  Arrays as in qmv_attn ([row][head][D] and so on).

    Returns (out, lse, mag, smax): mag[row][head][d] = sum_j p_j |v_j| / sum_j p_j and smax[row][head] =
    max_j scale * sum_d |q k_j|, from which the tests derive their tolerances."""
    q = q.astype(np.float64)
    rows, heads, d = q.shape
    kv = k_prefix if k_prefix is not None else k_pages
    hk = kv.shape[-2]
    out, mag = np.zeros((rows, heads, d)), np.zeros((rows, heads, d))
    lse, smax = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    page = k_pages.shape[1] if k_pages is not None else 1

    def paged(table, length):
        ok, ks, vs = [], [], []
        for j in range(length):
            p = int(table[j // page])
            good = 0 <= p < k_pages.shape[0]
            ok.append(good)
            ks.append(k_pages[p if good else 0, j % page])
            vs.append(v_pages[p if good else 0, j % page])
        return ok, ks, vs

    prefix = [], [], []
    if prefix_pages is not None:
        prefix = paged(prefix_pages, prefix_len)
    elif k_prefix is not None:
        prefix = [True] * len(k_prefix), list(k_prefix), list(v_prefix)
    suffixes = {}
    for r in range(rows):
        b = _place(r, row_start)
        ok, ks, vs = (list(x) for x in prefix)
        if b is not None and suffix_len is not None:
            n, length = row_start[b + 1] - row_start[b], max(0, int(suffix_len[b]))
            if b not in suffixes:
                suffixes[b] = paged(block_table[b], length)
            sok, sk, sv = suffixes[b]
            for j in range(length):
                slot = j - (length - int(n))
                if slot < 0:
                    seen = True
                elif tree_mask is not None:
                    seen = bool((int(tree_mask[r]) >> slot) & 1)
                else:
                    seen = slot <= r - row_start[b]
                ok.append(sok[j] and seen)
            ks, vs = ks + sk, vs + sv
        ok = np.array(ok, dtype=bool)
        if not ok.any():
            continue
        kk = np.array(ks)[ok].astype(np.float64)
        vv = np.array(vs)[ok].astype(np.float64)
        for h in range(heads):
            g = h // (heads // hk)
            prod = kk[:, g] * q[r, h]
            s = scale * prod.sum(-1)
            smax[r, h] = scale * np.abs(prod).sum(-1).max()
            m = s.max()
            p = np.exp(s - m)
            out[r, h] = (p[:, None] * vv[:, g]).sum(0) / p.sum()
            mag[r, h] = (p[:, None] * np.abs(vv[:, g])).sum(0) / p.sum()
            lse[r, h] = m + np.log(p.sum())
    return out, lse, mag, smax


def verify64(logits, tokens, row_start, u_accept, u_sample, draft_probs=None, temperature=None):
    """Rejection sampling of drafts in float64.  Returns (out_tokens, accepted, margin): margin[b] is the smallest
    distance of sequence b's comparisons from equality, relative to the sums compared."""
    logits = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    rows, v = logits.shape
    nseq = len(row_start) - 1
    out, accepted = np.full(rows, -1, np.int32), np.zeros(nseq, np.int32)
    margin = np.ones(nseq)
    for b in range(nseq):
        t = 1.0 if temperature is None else float(temperature[b])
        greedy = not t > 0
        for r in range(row_start[b], row_start[b + 1]):
            row, last = logits[r], r + 1 == row_start[b + 1]
            top = row.max()
            if top == -np.inf:
                break
            if greedy:
                p = np.zeros(v)
                p[int(np.flatnonzero(row == top)[0])] = 1.0
            elif top == np.inf:
                p = (row == np.inf).astype(np.float64)
            else:
                p = np.exp((row - top) / t)
            p = p / p.sum()
            w = p
            if not last:
                x = int(tokens[r + 1])
                known = 0 <= x < v
                if greedy or draft_probs is None:
                    q = np.zeros(v)
                    if known:
                        q[x] = 1.0
                else:
                    q = draft_probs[r].astype(np.float64)
                    q = np.where(q > 0, q, 0.0)
                if known:
                    lhs = float(u_accept[r]) * q[x] if not greedy else 0.0
                    if lhs < p[x]:
                        if p[x] > 0 and not greedy:
                            margin[b] = min(margin[b], abs(lhs - p[x]) / max(lhs, p[x]))
                        out[r] = x
                        accepted[b] += 1
                        continue
                    if not greedy and lhs > 0:
                        margin[b] = min(margin[b], abs(lhs - p[x]) / lhs)
                w = np.maximum(p - q, 0.0)
                if w.sum() == 0:
                    w = p
            cum = np.cumsum(w)
            goal = float(u_sample[b]) * cum[-1]
            some = np.flatnonzero(w)
            out[r] = min(int(np.searchsorted(cum, goal, side="right")), int(some[-1]))
            if not greedy and len(some) > 1:
                margin[b] = min(margin[b], np.abs(cum[some[:-1]] - goal).min() / cum[-1])
            break
    return out, accepted, margin

"""Pins of oracle/step.py: against values worked out by hand, torch's softmax in float64, and the statement that
rejection sampling returns the target's distribution."""
import numpy as np
import torch

from oracle.step import attn64, embed64, verify64


def test_embed_by_hand():
    w = np.array([[1.0, 2.0], [3.0, -4.0]], np.float32)
    got = embed64(w, [1, -1, 0, 2], 0.5)
    assert np.array_equal(got, [[1.5, -2.0], [0, 0], [0.5, 1.0], [0, 0]])


def test_attention_by_hand():
    # one row; scores 0 and log 3 (prefix), log 4 (suffix): weights 1/8, 3/8, 4/8
    q = np.ones((1, 1, 1))
    k = np.log(np.array([1.0, 3.0])).reshape(2, 1, 1)
    pages = np.zeros((2, 2, 1, 1))
    pages[1, 0] = np.log(4.0)
    vp = np.array([8.0, 16.0]).reshape(2, 1, 1)
    vpages = np.full((2, 2, 1, 1), np.nan)
    vpages[1, 0] = -2.0
    out, lse, mag, _ = attn64(q, [0, 1], 1.0, k, vp, k_pages=pages, v_pages=vpages, block_table=[[1]],
                              suffix_len=[1])
    assert np.allclose(out, 1.0 + 6.0 - 1.0) and np.allclose(lse, np.log(8.0)) and np.allclose(mag, 8.0)


def test_attention_against_softmax_and_masks():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(4, 4, 8)), rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8))
    kp, vp = rng.normal(size=(4, 2, 2, 8)), rng.normal(size=(4, 2, 2, 8))
    table, lens, start = [[2, 0], [3, 7]], [4, 3], [0, 2, 3]  # page 7 does not exist; row 3 is outside
    mask = [0b01, 0b10, 0b0, 0b1]
    for tree in (None, mask):
        out, lse, _, _ = attn64(q, start, 0.3, k, v, k_pages=kp, v_pages=vp, block_table=table, suffix_len=lens,
                                tree_mask=tree)
        for r, seen in enumerate([[0, 1, 2], [0, 1, 2, 3] if tree is None else [0, 1, 3],
                                  [0, 1], None]):
            for h in range(4):
                kk, vv = [k[:, h // 2]], [v[:, h // 2]]
                if seen is not None:
                    b = 0 if r < 2 else 1
                    flat_k = np.concatenate([kp[t] for t in table[b] if t < 4])[:, h // 2]
                    flat_v = np.concatenate([vp[t] for t in table[b] if t < 4])[:, h // 2]
                    kk.append(flat_k[seen]), vv.append(flat_v[seen])
                s = torch.from_numpy(np.concatenate(kk) @ q[r, h] * 0.3)
                want = torch.softmax(s, 0).numpy() @ np.concatenate(vv)
                assert np.allclose(out[r, h], want) and np.isclose(lse[r, h], torch.logsumexp(s, 0).item())
    out, lse, _, _ = attn64(q[:1], [0, 1], 1.0, k_pages=kp, v_pages=vp, block_table=[[9]], suffix_len=[1])
    assert not out.any() and np.all(np.isneginf(lse))


def test_verify_by_hand():
    # p = (.5, .25, .25); draft token 1 with q = (0, .75, .25): accepted below 1/3, else from (.5, 0, 0)
    logits = np.log(np.array([[2.0, 1.0, 1.0], [1.0, 1.0, 2.0]]))
    q = np.array([[0.0, 0.75, 0.25], [9.0, 9.0, 9.0]], np.float32)
    for u, us, want, acc in [(0.33, 0.3, [1, 1], 1), (0.33, 0.2, [1, 0], 1), (0.33, 0.51, [1, 2], 1),
                             (0.34, 0.99, [0, -1], 0)]:
        out, accepted, _ = verify64(logits, [7, 1], [0, 2], [u, 0], [us], q)
        assert list(out) == want and list(accepted) == [acc]
    # greedy: ties to the lowest index; a draft outside the vocabulary
    out, accepted, _ = verify64(np.array([[1.0, 3.0, 3.0], [5.0, 0, 0]]), [0, 1], [0, 2], [0, 0], [0.9], None, [0.0])
    assert list(out) == [1, 0] and accepted[0] == 1
    out, accepted, _ = verify64(logits, [0, 3], [0, 2], [0, 0], [0.6], q)
    assert list(out) == [0, -1] and accepted[0] == 0
    out, accepted, _ = verify64(np.full((1, 3), -np.inf), [0], [0, 1], [0], [0.5])
    assert list(out) == [-1] and accepted[0] == 0


def test_verification_returns_the_targets_distribution():
    rng = np.random.default_rng(1)
    logits = rng.normal(size=(2, 6))
    p = np.exp(logits[0]) / np.exp(logits[0]).sum()
    q = rng.random(6)
    q = (q / q.sum()).astype(np.float32)
    n, counts = 20000, np.zeros(6)
    drafts = rng.choice(6, n, p=q.astype(np.float64) / q.sum(dtype=np.float64))
    for i in range(n):
        out, _, _ = verify64(logits, [0, drafts[i]], [0, 2], rng.random(2), rng.random(1), np.stack([q, q]))
        counts[out[0]] += 1
    # five standard deviations of a binomial count
    assert np.all(np.abs(counts - n * p) < 5 * np.sqrt(n * p * (1 - p)))

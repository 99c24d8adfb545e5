"""examples/draft_and_verify.py: lookup, products, attention and verification as one decode step runs them."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_tokens_decoded_one_by_one_are_accepted_as_drafts():
    import draft_and_verify as ex
    plain, steps, _ = ex.decode(seqs=3, tokens=8)
    assert steps == 8 and all(len(set(x)) > 2 for x in plain)  # not one token over and over
    again, fewer, taken = ex.decode(seqs=3, tokens=8, drafts=4, known=plain)
    # the only differences are between tokens of nearly one likelihood: most of each sequence agrees
    same = ex.agreeing(plain, again)
    print(same, fewer, taken)
    assert same >= 18 and fewer <= 4 and taken >= 12
    # a draft that is wrong ends its sequence's run of accepted ones there, and the right token is drawn in its place
    wrong = [list(x) for x in plain]
    wrong[0][0] = (wrong[0][0] + 1) % ex.VOCAB
    again, _, fewer_taken = ex.decode(seqs=3, tokens=8, drafts=4, known=wrong)
    assert again[0][0] == plain[0][0] and fewer_taken < taken

"""The example with drafts end to end: its logits against dense attention over
the whole history, and tokens at temperature 0 against one token at a time.

Tolerance: as for the other serving example, a dozen roundings to bfloat16 a
layer, 2^-8 of an activation each at most, come to 2^-8 sqrt(24) = 2 % of the
logits' spread.  Activations are rounded to E4M3 on both sides from values that differ by such
a rounding, so one in some 2^4 2^-8 = 6 % of them falls to the other neighbour, a step of 2^-3
at most: over 512 products sqrt(0.06 / 3) 2^-3 = 2 % of a product's spread, nine products deep at
most 2 % sqrt(9) = 6 %.  Of 12 rows times 4096 logits the largest of these errors is some 4.5 times their
spread: 4.5 (2 % + 6 %) = 36 %; half of what unrelated logits would differ by is far above.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_steps_match_dense_attention(afx):
    import draft_steps
    tokens, stood, worst = draft_steps.run(steps=6, check=True, seed=1)
    assert worst < 0.36, worst
    assert all(len(t) >= 6 and all(0 <= v < draft_steps.VOCAB for v in t) for t in tokens)
    assert sum(map(len, tokens)) == 18 + stood
    assert draft_steps.run(steps=6, seed=1)[0] == tokens


def test_no_drafts_and_many(afx):
    import draft_steps
    for drafts in (0, 7):
        tokens, stood, worst = draft_steps.run(steps=3, drafts=drafts, check=True, seed=2)
        assert worst < 0.36, worst
        assert sum(map(len, tokens)) == 9 + stood and (drafts or stood == 0)

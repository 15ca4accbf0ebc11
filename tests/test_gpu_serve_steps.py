"""The serving example end to end: its logits against dense attention over
the whole history.  Tolerance: the two differ in where float32 sums round and,
at bfloat16's 2^-9 a rounding, in the softmax weights and in which neighbour a
rounded activation falls to; a dozen such roundings a layer, two layers, on a
logit of 512 products, come to at most a few times 2^-9 * sqrt(24) = 1 % of
the logits' spread; 5 % is the bound.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_steps_match_dense_attention(afx):
    import serve_steps
    tokens, worst = serve_steps.run(steps=5, check=True, seed=1)
    assert worst < 0.05, worst
    assert all(len(t) == 5 and all(0 <= v < serve_steps.VOCAB for v in t) for t in tokens)
    assert serve_steps.run(steps=5, seed=1)[0] == tokens

"""Sampling many rows of mixed parameters, which clusters take in an order of
their own, and top-p boundaries far down flat tails of 16-bit logits, where
hundreds of tokens share a value.  Inputs and tolerances: test_gpu_sample.
"""
import numpy as np
import pytest

from test_gpu_sample import _check, _logits, _u

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [305, 511, 512, 513, 1100])
def test_rows_of_mixed_parameters_in_any_number(afx, rows):
    rng = np.random.default_rng(rows)
    _check(afx, _logits(rows, 1500, "float32", rows), _u(rows, rows), temperature=rng.choice([0.0, 0.6, 1.0, 1.3], rows).tolist(),
           top_k=rng.choice([0, 0, 5, 1200], rows).tolist(), top_p=rng.choice([0.5, 0.9, 1.0], rows).tolist())


@pytest.mark.parametrize("kind", ["greedy", "whole", "top_k"])
def test_many_rows_of_one_kind(afx, kind):
    rows = 700
    t, k = {"greedy": (0.0, 0), "whole": (1.0, 0), "top_k": (1.0, 9)}[kind]
    _check(afx, _logits(rows, 900, "bfloat16", 8), _u(rows, 8), temperature=[t] * rows, top_k=[k] * rows, top_p=[0.7] * rows)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("temperature,top_p", [(1.0, 0.9), (1.3, 0.8), (1.0, 0.999), (3.0, 0.5)])
def test_top_p_far_down_a_flat_tail(afx, dtype, temperature, top_p):
    z = _logits(4, 151_936, dtype, 12)
    z[:, 77] = 14.0
    _check(afx, z, _u(4, 12), temperature=[temperature] * 4, top_p=[top_p] * 4)


def test_large_top_k_among_ties(afx):
    z = (_logits(3, 40_000, "float32", 13) * 2).round() / 2
    _check(afx, z, _u(3, 13), top_k=[700, 1024, 1023], top_p=[0.99, 1.0, 0.6])

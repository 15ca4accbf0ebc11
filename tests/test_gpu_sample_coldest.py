"""Sampling at temperatures around and below the smallest normal float32,
where 1 / T or a histogram's steps a unit of logits leave the type's range.
Inputs and tolerances: test_gpu_sample.

Below 3e-39 a temperature counts as 3e-39; only logits that differ by less
than about 1e-36 could tell.
"""
import math

import numpy as np
import pytest

from test_gpu_sample import PARAMS, _check, _logits, _run, _u

pytestmark = pytest.mark.gpu

COLDEST = [1e-37, 2e-38, 1.2e-38, 3e-39, 2.9e-39, 1e-39, 1e-45]


@pytest.mark.parametrize("temperature", COLDEST)
@pytest.mark.parametrize("name", ["plain", "min_p", "top_k", "top_k large", "top_p", "all"])
def test_the_coldest_temperatures_give_the_maximum(afx, temperature, name):
    rows = 5
    for vocab, dtype in ((777, "bfloat16"), (40_000, "float32")):
        params = {k: [v] * rows for k, v in PARAMS[name].items()}
        params["temperature"] = [temperature] * rows
        z = _logits(rows, vocab, dtype, vocab)
        _check(afx, z, _u(rows, 9), **params)
        assert (z.float().amax(1).cpu().numpy() == z.float().cpu().numpy()[range(rows), _run(afx, z, _u(rows, 3), **params)[0]]).all()


@pytest.mark.parametrize("temperature", COLDEST)
def test_ties_and_infinite_logits_at_the_coldest_temperatures(afx, temperature):
    import torch
    z = torch.randn((3, 3000), device="cuda")
    z[0, 17], z[0, 2000] = math.inf, math.inf
    z[1, 5], z[1, 9] = math.inf, -math.inf
    z[2, 40], z[2, 2990] = 9.0, 9.0
    for params in ({}, {"top_k": [3] * 3}, {"top_k": [2000] * 3}, {"top_p": [0.9] * 3}, {"min_p": [0.5] * 3}):
        params["temperature"] = [temperature] * 3
        token, logprob = _run(afx, z, [0.7] * 3, **params)
        assert token == [2000, 5, 2990]
        assert np.allclose(logprob, [-math.log(2), 0, -math.log(2)], rtol=0, atol=2.0 ** -20)
        assert _run(afx, z, [0.2] * 3, **params)[0] == [17, 5, 40]


@pytest.mark.parametrize("name", ["plain", "min_p", "top_k", "top_k large", "top_p", "all"])
@pytest.mark.parametrize("temperature", [1e-37, 2e-38, 1.2e-38, 1e-38])
def test_logits_as_small_as_the_temperature(afx, temperature, name):
    """Steps of 2^-149 are 2^-23 or less of such a temperature: no rounding but float32's in y."""
    import torch
    rows = 6
    g = torch.Generator(device="cuda").manual_seed(5)
    y = torch.randn((rows, 5000), generator=g, device="cuda") * 2.0
    params = {k: [v] * rows for k, v in PARAMS[name].items()}
    params["temperature"] = [temperature] * rows
    _check(afx, y * temperature, _u(rows, 4), **params)

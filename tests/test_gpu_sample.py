"""Sampling (afx_sample) against a float64 reference, row by row.

A token has to be the reference's wherever no decision (a top-p or min-p
boundary, the draw itself) came nearer to the other side than NEAR = 2e-6 of
the mass: float32 weights are within about 2^-22 of their values and 2^-44
steps add at most 2^19 * 2^-44.  In the other rows (large vocabularies have
tokens of less mass than that) it has to be one that decisions each off by at
most NEAR lead to.  Log probabilities: float32 y has an error of
2^-23 (|y| + 1) at most, the logarithm's sum 2^-22.
"""
import math

import numpy as np
import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu

NEAR = 2e-6


def _run(afx, logits, u, logprobs=True, **params):
    import torch
    rows = logits.shape[0]
    d = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in params.items()}
    token = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    logprob = torch.full((rows,), 9.0, device="cuda") if logprobs else None
    afx.afx_sample(logits, torch.tensor(u, dtype=torch.float32, device="cuda"), token, logprobs=logprob, **d)
    torch.cuda.synchronize()
    return token.tolist(), logprob.tolist() if logprobs else None


def _check(afx, logits, u, **params):
    token, logprob = _run(afx, logits, u, **params)
    z = logits.float().cpu().numpy()
    names = {"temperature": "t", "top_k": "k", "top_p": "p", "min_p": "min_p"}
    for r in range(z.shape[0]):
        # the parameters as the kernel gets them, in float32
        kw = {names[n]: (int(v[r]) if n == "top_k" else float(np.float32(v[r]))) for n, v in params.items()}
        want, lp, sure, allows = ref.sample(z[r], float(np.float32(u[r])), near=NEAR, **kw)
        if sure:
            assert token[r] == want, (r, kw)
        if want < 0:
            assert logprob[r] == -math.inf
            continue
        if not kw.get("t", 1.0) > 0:
            assert logprob[r] == 0
            continue
        low = high = lp
        if not sure:
            assert allows(token[r]) is not None, (r, kw, token[r], want)
            low, high = allows(token[r])
        top = float(np.nanmax(z[r]))
        y = 0.0 if z[r][token[r]] == top else abs(float(z[r][token[r]]) - top) / kw.get("t", 1.0)
        slack = 2.0 ** -22 * (y + 1) + 2.0 ** -21 * (1 + abs(lp)) + 2.0 ** -25 * z.shape[1] * 2.0 ** -16
        assert low - slack <= logprob[r] <= high + slack, r


def _logits(rows, vocab, dtype, seed, spread=2.5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((rows, vocab), generator=g, device="cuda") * spread
    return z.to(getattr(torch, dtype))


def _u(rows, seed):
    return np.random.default_rng(seed).random(rows).astype(np.float32).tolist()


PARAMS = {
    "plain": {},
    "warm": {"temperature": 1.7},
    "cold": {"temperature": 0.05},
    "top_k": {"top_k": 40},
    "top_k 1": {"top_k": 1},
    "top_k large": {"top_k": 3000},
    "top_p": {"top_p": 0.9},
    "top_p small": {"top_p": 1e-6},
    "top_p 0": {"top_p": 0.0},
    "min_p": {"min_p": 0.05},
    "min_p 2": {"min_p": 2.0},
    "all": {"temperature": 0.7, "top_k": 50, "top_p": 0.9, "min_p": 0.02},
    "greedy": {"temperature": 0.0, "top_k": 5, "top_p": 0.5},
}


@pytest.mark.parametrize("name", list(PARAMS))
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 8193, 65_537, 151_936])
def test_parameters_and_vocabularies(afx, name, vocab):
    rows = 9
    _check(afx, _logits(rows, vocab, "float32", vocab), _u(rows, vocab),
           **{k: [v] * rows for k, v in PARAMS[name].items()})


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_types_with_a_parameter_set_a_row(afx, dtype):
    rng = np.random.default_rng(3)
    rows = 64
    _check(afx, _logits(rows, 50_001, dtype, 5), _u(rows, 6),
           temperature=rng.choice([0.0, 0.5, 1.0, 1.4], rows).tolist(), top_k=rng.choice([-1, 0, 1, 7, 200, 60_000], rows).tolist(),
           top_p=rng.choice([0.1, 0.7, 0.99, 1.0], rows).tolist(), min_p=rng.choice([0.0, 0.01, 0.3], rows).tolist())


@pytest.mark.parametrize("name", ["plain", "top_k", "top_p", "all", "greedy", "top_k large"])
@pytest.mark.parametrize("values", [1, 2, 5, 40])
def test_ties_go_to_the_lowest_index(afx, name, values):
    """A few distinct logits, thousands of ties at every boundary."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(values)
    z = torch.randint(0, values, (8, 30_011), generator=g, device="cuda").float() * 0.25
    _check(afx, z, _u(8, values), **{k: [v] * 8 for k, v in PARAMS[name].items()})


def test_negative_zero_ties_with_zero(afx):
    import torch
    z = torch.full((1, 10), -5.0, device="cuda")
    z[0, 3], z[0, 7] = -0.0, 0.0
    assert _run(afx, z, [0.99], top_k=[1])[0] == [3]
    assert _run(afx, z, [0.99], temperature=[0.0])[0] == [3]


def test_masked_logits(afx):
    import torch
    z = torch.randn((6, 5000), device="cuda")
    z[0, :] = -math.inf                       # nothing left
    z[1, :] = math.nan                        # nothing left either
    z[2, 1:] = -math.inf                      # one token
    z[3, ::2] = math.nan
    z[4, ::3] = torch.finfo(torch.float32).min
    z[5, 100:] = -math.inf
    for params in ({}, {"top_k": [60] * 6}, {"top_p": [0.8] * 6}, {"temperature": [0.0] * 6}, {"min_p": [0.1] * 6}):
        _check(afx, z, _u(6, 1), **params)
        token = _run(afx, z, _u(6, 2), **params)[0]
        assert token[:3] == [-1, -1, 0] and token[3] % 2 == 1 and token[4] % 3 and token[5] < 100


def test_infinite_logits(afx):
    import torch
    z = torch.randn((2, 3000), device="cuda")
    z[0, 17], z[0, 2000] = math.inf, math.inf
    z[1, 5] = math.inf
    for params in ({}, {"top_k": [3] * 2}, {"top_p": [0.9] * 2}):
        assert _run(afx, z, [0.7, 0.7], **params)[0] == [2000, 5]
        assert _run(afx, z, [0.2, 0.7], **params)[0] == [17, 5]


@pytest.mark.parametrize("temperature", [1e-30, 1.0, 1e30, math.inf])
def test_infinite_logits_at_temperatures_far_out(afx, temperature):
    import torch
    z = torch.randn((2, 3000), device="cuda")
    z[0, 17], z[0, 2000] = math.inf, math.inf
    z[1, 5], z[1, 9] = math.inf, -math.inf
    for params in ({}, {"top_k": [3] * 2}, {"top_k": [2000] * 2}, {"top_p": [0.9] * 2}, {"min_p": [0.5] * 2}):
        assert _run(afx, z, [0.7, 0.7], temperature=[temperature] * 2, **params)[0] == [2000, 5]


def test_rows_of_the_types_lowest_value(afx):
    import torch
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        z = torch.full((2, 4096), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        z[1, 9] = 1.0
        assert _run(afx, z, [0.5, 0.5])[0] == [2048, 9]
        assert _run(afx, z, [0.5, 0.5], top_k=[2, 2])[0] == [1, 9]


@pytest.mark.parametrize("temperature", [1e-30, 1e-3, 100.0, 1e30, math.inf])
@pytest.mark.parametrize("name", ["plain", "top_k", "top_p"])
def test_temperatures_far_out(afx, temperature, name):
    """Weights all alike (every token in one histogram step) or all but one gone."""
    params = {k: [v] * 4 for k, v in PARAMS[name].items()}
    params["temperature"] = [temperature] * 4
    _check(afx, _logits(4, 40_000, "float32", 8), _u(4, 9), **params)


def test_draws_at_the_ends(afx):
    import torch
    z = torch.tensor([[1.0, 2.0, 3.0, -math.inf]] * 4, device="cuda")
    assert _run(afx, z, [0.0, 1.0, 0.99999994, math.nan])[0] == [0, 2, 2, 0]


def test_strided_and_unaligned_rows(afx):
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        whole = torch.randn((5, 20_003), device="cuda").to(dtype)
        for view in (whole[:, 1:], whole[:, 8:20_000], whole[::2, 3:-1]):
            rows = view.shape[0]
            _check(afx, view, _u(rows, 4), top_p=[0.95] * rows)


def test_the_largest_vocabulary(afx):
    v = afx.AFX_SAMPLE_MAX_VOCAB
    _check(afx, _logits(2, v, "bfloat16", 1), _u(2, 1), top_p=[0.9] * 2, top_k=[100_000] * 2)


def test_many_rows(afx):
    _check(afx, _logits(700, 3001, "float32", 2), _u(700, 2), top_k=[30] * 700)


def test_frequencies_follow_the_weights(afx):
    import torch
    rows = 20_000
    z = torch.tensor([0.0, 1.0, -1.0, 2.0], device="cuda").repeat(rows, 1)
    token = np.array(_run(afx, z, _u(rows, 5), logprobs=False)[0])
    share = np.bincount(token, minlength=4) / rows
    want = np.exp([0.0, 1.0, -1.0, 2.0]) / np.exp([0.0, 1.0, -1.0, 2.0]).sum()
    assert np.all(np.abs(share - want) < 5 * np.sqrt(want * (1 - want) / rows))


def test_the_same_call_gives_the_same_tokens(afx):
    z, u = _logits(32, 151_936, "bfloat16", 3), _u(32, 3)
    first = _run(afx, z, u, top_p=[0.95] * 32, temperature=[1.5] * 32)
    for _ in range(5):
        assert _run(afx, z, u, top_p=[0.95] * 32, temperature=[1.5] * 32) == first


def test_another_stream(afx):
    import torch
    z = _logits(4, 5000, "float32", 4)
    u = torch.tensor(_u(4, 4), device="cuda")
    want = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = torch.zeros_like(want)
    afx.afx_sample(z, u, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    afx.afx_sample(z, u, got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_sampling_refuses_bad_arguments(afx):
    import torch
    z, u = torch.randn((3, 100), device="cuda"), torch.rand(3, device="cuda")
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=z.double(), u=u, tokens=t), dict(logits=z[0], u=u, tokens=t), dict(logits=z.t(), u=u, tokens=t),
                dict(logits=z, u=u[:2], tokens=t), dict(logits=z, u=None, tokens=t), dict(logits=z, u=u, tokens=t.long()),
                dict(logits=z, u=u, tokens=t, top_k=u), dict(logits=z, u=u, tokens=t, top_p=u.double()),
                dict(logits=z.cpu(), u=u, tokens=t)):
        with pytest.raises(ValueError):
            afx.afx_sample(**bad)
    with pytest.raises(afx.AfxError) as err:
        afx.afx_sample(torch.zeros((1, afx.AFX_SAMPLE_MAX_VOCAB + 1), device="cuda"), u[:1], t[:1])
    assert err.value.status == afx.AFX_E_ARG
    with pytest.raises(afx.AfxError):
        afx.afx_sample(torch.zeros((1, 100), device="cuda").expand(3, 100), u, t)  # rows on top of one another

"""Verification of drafts against a 64-bit definition.

A weight e^y has an error of |y| 2^-23 (y's two roundings) and some 2^-22 (the
exponential), |y| up to 30.5, so shares are off by at most 1e-5 relative and
sums of them by as much of the whole; decisions that the definition takes by a
margin above 3e-5 have to come out the same, and a draw has to be a token within 3e-5 (of what is left over, for a
draw from differences).  Where float32 weights may keep a token at a top-p boundary or not, its share is added.  Log
probabilities: 1e-5, that share, and the logarithm's rounding, 2^-23 of its value and a last place.
"""
import math

import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
NEAR = 3e-5


def _params(requests, seed, which="mixed"):
    rng = np.random.RandomState(seed)
    pick = {"mixed": lambda: (rng.choice([0.0, 0.5, 1.0, 1.7]), rng.choice([0, 1, 5, 40, 3000]), rng.choice([1.0, 0.5, 0.9]), rng.choice([0.0, 0.0, 0.05])),
            "plain": lambda: (1.0, 0, 1.0, 0.0), "warm": lambda: (1.2, 0, 0.95, 0.0), "greedy": lambda: (0.0, 3, 0.5, 0.1)}[which]
    rows = [pick() for _ in range(requests)]
    return {"temperature": torch.tensor([r[0] for r in rows], device="cuda", dtype=F32),
            "top_k": torch.tensor([r[1] for r in rows], device="cuda", dtype=torch.int32),
            "top_p": torch.tensor([r[2] for r in rows], device="cuda", dtype=F32),
            "min_p": torch.tensor([r[3] for r in rows], device="cuda", dtype=F32)}


def _case(counts, vocab, kind, draft_kind, seed, closeness=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(counts) + len(counts)
    z = torch.randn((n, vocab), generator=g, device="cuda") * 3
    zd = z + closeness * torch.randn((n, vocab), generator=g, device="cuda")
    starts = np.concatenate([[0], np.cumsum(np.array(counts) + 1)])
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    likely = (zd + 0.8 * torch.randn((n, vocab), generator=g, device="cuda")).argmax(1)
    some = torch.rand(n, generator=g, device="cuda") < 0.9
    tokens[1:] = torch.where(some, likely, tokens)[:-1]
    return {"logits": z.to(kind), "draft_logits": zd.to(draft_kind) if draft_kind else None, "tokens": tokens.to(torch.int32),
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "u": torch.rand(n, generator=g, device="cuda"),
            "draw_u": torch.rand(len(counts), generator=g, device="cuda")}


def _run(afx, c, params, draft_params=None, logprobs=True, extra=0, out=None):
    n, requests = c["logits"].shape[0], c["starts"].numel() - 1
    o = out or {"tokens": torch.full((n,), -9, dtype=torch.int32, device="cuda"), "counts": torch.full((requests,), -9, dtype=torch.int32, device="cuda"),
                "logprobs": torch.full((n,), 9.0, device="cuda"), "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
                "workspace": torch.full((afx.afx_verify_workspace(n, requests) + extra,), 0xFF, dtype=torch.uint8, device="cuda")}
    afx.afx_verify(c["logits"], c["tokens"], c["starts"], c["u"], c["draw_u"], o["tokens"], o["counts"], o["workspace"], params=params,
                   draft_logits=c["draft_logits"], draft_params=draft_params, logprobs=o["logprobs"] if logprobs else None, status_dev=o["status"])
    return o


def _check(c, o, params, draft_params=None, least_sure=0.5):
    z, starts = c["logits"].double().cpu().numpy(), c["starts"].tolist()
    zd = c["draft_logits"].double().cpu().numpy() if c["draft_logits"] is not None else None
    tokens, u, draw_u = c["tokens"].tolist(), c["u"].double().tolist(), c["draw_u"].double().tolist()
    got, counts, logprobs = o["tokens"].tolist(), o["counts"].tolist(), o["logprobs"].double().tolist()
    assert o["status"].item() == 0
    n_sure = 0
    for r in range(len(starts) - 1):
        a, b = starts[r], starts[r + 1]
        if a == b:
            assert counts[r] == 0
            n_sure += 1
            continue
        one = lambda p: {k: v[r].item() for k, v in (p or {}).items()}  # noqa: E731
        rows = [ref.shares(z[t], **one(params), near=NEAR) for t in range(a, b)]
        others = [ref.shares(zd[t], **one(draft_params), near=NEAR) for t in range(a, b)] if zd is not None else None
        doubtful = [x[2] | (others[i][2] if others else set()) for i, x in enumerate(rows)]
        stood, may, sure = ref.verify([x[0] for x in rows], [x[0] for x in others] if others else None, tokens[a + 1:b], u[a:b], draw_u[r],
                                      [NEAR + x[3] + (others[i][3] if others else 0.0) for i, x in enumerate(rows)], doubtful)
        used = len(stood) + 1
        sure &= all(x[1] for x in rows[:used]) and (others is None or all(x[1] for x in others[:used]))
        if not sure:
            continue
        n_sure += 1
        drawn = got[a + used - 1]
        assert got[a:a + used - 1] == stood and drawn in may and got[a + used:b] == [-1] * (b - a - used), (r, got[a:b], stood, may)
        assert counts[r] == used - (drawn == -1)
        for i, token in enumerate(got[a:b]):
            p = rows[i][0][token] if i < used and token >= 0 else 0.0
            l = 0.0 if i >= used else math.log(p) if p else -math.inf
            if token in doubtful[i] and p == 0:
                continue
            assert logprobs[a + i] == l or abs(logprobs[a + i] - l) <= 1e-5 + 1.1 * rows[i][3] + 2.0 ** -22 * abs(l), (logprobs[a + i], l)
    assert n_sure >= least_sure * (len(starts) - 1), n_sure


@pytest.mark.parametrize("which", ["mixed", "plain", "warm", "greedy"])
@pytest.mark.parametrize("kind,draft_kind", [(F32, F32), (BF16, BF16), (FP16, FP16), (F32, BF16), (BF16, F32), (FP16, BF16), (F32, None), (BF16, None), (FP16, None)])
@pytest.mark.parametrize("vocab", [2, 100, 1001, 20_000])
def test_verify(afx, which, kind, draft_kind, vocab):
    counts = [0, 1, 4, 2, 0, 7, 3, 1, 5]
    c = _case(counts, vocab, kind, draft_kind, vocab + len(which))
    params, draft_params = _params(len(counts), 1, which), _params(len(counts), 2 if which == "mixed" else 1, which)
    _check(c, _run(afx, c, params, draft_params), params, draft_params)


@pytest.mark.parametrize("counts,vocab", [([4], 151_936), ([1, 0, 3] * 12, 151_936), ([700, 1030, 512, 511, 513], 37), ([2] * 600, 517), ([3], 524_288), ([0] * 5, 40_961)])
def test_verify_sizes(afx, counts, vocab):
    c = _case(counts, vocab, F32, F32, vocab, closeness=0.05 if max(counts) > 100 else 0.5)
    if max(counts) > 100:  # long runs of drafts that stand
        c["u"] *= 0.02
    params = _params(len(counts), 3)
    _check(c, _run(afx, c, params, params), params, params)


def test_longest_run(afx):
    n = 3000
    c = _case([n - 1], 64, F32, None, 5)
    c["logits"].fill_(-math.inf)
    c["logits"][torch.arange(n), c["tokens"].roll(-1).long()] = 1.0
    o = _run(afx, c, None)
    _check(c, o, None)
    assert o["counts"].item() == n
    c["tokens"][1500] = (c["tokens"][1500] + 1) % 64
    o = _run(afx, c, None)
    assert o["counts"].item() == 1500 and (o["tokens"][1500:] == -1).all()


def test_no_parameters_and_no_logprobs(afx):
    c = _case([3, 2], 300, F32, F32, 8)
    o = _run(afx, c, None)
    _check(c, o, None)
    without = _run(afx, c, None, logprobs=False)
    assert torch.equal(without["tokens"], o["tokens"]) and (without["logprobs"] == 9).all()


def test_without_drafts_it_draws_what_sampling_draws(afx):
    rows = 40
    c = _case([0] * rows, 5000, BF16, None, 11)
    params = _params(rows, 4)
    o = _run(afx, c, params)
    tokens, logprobs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")
    afx.afx_sample(c["logits"], c["draw_u"], tokens, logprobs=logprobs, **params)
    assert torch.equal(o["tokens"], tokens) and torch.equal(o["logprobs"], logprobs) and (o["counts"] == 1).all()


def test_ended_drafts_and_padding(afx):
    c = _case([4, 3, 2], 50, F32, F32, 21)
    c["tokens"][2] = -1        # request 0: one draft
    c["tokens"][6] = 50        # request 1: none
    c["starts"][3] = 11        # the last row belongs to none
    c["u"] *= 0
    o = _run(afx, c, None)
    _check(c, o, None)
    assert o["tokens"][11] == -9 and o["logprobs"][11] == 9.0


def test_rows_with_nothing_and_infinite_rows(afx):
    inf = math.inf
    c = _case([2, 2, 2, 2, 1], 64, F32, F32, 22)
    c["logits"][0] = -inf                      # nothing to draw from at once
    c["logits"][4, :] = float("nan")           # the same behind a draft that stands
    c["tokens"][4] = c["logits"][3].argmax()
    c["u"][3] = 0
    c["draft_logits"][6] = -inf                # a draft from nothing: its probability is 0
    c["tokens"][7] = c["logits"][6].argmax()
    c["logits"][9, 5] = c["logits"][9, 60] = inf   # two infinite logits share everything
    c["tokens"][10] = 60
    c["draft_logits"][12, 7] = c["draft_logits"][12, 8] = inf
    c["tokens"][13] = 7
    for which in (None, _params(5, 1, "warm"), _params(5, 1, "greedy")):
        o = _run(afx, c, which, which)
        got, counts = o["tokens"].tolist(), o["counts"].tolist()
        assert got[:3] == [-1, -1, -1] and counts[0] == 0 and o["logprobs"][0] == -inf
        assert got[3:6] == [c["tokens"][4].item(), -1, -1] and counts[1] == 1 and o["logprobs"][4] == -inf
        assert got[6] == c["tokens"][7].item()
        assert got[9] in (5, 60)
        if which is None:
            assert got[9] == (60 if c["u"][9] < 0.5 else 5) or got[9] == 60
            p = ref.shares(c["logits"][12].cpu().numpy())[0]
            assert (got[12] == 7) == (c["u"][12].item() * 0.5 < p[7])
    # temperature 0 on two infinite logits: the first
    assert got[9] == 5


def test_draft_that_its_own_logits_do_not_allow(afx):
    c = _case([1, 1], 32, F32, F32, 23)
    c["draft_logits"].copy_(c["logits"])
    params = _params(2, 1, "greedy")
    for r in range(2):  # the same rows, temperature 0, another token than the first
        c["tokens"][2 * r + 1] = c["logits"][2 * r].argmin()
    o = _run(afx, c, params, params)
    assert o["tokens"].tolist() == [c["logits"][0].argmax().item(), -1, c["logits"][2].argmax().item(), -1]


def test_strided_and_unaligned_rows(afx):
    for offset, width in ((0, 1040), (1, 1030), (4, 1036)):
        c = _case([2, 3], 1024, BF16, BF16, 24)
        for k in ("logits", "draft_logits"):
            wide = torch.full((c[k].shape[0], width), 100.0, dtype=BF16, device="cuda")
            wide[:, offset:offset + 1024] = c[k]
            c[k] = wide[:, offset:offset + 1024]
        params = _params(2, 5)
        _check(c, _run(afx, c, params, params), params, params)


@pytest.mark.parametrize("starts", [[1, 3, 5], [0, 4, 3], [0, 3, 6], [0, -1, 5], [-1, 2, 5]])
def test_bad_starts(afx, starts):
    c = _case([2, 1], 200, F32, F32, 25)
    c["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    o = _run(afx, c, None)
    assert o["status"].item() == afx.AFX_DEV_BAD_LENGTH and (o["counts"] == 0).all() and (o["tokens"] == -9).all()


def test_requests_without_rows(afx):
    c = _case([1, 2], 100, F32, F32, 26)
    c["starts"] = torch.tensor([0, 0, 2, 2, 5, 5], dtype=torch.int32, device="cuda")
    c["draw_u"] = torch.rand(5, device="cuda")
    _check(c, _run(afx, c, None), None)
    c["starts"].zero_()
    o = _run(afx, c, None)
    assert (o["counts"] == 0).all() and (o["tokens"] == -9).all() and o["status"].item() == 0


def test_ties_in_16_bits(afx):
    """Hundreds of equal logits around a top-k boundary: the ones of lowest index are kept."""
    c = _case([3] * 8, 4000, BF16, BF16, 27)
    for k in ("logits", "draft_logits"):
        c[k] = (c[k].float() / 3).round().to(BF16)
    params = {"top_k": torch.full((8,), 700, dtype=torch.int32, device="cuda")}
    _check(c, _run(afx, c, params, params), params, params)
    params = {"top_p": torch.full((8,), 0.8, device="cuda")}
    _check(c, _run(afx, c, params, params), params, params, least_sure=0.2)


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_are_distributed_as_the_target(afx, drawn):
    """16,384 requests of one pair of rows: the first token's frequencies are p's, within 5 standard deviations."""
    n, vocab = 16_384, 6
    g = torch.Generator(device="cuda").manual_seed(31)
    z = torch.tensor([0.0, 1.0, -1.0, 0.5, 2.0, -0.5], device="cuda")
    zd = torch.tensor([1.0, 0.0, 0.5, 0.5, 0.5, -1.0], device="cuda")
    draft = torch.zeros(n, dtype=torch.int32, device="cuda")
    if drawn:
        afx.afx_sample(zd.expand(n, vocab).contiguous(), torch.rand(n, generator=g, device="cuda"), draft)
    else:
        draft = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
    tokens = torch.zeros(2 * n, dtype=torch.int32, device="cuda")
    tokens[1::2] = draft
    c = {"logits": z.expand(2 * n, vocab).contiguous(), "draft_logits": zd.expand(2 * n, vocab).contiguous() if drawn else None, "tokens": tokens,
         "starts": torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda"), "u": torch.rand(2 * n, generator=g, device="cuda"),
         "draw_u": torch.rand(n, generator=g, device="cuda")}
    o = _run(afx, c, None)
    p = torch.softmax(z.double(), 0)
    seen = torch.bincount(o["tokens"][::2].long(), minlength=vocab).double() / n
    assert ((seen - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all(), (seen, p)
    both = o["counts"] == 2
    assert 0.1 < both.double().mean().item() < 0.9
    if drawn:
        q = torch.softmax(zd.double(), 0)
        stood = torch.minimum(p, q).sum().item()
        assert abs(both.double().mean().item() - stood) <= 5 * (stood * (1 - stood) / n) ** 0.5


def test_captured_and_repeated(afx):
    counts = [2, 3, 1]
    c = _case(counts, 3000, F32, F32, 41)
    params = _params(3, 6)
    o = _run(afx, c, params, params)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(afx, c, params, params, out=o)
    for seed in (42, 43):
        new = _case(counts, 3000, F32, F32, seed)
        for k in c:
            c[k].copy_(new[k])
        graph.replay()
        first = {k: v.clone() for k, v in o.items()}
        _check(c, o, params, params)
        graph.replay()
        assert all(torch.equal(first[k], o[k]) for k in ("tokens", "counts", "logprobs"))


def test_a_workspace_too_small_is_refused(afx):
    c = _case([2], 100, F32, F32, 1)
    with pytest.raises(afx.AfxError):
        _run(afx, c, None, extra=-256)


def test_more_rows_than_a_grid_has(afx):
    """16,384 requests of five rows each: the same as in calls of 1024 requests."""
    n, k, vocab = 16_384, 5, 24
    c = _case([k - 1] * n, vocab, F32, BF16, 51)
    params = {"temperature": torch.linspace(0, 2, n, device="cuda"), "top_k": torch.arange(n, dtype=torch.int32, device="cuda") % 9}
    whole = _run(afx, c, params, params)
    assert whole["status"].item() == 0 and (whole["counts"] >= 1).all()
    for r in range(0, n, 1024):
        part = {key: v[r * k:(r + 1024) * k] if v.shape[0] == n * k else v[r:r + 1024] for key, v in c.items() if key != "starts"}
        part["starts"] = c["starts"][:1025].clone()
        p = {key: v[r:r + 1024].clone() for key, v in params.items()}
        o = _run(afx, part, p, p)
        assert torch.equal(o["counts"], whole["counts"][r:r + 1024])
        assert torch.equal(o["tokens"], whole["tokens"][r * k:(r + 1024) * k]) and torch.equal(o["logprobs"], whole["logprobs"][r * k:(r + 1024) * k])


def test_two_calls_at_once(afx):
    cases = [_case([3] * 20, 30_000, kind, kind, 61 + i) for i, kind in enumerate((F32, BF16))]
    params = _params(20, 7)
    want = [_run(afx, c, params, params) for c in cases]
    streams, outs = [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    for c, stream in zip(cases, streams):
        with torch.cuda.stream(stream):
            outs.append(_run(afx, c, params, params))
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(a[k], b[k]) for k in ("tokens", "counts", "logprobs"))


def test_min_p_alone_and_flat_rows(afx):
    """Rows of equal logits, where every boundary lies among ties, and min-p without another cut."""
    c = _case([2, 3, 1], 3000, F32, F32, 71)
    for key in ("logits", "draft_logits"):
        c[key][:4] = 1.25
    for params in ({"min_p": torch.tensor([0.02, 0.3, 1.0], device="cuda")}, {"top_k": torch.tensor([7, 2999, 3000], dtype=torch.int32, device="cuda")},
                   {"top_p": torch.tensor([0.3, 0.7, 0.999], device="cuda")}):
        _check(c, _run(afx, c, params, params), params, params, least_sure=0.3)
        _check(c, _run(afx, c, params, None), params, None, least_sure=0.3)
        _check(c, _run(afx, c, None, params), None, params, least_sure=0.3)


def test_extreme_temperatures(afx):
    c = _case([2] * 6, 500, F32, F32, 81)
    params = {"temperature": torch.tensor([1e-38, 1e-3, 1e30, math.inf, float("nan"), -1.0], device="cuda")}
    o = _run(afx, c, params, params)
    assert o["status"].item() == 0 and ((o["tokens"] >= -1) & (o["tokens"] < 500)).all()
    top = c["logits"].argmax(1).tolist()
    got = o["tokens"].tolist()
    for r in (0, 4, 5):  # so cold that the largest logit alone is left, or temperature 0
        at = 3 * r
        assert got[at] == top[at]

"""Rotary positions against 64-bit definitions.

A turned element is off by: its angle's rounding, at most 2^-24 of half a turn
(1.9e-7), the sine's and cosine's (two last places), the amplitude's product and the two products'
and the sum's, 2^-24 each, all relative to |a| + |b|: together below 2^-21; the
frequency in 53 bits, 2^-51 of position * frequency; and one rounding to the
result's type.
"""
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _plan(afx, dim, rotary, sections, order, pairs, base=10_000.0, **more):
    plan = afx.rotary(dim, rotary_dim=rotary, base=base, sections=sections, order=order, pairs=pairs, **more)
    left, axes = list(sections), []
    while len(axes) < rotary // 2:
        for a in range(len(left)):
            while left[a] and order == "blocks":
                axes.append(a)
                left[a] -= 1
            if left[a]:
                axes.append(a)
                left[a] -= 1
    return plan, axes, [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def _check(y, x, positions, freq, axes, rotary, pairs, amplitude=1.0):
    positions = positions.cpu().reshape(-1, x.shape[0])
    want, reach = ref.rotate(x, positions, freq, axes, rotary, pairs, amplitude)
    far = max(abs(f) for f in freq) * positions.abs().max().item() if positions.numel() else 0
    bound = reach * (2.0 ** -21 + far * 2.0 ** -51)
    bound = bound + ref.round_error(want.abs() + bound, y.dtype)
    bound[..., rotary:] = ref.round_error(want[..., rotary:], y.dtype)
    assert ((y.double().cpu() - want).abs() <= bound).all(), ((y.double().cpu() - want).abs() / bound).max()


def _positions(n, axes, seed, far=100_000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-5, far, (axes, n), generator=g, device="cuda", dtype=torch.int32)


SHAPES = [  # tokens, heads, dim, rotary, sections
    (1, 1, 128, 128, [64]), (3, 5, 128, 128, [16, 24, 24]), (17, 2, 64, 32, [16]), (9, 3, 96, 48, [8, 8, 8]), (5, 4, 80, 20, [10]),
    (2, 1, 2, 2, [1]), (4, 2, 256, 256, [100, 28]), (6, 3, 66, 34, [5, 5, 7]), (2600, 7, 64, 64, [8, 12, 12]), (2433, 1, 128, 64, [32]),
    (130, 40, 128, 128, [64]), (8, 2, 128, 112, [56])]


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("order", ["blocks", "interleaved"])
@pytest.mark.parametrize("n,heads,dim,rotary,sections", SHAPES)
def test_rotate(afx, n, heads, dim, rotary, sections, order, pairs):
    plan, axes, freq = _plan(afx, dim, rotary, sections, order, pairs)
    positions = _positions(n, len(sections), n + dim)
    for kind, out in ((BF16, BF16), (FP16, FP16), (F32, BF16), (F32, FP16), (F32, F32), (BF16, F32), (BF16, FP16), (FP16, BF16), (FP16, F32)):
        if n > 1000 and kind != out:
            continue
        x = torch.randn((n, heads, dim), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(kind)
        y = torch.full(x.shape, 9.0, dtype=out, device="cuda")
        afx.afx_rotate(plan, positions, x, y)
        _check(y, x, positions, freq, axes, rotary, pairs)


def test_far_positions(afx):
    plan, axes, freq = _plan(afx, 128, 128, [64], "blocks", "halves")
    positions = torch.tensor([0, 1, -1, 131_071, 1 << 24, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    x = torch.randn((8, 3, 128), device="cuda")
    y = torch.empty_like(x)
    afx.afx_rotate(plan, positions, x, y)
    _check(y, x, positions, freq, axes, 128, "halves")
    assert torch.equal(y[0], x[0])


def test_given_frequencies_and_amplitude(afx):
    freq = [0.0, -0.25, 1.0, 3.0, 7.5, 100.0, 1e-9, 0.5, 6.283185307179586, 12.0, 1e-30, 0.125, 2.0, -3.0, 0.75, 1e6]
    plan = afx.rotary(32, frequencies=freq, amplitude=1.25)
    positions = torch.arange(-20, 21, dtype=torch.int32, device="cuda")
    x = torch.randn((41, 2, 32), device="cuda")
    y = torch.empty_like(x)
    afx.afx_rotate(plan, positions, x, y)
    _check(y, x, positions, freq, [0] * 16, 32, "halves", 1.25)


def test_in_place_and_strided(afx):
    plan, axes, freq = _plan(afx, 64, 64, [32], "blocks", "halves")
    positions = _positions(50, 1, 1)
    for offset, width in ((0, 64), (3, 67), (8, 80)):
        rows = torch.randn((50, 6, width + 8), device="cuda").to(BF16)
        before = rows.clone()
        x = rows[:, 1:5, offset:offset + 64]
        afx.afx_rotate(plan, positions[0], x, x)
        _check(x, before[:, 1:5, offset:offset + 64], positions, freq, axes, 64, "halves")
        rest = torch.ones(rows.shape, dtype=torch.bool, device="cuda")
        rest[:, 1:5, offset:offset + 64] = False
        assert torch.equal(rows[rest], before[rest])
    # heads before tokens
    x = torch.randn((4, 50, 64), device="cuda").transpose(0, 1)
    y = torch.empty((4, 50, 64), device="cuda").transpose(0, 1)
    afx.afx_rotate(plan, positions[0], x, y)
    _check(y, x, positions, freq, axes, 64, "halves")


def _pools(pages, page, heads, dim, kind, order):
    whole = torch.randn((pages, page, heads, dim), device="cuda").to(kind)
    shape = {"pth": (0, 1, 2, 3), "hpt": (2, 0, 1, 3), "pht": (0, 2, 1, 3)}[order]
    back = [shape.index(i) for i in range(4)]
    return [whole.permute(shape).contiguous().permute(back).clone(memory_format=torch.preserve_format) for _ in range(2)]


@pytest.mark.parametrize("kind,cache_kind", [(BF16, BF16), (FP16, FP16), (F32, BF16), (F32, FP16), (FP16, BF16)])
@pytest.mark.parametrize("n,q_heads,kv_heads,dim,rotary,page,order", [
    (1, 1, 1, 64, 64, 16, "pth"), (37, 10, 2, 128, 128, 16, "hpt"), (2500, 3, 1, 64, 48, 32, "pht"), (64, 40, 8, 128, 128, 64, "pth"),
    (20, 0, 4, 64, 64, 256, "pth"), (9, 6, 3, 128, 36, 128, "hpt")])
def test_rotate_write(afx, kind, cache_kind, n, q_heads, kv_heads, dim, rotary, page, order):
    plan, axes, freq = _plan(afx, dim, rotary, [rotary // 2], "blocks", "neighbours" if n % 2 else "halves")
    pairs = "neighbours" if n % 2 else "halves"
    positions = _positions(n, 1, n)
    pages = n // page + 3
    k_pool, v_pool = _pools(pages, page, kv_heads, dim, cache_kind, order)
    before = [k_pool.clone(), v_pool.clone()]
    rows = torch.randn((n, (q_heads + 2 * kv_heads), dim), device="cuda").to(kind)
    q, k, v = rows.split([q_heads, kv_heads, kv_heads], 1)
    slots = torch.randperm(pages * page, device="cuda")[:n].to(torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if n > 10:
        slots[3], slots[7] = -1, pages * page  # padding; past the pool
    q_out = torch.full((n, q_heads, dim), 3.0, dtype=cache_kind, device="cuda")
    afx.afx_rotate_write(plan, positions, q if q_heads else None, k, v, q_out if q_heads else None, afx.kv_cache(k_pool, v_pool), slots,
                         status_dev=status)
    assert status.item() == (afx.AFX_DEV_BAD_PAGE if n > 10 else 0)
    live = slots >= 0
    held = live & (slots < pages * page)
    at = slots[held].long()
    if q_heads:
        _check(q_out[live], q[live], positions[:, live], freq, axes, rotary, pairs)
        assert (q_out[~live] == 3).all()
    _check(k_pool[at // page, at % page], k[held], positions[:, held], freq, axes, rotary, pairs)
    assert torch.equal(v_pool[at // page, at % page], v[held].to(cache_kind))
    other = torch.ones((pages, page), dtype=torch.bool, device="cuda")
    other[at // page, at % page] = False
    assert torch.equal(k_pool[other], before[0][other]) and torch.equal(v_pool[other], before[1][other])


def test_same_as_rotation_and_write_apart(afx):
    plan = afx.rotary(128, base=1e6, sections=[16, 24, 24], order="interleaved")
    n = 301
    positions = _positions(n, 3, 2)
    rows = torch.randn((n, 24, 128), device="cuda").to(BF16)
    q, k, v = rows.split([16, 4, 4], 1)
    slots = torch.randperm(20 * 16, device="cuda")[:n].to(torch.int32)
    pools = [torch.zeros((20, 16, 4, 128), dtype=BF16, device="cuda") for _ in range(4)]
    turned = torch.empty((n, 4, 128), dtype=BF16, device="cuda")
    q1, q2 = (torch.empty((n, 16, 128), dtype=BF16, device="cuda") for _ in range(2))
    afx.afx_rotate(plan, positions, q, q1)
    afx.afx_rotate(plan, positions, k, turned)
    afx.afx_kv_write(afx.kv_cache(pools[0], pools[1]), turned, v.contiguous(), slots)
    afx.afx_rotate_write(plan, positions, q, k, v, q2, afx.kv_cache(pools[2], pools[3]), slots)
    assert torch.equal(q1, q2) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    # queries in place
    afx.afx_rotate_write(plan, positions, q, k, v, q, afx.kv_cache(pools[2], pools[3]), slots)
    assert torch.equal(q, q1)


def test_special_values_pass(afx):
    plan, _, _ = _plan(afx, 64, 32, [16], "blocks", "halves")
    x = torch.ones((2, 1, 64), dtype=FP16, device="cuda")
    x[0, 0, 3] = float("nan")
    x[1, 0, 40] = float("inf")
    y = torch.empty_like(x)
    afx.afx_rotate(plan, torch.tensor([5, 6], dtype=torch.int32, device="cuda"), x, y)
    assert y[0, 0, 3].isnan() and y[0, 0, 19].isnan() and y[0].isnan().sum() == 2
    assert y[1, 0, 40] == float("inf") and y[1].isfinite().sum() == 63


def test_captured(afx):
    plan, axes, freq = _plan(afx, 128, 128, [64], "blocks", "halves")
    positions = torch.zeros(8, dtype=torch.int32, device="cuda")
    x, y = torch.randn((8, 2, 128), device="cuda"), torch.empty((8, 2, 128), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        afx.afx_rotate(plan, positions, x, y)
    for start in (0, 1000, 77):
        positions.copy_(torch.arange(start, start + 8))
        graph.replay()
        _check(y, x, positions, freq, axes, 128, "halves")

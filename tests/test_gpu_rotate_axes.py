"""Positions of several axes at any distance: one row for all of them, as text has, or rows that overlap."""
import ctypes

import pytest
import torch

from test_step_host import P

BF16 = torch.bfloat16


def test_no_distance_is_refused(afx):
    """A call comes to the check of its memory, which is the host's here, whatever the axes' distance is."""
    plan = afx.rotary(64, sections=[8, 12, 12])
    for stride in (0, 1, 4, 5):
        assert afx._lib.afx_rotate(ctypes.byref(plan), P, stride, 5, P, 2, 64, 64, 1, P + 4096, 2, 64, 64, None) == afx.AFX_E_ARG
        assert b"memory of the current device" in afx._lib.afx_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["blocks", "interleaved"])
@pytest.mark.parametrize("n", [1, 37, 3001])
def test_one_row_for_all_axes(afx, n, order):
    plan = afx.rotary(128, sections=[16, 24, 24], order=order)
    row = torch.randint(-9, 200_000, (n + 4,), device="cuda", dtype=torch.int32)
    rows = torch.randn((n, 6, 128), device="cuda").to(BF16)
    q, k, v = rows.split([4, 1, 1], 1)
    slots = torch.randperm(200 * 16, device="cuda")[:n].to(torch.int32)
    # the same positions on all axes; each axis two tokens further on than the one before
    for given in (row[:n].expand(3, n), torch.as_strided(row, (3, n), (2, 1))):
        results = []
        for positions in (given, given.contiguous()):
            y, turned = torch.empty((n, 4, 128), dtype=BF16, device="cuda"), torch.empty((n, 4, 128), dtype=BF16, device="cuda")
            pools = [torch.zeros((200, 16, 1, 128), dtype=BF16, device="cuda") for _ in range(2)]
            afx.afx_rotate(plan, positions, q, y)
            afx.afx_rotate_write(plan, positions, q, k, v, turned, afx.kv_cache(*pools), slots)
            assert torch.equal(y, turned)
            results.append([y, *pools])
        assert all(torch.equal(a, b) for a, b in zip(*results))
    # one row is what a plan of one axis turns by
    one = torch.empty((n, 4, 128), dtype=BF16, device="cuda")
    afx.afx_rotate(afx.rotary(128), row[:n], q, one)
    afx.afx_rotate(plan, row[:n].expand(3, n), q, y)
    assert torch.equal(one, y)

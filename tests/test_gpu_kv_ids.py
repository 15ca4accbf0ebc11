"""Page tables with ids outside the pool among pages that only come back: no
request takes them in the same call, and the status says so all the same."""
import pytest

from test_gpu_kv import _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 5, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("grows", [False, True])
def test_an_id_outside_the_pool_that_comes_back_is_flagged(afx, grows, bad):
    """Three pages come back, the first of them none; a request that grows takes the last of them."""
    import torch
    old, new = [40, 16], [0, 17 if grows else 16]
    table = [[bad, 2, 4], [1, -7, -7]]
    stack, count = [0, 3, -9, -9, -9], 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _call(afx, 16, old, new, table, stack, count, 1, status)
    assert status.item() == afx.AFX_DEV_BAD_PAGE
    assert got["out"] == [2 + 3 - grows] and got["stack"][:2] == [0, 3]
    assert got["slots"] == [4 * 16 if grows else -1]


def test_ids_past_a_requests_pages_are_not_looked_at(afx):
    import torch
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _call(afx, 16, [40], [16], [[0, 2, 4, 99, -1]], [1, -9, -9, -9, -9], 1, 0, status)
    assert status.item() == 0
    assert got["out"] == [3] and got["stack"] == [1, 2, 4, -9, -9]

"""Looked-up drafts have no logits, so the drafts' parameters are ignored, whatever they point to."""
import ctypes

import pytest
import torch

from test_gpu_verify import F32, _case, _check, _params, _run

pytestmark = pytest.mark.gpu


def test_parameters_of_drafts_without_logits_are_not_read(afx):
    c = _case([3, 0, 5, 1], 1001, F32, None, 91)
    params = _params(4, 8)
    want = _run(afx, c, params)
    _check(c, want, params)
    # numbers that are no addresses of the device's memory, as a caller may leave them in what counts for nothing
    nowhere = afx.afx_sampling(8, 16, 24, 32)
    given = afx._sampling(params, 4)
    n = c["logits"].shape[0]
    got = {k: torch.full_like(v, -5) for k, v in want.items() if k not in ("workspace", "status")}
    args = afx.afx_verify_args(c["logits"].data_ptr(), None, 1001, 7, afx.AFX_TYPE_F32, 99, 1001, 4, n, 0, c["starts"].data_ptr(),
                               c["tokens"].data_ptr(), given, nowhere, c["u"].data_ptr(), c["draw_u"].data_ptr())
    status = afx._lib.afx_verify(ctypes.byref(args), got["tokens"].data_ptr(), got["counts"].data_ptr(), got["logprobs"].data_ptr(),
                                 want["workspace"].data_ptr(), want["workspace"].numel(), torch.cuda.current_stream().cuda_stream, None)
    assert status == afx.AFX_OK
    assert all(torch.equal(got[k], want[k]) for k in got)

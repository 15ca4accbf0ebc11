"""E4M3 products in whose shared memory an odd number of stages fits, five at the least: 121 tokens or more of a
CTA's own tile, and results that are not whole sectors.  More steps than the
ring has stages, alone and beside other traffic; bounds as in test_gpu_fp8.py,
and the same bits each time."""
import pytest
import torch

from test_gpu_fp8 import BF16, F32, _activations, _check_product, _product, _quantized, _weights

pytestmark = pytest.mark.gpu


def _inputs(afx, n, rows, cols):
    q, x_scales = _quantized(afx, _activations(n, cols, BF16, n + rows, spread=False))
    return (*_weights(rows, cols, cols), q, x_scales)


# room for five stages, for others with fewer tokens; the last into rows that start off 32 bytes
@pytest.mark.parametrize("n,rows,cols,offset", [(128, 17_400, 17_408, 0), (123, 17_401, 5120, 0), (128, 50_257, 5120, 0), (1000, 9999, 5120, 0), (128, 9001, 5120, 0),
                                                (90, 8009, 5120, 0), (128, 17_408, 5120, 1)])
def test_odd_rings(afx, n, rows, cols, offset):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    inputs = _inputs(afx, n, rows, cols)
    for kind in (BF16, F32):
        y = torch.full((n, rows + offset), 77.0, dtype=kind, device="cuda")[:, offset:]
        afx.afx_fp8_product(*inputs, y, status_dev=status)
        _check_product(*inputs, y)
        first = y.clone()
        for _ in range(60):
            y.fill_(77.0)
            afx.afx_fp8_product(*inputs, y, status_dev=status)
            assert torch.equal(y, first)
        # copies of other memory beside it, so that its own come in another order
        other, a = torch.cuda.Stream(), torch.empty(1 << 27, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(20):
                a[1 << 26:].copy_(a[:1 << 26])
        for _ in range(20):
            y.fill_(77.0)
            afx.afx_fp8_product(*inputs, y, status_dev=status)
            assert torch.equal(y, first)
        torch.cuda.synchronize()
    assert status.item() == 0


def test_odd_rings_side_by_side(afx):
    sets = [_inputs(afx, n, rows, cols) for n, rows, cols in ((128, 17_401, 2560), (125, 9007, 5120))]
    want = [_product(afx, *s, F32) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[torch.empty_like(w) for w in want] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, stream in enumerate(streams):
            for i in (k, 1 - k):
                afx.afx_fp8_product(*sets[i], got[k][i], stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for one in got for a, b in zip(one, want))

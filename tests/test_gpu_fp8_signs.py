"""Signs of zeros through the rounding to E4M3: -0 / scale is -0, and so is a negative quotient too small for a value."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("largest", [448.0, 3.0, 6e-8, 0.0])
def test_signs_of_zeros(afx, kind, largest):
    x = torch.zeros((9, 300), dtype=kind, device="cuda")
    x[:, 1::2] = -0.0
    x[:, 4::8] = torch.tensor(1e-7 * largest, dtype=kind, device="cuda")
    x[:, 5::8] = torch.tensor(-1e-7 * largest, dtype=kind, device="cuda")
    x[:, 128 * 2 + 3] = x[:, 7] = largest
    x[:, 130] = -largest
    for offset in (0, 1):  # rows that are aligned for wide loads, and that are not
        rows = torch.zeros((9, 304 + offset), dtype=kind, device="cuda")[:, offset:offset + 300]
        rows.copy_(x)
        q = torch.zeros((9, 304), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((3, 9), device="cuda")
        afx.afx_fp8_quantize(rows, q, scales)
        assert torch.equal(q[:, :300] >> 7, torch.signbit(rows.float()).to(torch.uint8))
        assert (q[:, 0] == 0).all() and (q[:, 1] == 0x80).all()
        if largest:
            assert (q[:, 7] == 0x7E).all() and (q[:, 130] == 0xFE).all()

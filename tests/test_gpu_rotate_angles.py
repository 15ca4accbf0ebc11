"""Sines and cosines of angles near their zeros, and everywhere else, relative to themselves.

A head (1, 0) becomes (cos, sin).  Each is off by the function's two last
places, 2^-22, and by one rounding each, 2^-24, of the turn by the angle's rest,
of the amplitude's product and of the result's: below 2^-21 of itself.  The rest of the angle is
right to 2^-22 of itself, at most 2^-22, so to 2^-44 and to 2^-22 of the sine or cosine where that is all there is of it; what
turning by it leaves out, half its square, is below 2^-45; a frequency in 53 bits to 2^-51 of position * frequency.
"""
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu


def test_angles_beside_half_a_turn_and_a_whole_one(afx):
    """A frequency of half a turn and a little, of a turn and a little: every angle is beside a zero of the sine."""
    turn = 6.283185307179586476925286766559
    for little in (1e-9, -1e-9, 3e-8, -3e-8, 2.0 ** -25, 1e-5):
        for base in (turn / 2, turn, 0.0):
            frequency = base + little
            plan = afx.rotary(2, frequencies=[frequency])
            positions = torch.tensor([1, -1, 2, -2, 3, 5, 40, 127, 128, 129, -1001], dtype=torch.int32, device="cuda")
            x = torch.zeros((len(positions), 1, 2), device="cuda")
            x[:, 0, 0] = 1.0
            y = torch.empty_like(x)
            afx.afx_rotate(plan, positions, x, y)
            want, _ = ref.rotate(x, positions.cpu()[None], [frequency], [0], 2, "halves")
            far = positions.double().abs().cpu()[:, None, None] * abs(frequency)
            bound = want.abs() * 2.0 ** -21 + 2.0 ** -43 + far * 2.0 ** -51
            assert ((y.double().cpu() - want).abs() <= bound).all(), (little, base)


@pytest.mark.parametrize("frequency,amplitude", [(1.0, 1.0), (0.5, 1.25), (3.0, 1.0), (1.0 / 3, 0.75)])
def test_sines_and_cosines(afx, frequency, amplitude):
    # multiples of pi and of its half come near integers at these
    near = [p * m for p in (1, 11, 22, 33, 355, 710, 103_993, 104_348, 208_341, 312_689, 833_719, 1_146_408, 4_272_943) for m in (1, -1, 3, 7)]
    many = torch.randint(-1_000_000, 1_000_000, (4000,), generator=torch.Generator().manual_seed(3)).tolist()
    positions = torch.tensor(near + many, dtype=torch.int32, device="cuda")
    plan = afx.rotary(2, frequencies=[frequency], amplitude=amplitude)
    for first in (0, 1):  # (1, 0): cosine and sine; (0, 1): minus the sine and the cosine
        x = torch.zeros((len(positions), 1, 2), device="cuda")
        x[:, 0, first] = 1.0
        y = torch.empty_like(x)
        afx.afx_rotate(plan, positions, x, y)
        want, _ = ref.rotate(x, positions.cpu()[None], [frequency], [0], 2, "halves", amplitude)
        far = positions.double().abs().cpu()[:, None, None] * frequency
        bound = want.abs() * 2.0 ** -21 + amplitude * (2.0 ** -43 + far * 2.0 ** -51)
        worst = ((y.double().cpu() - want).abs() / bound).max().item()
        assert worst <= 1, worst
    # some are near zeros indeed: where a float32 angle would be off by more than these are large
    assert want.abs().min().item() < 1e-4

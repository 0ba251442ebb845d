"""Frequencies for a longer context, "parts": what its description says of each of them (CPU)."""
import math

import pytest
import torch

from selective_state_space_48_amd import selscan as S


@pytest.mark.parametrize("rot,original,fast,slow", [
    (64, 4096, 32.0, 1.0),
    (64, 100, 32.0, 1.0),      # none turns fast
    (64, 512, 200.0, 100.0),   # all turn slowly, the first one too
    (16, 5, 32.0, 1.0),
    (2, 3, 32.0, 1.0),
    (2, 4096, 32.0, 1.0),
    (8, 1 << 24, 32.0, 1.0),   # all turn fast
])
def test_parts(rot, original, fast, slow):
    f = S.rotary_frequencies(rot).double()
    p = S.rotary_frequencies(rot, scaling="parts", factor=8.0, original=original, fast=fast, slow=slow).double()
    turns = original * f / (2 * math.pi)
    share = (1 - p / f) * 8 / 7  # 0: left as it is, 1: divided by the factor
    # (p and f are each rounded to fp32 once: a share is off by 2 x 2^-24 x 8 / 7 and the factor's own rounding)
    room = 4 * 2.0 ** -24
    assert (share[turns > fast * (1 + 1e-6)].abs() <= room).all()
    assert ((share[turns < slow * (1 - 1e-6)] - 1).abs() <= room).all()
    assert (share >= -room).all() and (share <= 1 + room).all() and (share.diff() >= -room).all()

"""The oracle's scale of a group whose range is a few fp32 steps of its offset, pinned by hand."""
import numpy as np
import pytest

from oracle import quant4 as q4


@pytest.mark.parametrize("z,steps,bits", [
    # fp32 steps near 1000 are 2^-14. 15 s + 1000 reaches 1000 + 2^-14 from half a step on (a tie goes
    # to the even 1000): 15 s > 2^-15, s > 34.13 * 2^-24; the quotient 2^-14 / 15 is 68.27 * 2^-24.
    (1000.0, 1, 35),
    # steps of 2^-17 near 100, the same: s > 2^-18 / 15 = 4.27 * 2^-24
    (100.0, 1, 5),
    # 32 + 2 steps of 2^-18: from 1.5 steps on, a tie to the even second: 15 s >= 1.5 * 2^-18, s >= 6.4 * 2^-24
    (32.0, 2, 7),
    # below zero: -1000 + one step of 2^-14 has an odd last bit too, s > 34.13 * 2^-24
    (-1000.0, 1, 35),
])
def test_scales_of_narrow_groups_by_hand(z, steps, bits):
    top = np.float32(z) + np.float32(steps) * np.spacing(np.abs(np.float32(z)))
    s, zero = q4.group_params(z, top)
    assert zero == z and s == bits * 2.0 ** -24
    for k, enough in ((bits, True), (bits - 1, False)):
        assert (np.float32(15 * k * 2.0 ** -24 + z) >= top) == enough

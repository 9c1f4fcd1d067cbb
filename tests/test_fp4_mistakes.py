"""Mistakes planted in the oracle's fp4 quantiser: its comparison with exact
rationals (test_fp4_format.py) has to reject each."""
import numpy as np
import pytest

import oracle
from test_fp4_format import test_oracle_matches_exact_rationals as compare

NEAREST = oracle._nearest_even


def scales_only(change):
    """The quantiser rounds block scales to 127 magnitudes and values to 8: change what goes in for the former."""
    return lambda mags, a: NEAREST(mags, change(a) if len(mags) == 127 else a)


def pair_maxima(a):
    """Blocks of 32: both halves get the larger one's scale."""
    p = a.reshape(a.shape[:-1] + (-1, 2))
    return np.repeat(p.max(-1), 2, axis=-1)


MISTAKES = {
    "block of 32": scales_only(pair_maxima),
    "the next block's scale": scales_only(lambda a: np.roll(a, 1, axis=-1)),
    "scale by 4 for 6": scales_only(lambda a: a * 1.5),
    "scale rounded up": lambda mags, a: np.minimum(np.searchsorted(mags, a), 126) if len(mags) == 127 else NEAREST(mags, a),
    "value towards zero": lambda mags, a: NEAREST(mags, a) if len(mags) == 127 else np.searchsorted(mags, a, side="right") - 1,
    "value ties up": lambda mags, a: NEAREST(mags, a) if len(mags) == 127
                     else np.searchsorted((mags[1:] + mags[:-1]) / 2, a, side="right"),
}


def test_the_quantiser_as_it_is_passes():
    compare(256)


@pytest.mark.parametrize("mistake", MISTAKES)
def test_each_mistake_is_rejected(monkeypatch, mistake):
    monkeypatch.setattr(oracle, "_nearest_even", MISTAKES[mistake])
    with pytest.raises(AssertionError):
        compare(256)

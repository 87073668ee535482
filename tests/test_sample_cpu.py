"""Pins of the token choice's 64-bit form (oracle/decode.py)."""

import numpy as np

from oracle import decode as ref


def test_reference_min_p_past_one_leaves_the_first_token():
    z = np.array([0.0, 3.0, 3.0, 1.0, 3.0])
    for u in (0.0, 0.5, 0.99):
        for min_p in (1.0 + 2.0 ** -23, 1.5, np.inf):
            assert ref.sample(z, u, min_p=min_p)[:3] == (1, 0.0, True)
    assert {ref.sample(z, u, min_p=1.0)[0] for u in (0.1, 0.5, 0.9)} == {1, 2, 4}

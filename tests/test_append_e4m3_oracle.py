"""The oracle's append to pages in 8 bits against the definition it states:
what a page's older rows stand for does not change by more than their rounding."""
import numpy as np
import pytest

import oracle.paged_e4m3 as ref


@pytest.mark.parametrize("old", [0.0, 2.0 ** -12, 2.0 ** -3, 3.0])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -8, 1.0, 2.0 ** 12])
def test_older_rows_keep_their_values(old, size):
    rng = np.random.default_rng(11)
    codes = ref.encode(rng.standard_normal((1, 1, 16, 8)) * 40)
    scales = np.full((1, 1), old)
    rows = rng.standard_normal((5, 1, 8)) * size
    table, offs = np.zeros((1, 1), np.int32), [0, 5]
    got, s = ref.append(codes, scales, rows, table, [12], offs)
    was, now = ref.decode(codes, scales)[0, 0, :7], ref.decode(got, s)[0, 0, :7]
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the new scale near zero
    assert np.all(np.abs(now - was) <= np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** -10 * s[0, 0]))
    if old == 0:
        assert np.all(now == 0)
    new = ref.decode(got, s)[0, 0, 7:12]
    assert np.all(np.abs(new - rows[:, 0]) <= np.maximum(2.0 ** -4 * np.abs(rows[:, 0]), 2.0 ** -10 * s[0, 0]))
    assert np.array_equal(got[0, 0, 12:], codes[0, 0, 12:])

"""What a page's score bounds: the rounded query's product from above, the query's own up to a slack."""
import numpy as np
import pytest

import oracle.paged_ref as paged


@pytest.mark.parametrize("seed", range(10))
def test_the_score_bounds_the_rounded_query(seed):
    rng = np.random.default_rng(seed)
    d = 64
    q = rng.normal(size=d).astype(np.float32).astype(np.float64)
    q[rng.integers(d)] *= 50                        # a large channel makes the small ones' codes coarse
    rows = rng.normal(size=(16, d)).astype(np.float32).astype(np.float64)
    codes, scale = paged.bounds(rows)
    c, sq = paged._codes(q)
    score = float(paged.page_score(q, codes, scale))
    size = np.abs(rows).sum(1).max()
    # a key's bound is off by at most 3 half steps of it (scale, quotient, product), the score's fp32
    # steps by 3 half steps of the sum of magnitudes: 6 half steps of max |q~| sum |k| at most, twice
    # that where codes are clamped to 127
    rounding = 12 * 2.0 ** -24 * float(sq) * 127 * (np.abs(codes).max(0) * float(scale)).sum()
    assert (rows @ (float(sq) * c)).max() <= score + rounding
    assert (rows @ q).max() <= score + float(sq) / 2 * size + rounding


def test_the_query_itself_may_lie_above_the_score():
    q, rows = np.zeros(64), np.zeros((16, 64))
    q[0], q[1], rows[:, 1] = 1.0, 0.0039, 100.0     # channel 1 rounds to code 0 beside channel 0
    score = float(paged.page_score(q, *paged.bounds(rows)))
    assert score == 0.0 and abs((rows @ q).max() - 0.39) < 1e-12
    assert 0.39 <= 0.5 / 127 * 100 * (1 + 1e-6)     # within s_q / 2 * sum |k|

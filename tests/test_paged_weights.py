"""The 24-bit weight inputs, checked on the CPU: three bf16 parts of a weight meet the tolerance the
GPU tests use, one and two parts do not."""
import numpy as np
import pytest

import paged_exact as px


def bf16(x):
    """fp32 to bf16 and back, to nearest even."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)


def in_parts(p, parts):
    total, rest = np.zeros_like(p), p.copy()
    for _ in range(parts):
        x = bf16(rest)
        total = (total + x).astype(np.float64)
        rest = (rest - x).astype(np.float32)
    return total


def worst(n, g, parts, w=1.0):
    """Largest relative error of a weight that enters the product in `parts` bf16 parts."""
    s = px.weight_queries(g) @ px.weight_keys(n).T
    p = np.exp2(s).astype(np.float32)
    got = in_parts((np.float32(w) * p).astype(np.float32), parts) / w / p.astype(np.float64).sum(1, keepdims=True)
    return (np.abs(got - px.weights_exact(n, g)) / px.weights_exact(n, g)).max()


def test_scores_are_exact_in_any_order():
    for n in px.WEIGHT_LENS:
        s = px.weight_queries(16) @ px.weight_keys(n).T
        assert np.array_equal(s * 32, np.rint(s * 32)) and s.max() == 0 and s.min() > -2
        assert np.array_equal(bf16(px.weight_keys(n)), px.weight_keys(n))
        assert np.array_equal(bf16(px.weight_queries(16)), px.weight_queries(16))
    # the scale times log2(e), as the library rounds it, is 1
    assert np.float32(px.WEIGHT_SCALE) * np.float32(1.4426950408889634) == np.float32(1)


@pytest.mark.parametrize("n", [n for n in px.WEIGHT_LENS if n > 4])
def test_fewer_parts_of_a_weight_fail_the_tolerance(n):
    assert worst(n, 4, 3) <= px.WEIGHT_TOL and worst(n, 4, 3, 0.5) <= px.WEIGHT_TOL
    assert worst(n, 4, 2) > 1.5 * px.WEIGHT_TOL
    assert worst(n, 4, 1) > 100 * px.WEIGHT_TOL

"""The paged oracle against closed forms, against the dense oracle, and with planted mistakes."""
import math
import random

import numpy as np
import pytest

import oracle.kvshare_ref as ref
import oracle.paged_ref as paged


def test_plan_small_example():
    # page 4: lengths 3 and 4, one and five new tokens; free pages 7, 8, 9 from ring entry 2 on (wrapping)
    out, faults = paged.plan([3, 4], [1, 5], [[1, -1, -1], [2, -1, -1]], [9, 5, 7, 8], 2, 3, 4, 8)
    assert not faults
    assert out["block_table"] == [[1, -1, -1], [2, 7, 8]]
    assert out["slot_map"] == [7, 28, 29, 30, 31, 32, -1, -1]
    assert out["position"] == [3, 4, 5, 6, 7, 8, 0, 0]
    assert out["token_start"] == [0, 1, 6] and out["lengths"] == [4, 9] and out["ring_state"] == [0, 1]


def test_plan_returns_pages_behind_the_ring_and_holds_back_what_does_not_fit():
    out, faults = paged.plan([5, 0, 1], [-1, 9, 1], [[3, 4, -1], [-1, -1, -1], [0, -1, -1]], [1, 2, 6, 6, 6], 0, 2, 4, 16)
    assert faults == {"pool"}                       # nine tokens need three pages, two are free
    assert out["ring"][:4] == [1, 2, 3, 4] and out["ring_state"] == [0, 4]
    assert out["lengths"] == [0, 0, 2] and out["slot_map"][:2] == [1, -1]


@pytest.mark.parametrize("seed", range(20))
def test_plan_never_gives_a_page_twice(seed):
    r = random.Random(seed)
    page, B, blocks, N = 16, 9, 12, 60
    ids = list(range(N))
    r.shuffle(ids)
    lens = [0] * B
    table = [[-1] * blocks for _ in range(B)]
    ring, state = list(ids), [r.randrange(N), N]
    ring = [ids[(i - state[0]) % N] for i in range(N)]
    for _ in range(30):
        new = [r.choice([-1, 0, 1, 1, 1, r.randrange(60)]) for _ in range(B)]
        out, _ = paged.plan(lens, new, table, ring, state[0], state[1], page, 200)
        lens, table, ring, state = out["lengths"], out["block_table"], out["ring"], out["ring_state"]
        owned = [p for b in range(B) for p in table[b][: -(-lens[b] // page)]]
        free = [ring[(state[0] + i) % N] for i in range(state[1])]
        assert sorted(owned + free) == list(range(N))
        live = [s for s in out["slot_map"] if s >= 0]
        assert len(set(live)) == len(live)


def test_bounds_hold_every_key_and_are_tight():
    rng = np.random.default_rng(0)
    rows = ref.bf16_bits_to_f64((rng.normal(size=(33, 64)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16))
    codes, scale = paged.bounds(rows)
    hi, lo = codes.astype(np.float64) * float(scale)
    # one fp32 division and one product, each within half a step of the value
    slack = np.abs(rows).max() * 2.0 ** -22
    assert np.all(rows <= hi + slack) and np.all(rows >= lo - slack)
    assert np.all(hi - rows.max(0) <= float(scale) + slack) and np.all(rows.min(0) - lo <= float(scale) + slack)
    assert codes.max() == 127 or codes.min() == -127
    zero, s = paged.bounds(np.zeros((4, 64)))
    assert s == 0 and not zero.any()


def test_score_is_an_upper_bound_of_the_codes_dot_product():
    rng = np.random.default_rng(1)
    q = rng.normal(size=64)
    rows = rng.normal(size=(16, 64))
    codes, scale = paged.bounds(rows)
    c, sq = paged._codes(q)
    # |q - sq c| <= sq / 2 per channel
    worst = (rows @ q).max()
    slack = float(sq) / 2 * np.abs(rows).sum(1).max() + 1e-4
    assert float(paged.page_score(q, codes, scale)) >= worst - slack


def test_selection_forced_blocks_ties_and_order():
    q = np.array([[1.0, 0.0]])
    level = [0, 3, 1, 3, 3, 2, 0]                   # block scores
    codes_of = lambda p, src: (np.array([[level[p], 0], [0, 0]], np.int8), np.float32(1))  # noqa: E731
    assert paged.select(q, codes_of, 7 * 16, 16, 4, 1, 1) == [0, 1, 3, 6]
    assert paged.select(q, codes_of, 7 * 16, 16, 4, 0, 1) == [1, 3, 4, 6]
    assert paged.select(q, codes_of, 7 * 16 - 15, 16, 7, 1, 1) == list(range(7))
    assert paged.select(q, codes_of, 0, 16, 3, 1, 1) == []


def test_paged_rows_equal_the_dense_cache():
    rng = np.random.default_rng(2)
    page, n, d, pages = 16, 53, 8, 9
    dense = rng.normal(size=(n, d))
    table = rng.permutation(pages)[:4]
    pool = np.full((pages, page, d), np.nan)
    for t in range(n):
        pool[table[t // page], t % page] = dense[t]
    got = paged.rows_of(pool, table, range(4), n, page, pages)
    assert np.array_equal(got, dense)
    assert np.array_equal(paged.rows_of(pool, table, [1, 3], n, page, pages), np.concatenate([dense[16:32], dense[48:]]))
    table[1] = pages
    assert not paged.rows_of(pool, table, [1], n, page, pages).any()
    q = rng.normal(size=(2, d))
    o, lse = paged.attend(q, dense, dense, d ** -0.5)
    z = q @ dense.T * d ** -0.5
    p = np.exp(z - lse[:, None])
    assert np.allclose(p.sum(1), 1, atol=1e-14) and np.allclose(p @ dense, o, atol=1e-14)
    o, lse = paged.attend(q, dense[:0], dense[:0], 1.0)
    assert not o.any() and np.all(np.isneginf(lse))


def test_planted_mistakes_are_seen():
    rng = np.random.default_rng(3)
    rows = rng.normal(size=(16, 32))
    codes, scale = paged.bounds(rows)
    inward = np.stack([np.floor(rows.max(0).astype(np.float32) / scale), np.ceil(rows.min(0).astype(np.float32) / scale)])
    assert np.any(inward * float(scale) < np.stack([rows.max(0), rows.min(0)]) * np.array([[1], [-1]]) - 1e-6)
    assert not np.array_equal(inward.astype(np.int8), codes)
    q = rng.normal(size=32)
    swapped = codes[::-1]
    assert paged.page_score(q, swapped, scale) < paged.page_score(q, codes, scale)
    assert math.isfinite(float(paged.page_score(q, codes, scale)))

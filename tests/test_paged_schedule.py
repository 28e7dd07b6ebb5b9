"""The paged decode's split, modelled on the CPU: every tile has one warp, and the CTAs a unit's
join waits for are exactly those that hold a part of it (a mismatch would leave a partial
unjoined, or an arrival counter that never returns to zero)."""
import random

import pytest


def shares(W, nw, ctas):
    nc = max(1, min(ctas, -(-W // nw)))
    workers = nc * nw
    share, more = divmod(W, workers)
    return nc, workers, [(share * i + min(i, more), share * (i + 1) + min(i + 1, more)) for i in range(workers)]


def owner(x, W, workers):
    share, more = divmod(W, workers)
    big = more * (share + 1)
    return x // (share + 1) if x < big else more + (x - big) // share


@pytest.mark.parametrize("seed", range(40))
def test_join_counts_match_the_shares(seed):
    r = random.Random(seed)
    nw = r.choice([2, 4, 8])
    ctas = r.choice([1, 3, 17, 148])
    heads = r.choice([1, 2, 5, 8])
    tiles = [r.choice([0, 1, 2, 3, r.randrange(0, 40), r.randrange(0, 3000)]) for _ in range(r.randrange(1, 30))]
    units = [t for t in tiles for _ in range(heads) if t]
    W = sum(units)
    if W == 0:
        return
    nc, workers, parts = shares(W, nw, ctas)
    assert parts[0][0] == 0 and parts[-1][1] == W and all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
    # every CTA holds a tile, so none between a unit's first and last is missing
    assert all(parts[c * nw][0] < parts[c * nw + nw - 1][1] for c in range(nc))
    begin = 0
    slots = set()
    for n in units:
        first, last = owner(begin, W, workers), owner(begin + n - 1, W, workers)
        assert parts[first][0] <= begin < parts[first][1]
        assert parts[last][0] <= begin + n - 1 < parts[last][1]
        holders = {i // nw for i, (a, b) in enumerate(parts) if a < begin + n and b > begin}
        assert holders == set(range(first // nw, last // nw + 1))
        if first // nw != last // nw:
            # one slot per partial: a CTA begins at most one unit it does not end
            mine = {2 * c + (1 if c == first // nw else 0) for c in holders}
            assert not mine & slots
            slots |= mine
        begin += n
    assert all(s < 2 * ctas for s in slots)


@pytest.mark.parametrize("seed", range(60))
def test_whole_ctas_per_unit_cover_every_tile_once(seed):
    r = random.Random(1000 + seed)
    nw, ctas, heads = r.choice([2, 4, 8, 12]), r.choice([17, 148]), r.choice([1, 2, 5, 8])
    top = r.choice([3, 30, 900])
    rows = [r.choice([0, 1, r.randrange(0, top)]) for _ in range(r.randrange(1, ctas // heads + 1))]
    W = sum(rows) * heads
    most = ctas * nw
    s0 = max(1, -(-W // most))
    if len(rows) * heads > (ctas if s0 <= 6 else ctas // 8):
        return
    for s in range(s0, s0 + (2 if s0 <= 6 else 1)):
        pieces = [-(-t // (nw * s)) for t in rows]
        if sum(pieces) * heads <= ctas:
            break
    else:
        return
    seen = [[set() for _ in range(heads)] for _ in rows]
    for cta in range(ctas):
        base = 0
        for b, m in enumerate(pieces):
            if base + m * heads > cta:
                j, seg = divmod(cta - base, m)
                share, more = divmod(rows[b], m * nw)
                mine = 0
                for w in range(nw):
                    me = seg * nw + w
                    t0 = share * me + min(me, more)
                    n = share + (1 if me < more else 0)
                    tiles = set(range(t0, t0 + n))
                    assert not tiles & seen[b][j] and n <= s + 1
                    seen[b][j] |= tiles
                    mine += n
                assert mine > 0                                  # every CTA of a unit takes part in its join
                break
            base += m * heads
    for b, t in enumerate(rows):
        assert all(x == set(range(t)) for x in seen[b])


def test_windows_of_page_entries_cover_a_tile():
    # 32 entries from a tile's first block: the tile's later pieces stay inside the window
    for page, tile in ((16, 16), (16, 32), (32, 32), (64, 32), (128, 16), (256, 32)):
        for start in range(0, 200):
            base = None
            for t in range(start, start + 200):
                blk = t * tile // page
                if base is None or blk >= base + 32:
                    base = blk
                pieces = {(t * tile + r) // page - base for r in range(0, tile, min(page, tile))}
                assert min(pieces) >= 0 and max(pieces) <= 31

"""Paged shared cache in fp64 and whole numbers: planning, append with bounds, selection, decode.

Test infrastructure, as the rest of this folder: one sequence, one head and one page at a
time, from the definitions in include/kvshare.h. Floating storage is passed as float64
arrays holding exactly the stored values.
"""
import math

import numpy as np


def plan(lengths, new_tokens, table, ring, head, count, page, max_tokens, num_pages=None):
    """Returns a dict of the outputs and the set of faults ('range', 'pool') the step reports.

    A page outside [0, num_pages) is reported: its tokens get no slot, and it keeps its place where it
    returns to the ring. None: no page is looked at.
    """
    table, ring = [list(r) for r in table], list(ring)
    B, blocks, N = len(lengths), len(table[0]), len(ring)
    cap = blocks * page
    faults = set()
    old_table = [list(r) for r in table]
    taken = asked_pages = asked_tokens = returned = 0
    out_len, start, slots, pos = [], [0], [], []
    room = N - count
    given = 0

    def exists(p):
        if num_pages is None or 0 <= p < num_pages:
            return True
        faults.add("range")
        return False
    for b in range(B):
        n, m = int(lengths[b]), int(new_tokens[b])
        if n < 0 or n > cap:
            faults.add("range")
            n = min(max(n, 0), cap) if m >= 0 else 0        # nobody knows the pages of one that leaves
        held = -(-n // page)
        if m < 0:
            given += held
            if held and given > room:
                faults.add("range")
            else:
                for i in range(held):
                    # entries behind the ring's last, in order
                    exists(old_table[b][i])
                    ring[(head + count + given - held + i) % N] = old_table[b][i]
                returned += held
            out_len.append(0)
            start.append(len(slots))
            continue
        want = m
        if n + want > cap:
            faults.add("range")
            want = 0
        need = -(-(n + want) // page) - held
        asked_pages += need
        asked_tokens += want
        if not ((need == 0 or asked_pages <= count) and asked_tokens <= max_tokens):
            if want:
                faults.add("pool")
            want = need = 0
        for i in range(need):
            table[b][held + i] = ring[(head + taken + i) % N]
        taken += need
        for t in range(n, n + want):
            p = table[b][t // page]
            slots.append(p * page + t % page if exists(p) else -1)
            pos.append(t)
        out_len.append(n + want)
        start.append(len(slots))
    slots += [-1] * (max_tokens - len(slots))
    pos += [0] * (max_tokens - len(pos))
    return dict(block_table=table, ring=ring, ring_state=[(head + taken) % N, count - taken + returned],
                lengths=out_len, token_start=start, slot_map=slots, position=pos), faults


INV_127 = np.float32(1) / np.float32(127)


def bounds(rows):
    """int8 codes [2][d] and fp32 scale of one page's keys rows [n][d] (fp32 steps as stated)."""
    hi = rows.max(axis=0).astype(np.float32)
    lo = rows.min(axis=0).astype(np.float32)
    scale = np.float32(max(np.abs(hi).max(), np.abs(lo).max())) * INV_127
    if scale == 0:
        return np.zeros((2, rows.shape[1]), np.int8), scale
    up = np.minimum(np.ceil(hi / scale), 127)
    down = np.maximum(np.floor(lo / scale), -127)
    return np.stack([up, down]).astype(np.int8), scale


def append(k, v, codes, scales, k_new, v_new, slot_map, page):
    """In place on one slot's pool k, v [pages][Hkv][page][d] (and codes, scales, or None)."""
    last = {}
    for i, s in enumerate(slot_map):
        if s < 0 or s // page >= k.shape[0]:
            continue
        k[s // page, :, s % page] = k_new[i]
        v[s // page, :, s % page] = v_new[i]
        last[s // page] = max(last.get(s // page, -1), s % page)
    if codes is not None:
        for p, r in last.items():
            for j in range(k.shape[1]):
                codes[p, j], scales[p, j] = bounds(k[p, j, : r + 1])


def _codes(q):
    scale = np.float32(np.abs(q).max()) * INV_127
    if scale == 0:
        return np.zeros(q.shape, np.int64), scale
    return np.rint(q.astype(np.float32) / scale).astype(np.int64), scale


def page_score(q, codes, scale):
    """fp32 score of one head's query against one page's codes [2][d]."""
    c, sq = _codes(q)
    hi, lo = codes.astype(np.int64)
    dot = int(np.where(c > 0, c * hi, c * lo).sum())
    return np.float32(np.float32(np.float32(dot) * sq) * np.float32(scale))


def select(q, codes_of, n, page, top, first, last, w=None):
    """Blocks one kv head keeps. q [g][d]; codes_of(block, source) -> (codes, scale); w: mix weight or None."""
    held = -(-n // page)
    score = []
    for p in range(held):
        best = -math.inf
        for h in range(q.shape[0]):
            s = page_score(q[h], *codes_of(p, 0))
            if w is not None:
                w32 = np.float32(w)
                s2 = page_score(q[h], *codes_of(p, 1))
                s = np.float32(np.float32(w32 * s) + np.float32(np.float32(np.float32(1) - w32) * s2))
            best = max(best, float(s))
        score.append(best)
    if held <= top:
        return list(range(held))
    forced = {p for p in range(held) if p < first or p >= held - last}
    rest = sorted((p for p in range(held) if p not in forced), key=lambda p: (-score[p], p))
    return sorted((sorted(forced) + rest)[:top])


def rows_of(pool, table_row, blocks, n, page, num_pages):
    """The tokens of the listed blocks, in their order: pool [pages][page][d] of one slot and head.

    A page outside the pool reads as zeros; a block outside the sequence is skipped.
    """
    out = []
    for blk in blocks:
        if blk < 0 or blk >= -(-n // page):
            continue
        rows = min(page, n - blk * page)
        ph = int(table_row[blk])
        out.append(pool[ph, :rows] if 0 <= ph < num_pages else np.zeros((rows, pool.shape[-1])))
    return np.concatenate(out) if out else np.zeros((0, pool.shape[-1]))


def attend(q, k, v, scale):
    """q [g][d] over k, v [n][d]: outputs [g][d] and natural-log lse [g]; no token: 0 and -inf."""
    if len(k) == 0:
        return np.zeros(q.shape), np.full(q.shape[0], -np.inf)
    z = (q @ k.T) * scale
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    total = e.sum(axis=1, keepdims=True)
    return (e @ v) / total, (m + np.log(total))[:, 0]

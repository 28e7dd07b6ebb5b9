"""Paged decode where the warps' shares are long: the evenly split line with units that straddle
CTAs, whole CTAs of several tiles a warp, windows of block-table entries reloaded in mid-stream,
and rings that go round many times. And weights that need all 24 bits. Against 64 bits with a
bound for every element (paged_exact)."""
import random

import numpy as np
import pytest

from paged_exact import (WEIGHT_LENS, WEIGHT_SCALE, WEIGHT_TOL, check_exact, exact_decode, weight_keys, weight_queries,
                         weights_exact)
from paged_helpers import Pool, torch_mod

pytestmark = pytest.mark.gpu

# shares here are at most 65 tiles of 3 half steps; joins of at most 12 warps and 148 CTAs
STEPS = 3 * 65 + 12 + 148


@pytest.fixture(scope="module")
def K():
    from cross_layer_kv_shared_b200 import kvshare
    return kvshare


def ragged(n, lo, hi, seed):
    r = random.Random(seed)
    return [r.randrange(lo, hi) for _ in range(n)]


LINES = {
    # dtype, d, Hkv, g, page, lens, list length (0: every block), blocks of a table row (0: the longest's)
    "bf16-d64": ("bf16", 64, 4, 4, 64, ragged(40, 500, 3000, 1), 0, 0),
    "bf16-d64-page16": ("bf16", 64, 3, 16, 16, ragged(50, 500, 3000, 2), 0, 0),
    "bf16-d128": ("bf16", 128, 4, 8, 32, ragged(40, 200, 900, 3) + [0, 1, 17], 0, 0),
    "bf16-d128-page16-long": ("bf16", 128, 8, 2, 16, ragged(40, 1500, 5000, 4), 0, 0),
    "bf16-d64-lists": ("bf16", 64, 4, 4, 16, ragged(40, 500, 3000, 5), 90, 0),
    "bf16-d128-lists": ("bf16", 128, 4, 16, 64, ragged(40, 500, 3000, 6), 12, 0),
    "f32-d64": ("f32", 64, 4, 4, 16, ragged(40, 500, 3000, 7), 0, 0),
    "f32-d64-g16": ("f32", 64, 2, 16, 128, ragged(75, 500, 1500, 8), 0, 0),
    "f32-d128-g8": ("f32", 128, 4, 8, 32, ragged(40, 200, 900, 9) + [0, 1, 17], 0, 0),
    "f32-d128-page16-long": ("f32", 128, 4, 3, 16, ragged(40, 1500, 5000, 10), 0, 0),
    "f32-d64-lists": ("f32", 64, 4, 8, 32, ragged(40, 500, 3000, 11), 45, 0),
    # whole CTAs per unit, 2 tiles a warp; and 7, of few long units
    "bf16-two-tiles": ("bf16", 128, 4, 4, 32, ragged(16, 420, 500, 12), 0, 100),
    "f32-two-tiles": ("f32", 64, 4, 4, 32, ragged(16, 420, 500, 13), 0, 100),
    "bf16-few-long": ("bf16", 128, 4, 4, 256, [15000, 14321], 0, 0),
    "f32-few-long": ("f32", 64, 4, 2, 256, [15000, 14321], 0, 0),
    "bf16-one-long": ("bf16", 128, 3, 4, 64, [1, 60001], 0, 0),
    "f32-one-long": ("f32", 128, 3, 1, 64, [30011, 5, 0], 0, 0),
    # few units whose lengths leave no room for whole CTAs
    "bf16-few-even": ("bf16", 128, 4, 4, 128, [16400, 16390], 0, 0),
    "f32-few-even": ("f32", 64, 4, 8, 128, [16400, 16390], 0, 0),
}


@pytest.mark.parametrize("mix", [False, True], ids=["single", "mix"])
@pytest.mark.parametrize("name", list(LINES))
def test_long_shares_against_64_bits(K, name, mix):
    torch = torch_mod()
    dtype, d, Hkv, g, page, lens, top, blocks = LINES[name]
    B, Hq = len(lens), Hkv * g
    lmap = [(K.KVS_SRC_MIX, 1, 0)] if mix else [(K.KVS_SRC_SINGLE, 0, 0)]
    w = np.linspace(0.2, 0.7, Hkv, dtype=np.float32)[None] if mix else None
    pool = Pool(K, dtype, 2 if mix else 1, Hkv, page, d, lens, seed=len(name), max_blocks=blocks or None)
    _, h = K.kvshare_create(1, Hq, Hkv, d, K.KVS_F32 if dtype == "f32" else K.KVS_BF16, B, pool.table.shape[1] * page)
    K.kvshare_set_map(h, lmap, w)
    try:
        gen = torch.Generator(device="cuda").manual_seed(len(name))
        q = torch.randn(1, B, Hq, d, generator=gen, device="cuda").to(pool.tdt)
        sel = None
        if top:
            rng = np.random.default_rng(3)
            lists = np.full((1, B, Hkv, top), -1, np.int32)
            for b, n in enumerate(lens):
                for j in range(Hkv):
                    held = -(-n // page)
                    pick = rng.permutation(held)[:top]          # any order
                    lists[0, b, j, :len(pick)] = pick
            sel = torch.from_numpy(lists).cuda()
        want = exact_decode(pool, q, lmap, w, None if sel is None else lists, steps=STEPS)
        pages = pool.pages()
        runs = []
        for _ in range(2):                                       # again: the same bits, counters back at zero
            out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:3], float("nan"), device="cuda")
            K.kvshare_decode_paged(h, pages, q, out, lse, selected=sel)
            runs.append((out, lse))
        assert K.kvshare_sync_status(h) == K.KVS_OK
        check_exact(*runs[0], want, name)
        assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    finally:
        K.kvshare_destroy(h)


@pytest.mark.parametrize("mix", [False, True], ids=["single", "mix"])
@pytest.mark.parametrize("dtype,d,g,page", [("bf16", 64, 4, 16), ("bf16", 64, 16, 64), ("bf16", 128, 8, 16),
                                            ("bf16", 128, 12, 32), ("f32", 64, 4, 16), ("f32", 128, 16, 32)])
def test_weights_keep_24_bits(K, dtype, d, g, page, mix):
    """Scores exact, one value per token in a channel of its own: an output is one weight."""
    torch = torch_mod()
    lens, Hkv = WEIGHT_LENS, 1
    lmap = [(K.KVS_SRC_MIX, 0, 1)] if mix else [(K.KVS_SRC_SINGLE, 0, 0)]
    pool = Pool(K, dtype, 2, Hkv, page, d, lens, seed=1)
    q = torch.zeros(1, len(lens), g, d, dtype=pool.tdt, device="cuda")
    q[..., :2] = torch.from_numpy(weight_queries(g)).to(q)
    want = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        ph, r = torch.from_numpy(pool.table[b]).cuda().long()[t // page], t % page
        k, v = torch.zeros(n, d, device="cuda"), torch.zeros(n, d, device="cuda")
        k[:, :2] = torch.from_numpy(weight_keys(n)).to(k)
        v[t, t] = 1.0
        for s in range(2):
            pool.k[s, ph, 0, r], pool.v[s, ph, 0, r] = k.to(pool.tdt), v.to(pool.tdt)
        want[0, b, :, :n] = torch.from_numpy(weights_exact(n, g)).cuda()
    _, h = K.kvshare_create(1, g, Hkv, d, K.KVS_F32 if dtype == "f32" else K.KVS_BF16, len(lens), 64,
                            softmax_scale=WEIGHT_SCALE)
    K.kvshare_set_map(h, lmap, np.full((1, 1), 0.5, np.float32) if mix else None)
    try:
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        err = (out.double() - want).abs()
        assert (err <= want * WEIGHT_TOL).all(), (err / want.clamp_min(1e-30))[want > 0].max().item() / WEIGHT_TOL
    finally:
        K.kvshare_destroy(h)

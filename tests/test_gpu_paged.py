"""Paged cache operators on the GPU against the fp64 oracle.

Tolerances follow from the arithmetic (paged_helpers.oracle_decode): outputs are fp32 and the
weights keep 24 bits, so errors are a few fp32 rounding steps of the scores' and values'
magnitudes. Whole numbers (plans, bound codes, selections) must be equal.
"""
import numpy as np
import pytest

import oracle.paged_ref as paged
from paged_helpers import Pool, check, oracle_decode, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from cross_layer_kv_shared_b200 import kvshare
    return kvshare


def make(K, dtype, layer_map, Hq, Hkv, d, B, ctx, w=None):
    _, h = K.kvshare_create(len(layer_map), Hq, Hkv, d, K.KVS_F32 if dtype == "f32" else K.KVS_BF16, B, ctx)
    K.kvshare_set_map(h, layer_map, w)
    return h


def queries(pool, L, Hq, seed, scale=1.0):
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(L, len(pool.lens), Hq, pool.d, generator=gen, device="cuda") * scale).to(pool.tdt)


def outputs(q):
    torch = torch_mod()
    return torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:3], float("nan"), device="cuda")


# ------------------------------------------------------------------------------- decode
RAGGED = [0, 1, 15, 16, 17, 0, 31, 33, 64, 100, 257, 2]
DECODE = [
    # dtype, d, Hkv, g, page, lens
    ("bf16", 64, 2, 4, 16, RAGGED),
    ("bf16", 64, 1, 8, 64, [300, 1, 0, 64, 65]),
    ("bf16", 64, 5, 3, 32, [33, 7]),
    ("bf16", 128, 2, 1, 16, RAGGED),
    ("bf16", 128, 3, 16, 128, [129, 128, 1]),
    ("bf16", 128, 4, 5, 256, [511, 0, 256]),
    ("bf16", 64, 2, 16, 16, [49, 200]),
    ("bf16", 128, 1, 8, 32, [4000]),                      # one unit over many CTAs
    ("bf16", 64, 8, 2, 16, [3, 5, 1, 16] * 40),           # far more units than CTAs
    ("bf16", 128, 2, 4, 32, [0] * 40 + [5] + [0] * 60 + [700] + [0] * 30 + [16] * 50),   # idle rows between
    ("bf16", 128, 4, 16, 64, [1500, 0, 900]),             # groups of 16 over several CTAs
    ("f32", 64, 2, 4, 16, RAGGED),
    ("f32", 64, 1, 7, 64, [300, 1, 0, 64, 65]),
    ("f32", 64, 2, 16, 32, [65, 31]),
    ("f32", 128, 2, 1, 32, RAGGED),
    ("f32", 128, 3, 8, 128, [129, 128, 1]),
    ("f32", 128, 1, 16, 256, [700]),
]


@pytest.mark.parametrize("mix", [False, True], ids=["single", "mix"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_against_the_oracle(K, case, mix):
    dtype, d, Hkv, g, page, lens = DECODE[case]
    lmap = [(K.KVS_SRC_SINGLE, 1, 0), (K.KVS_SRC_MIX, 0, 1)] if mix else [(K.KVS_SRC_SINGLE, 1, 0)]
    L = len(lmap)
    w = np.linspace(0.0, 1.0, L * Hkv, dtype=np.float32).reshape(L, Hkv) if mix else None
    pool = Pool(K, dtype, 2, Hkv, page, d, lens, seed=100 + case)
    Hq = Hkv * g
    h = make(K, dtype, lmap, Hq, Hkv, d, len(lens), pool.table.shape[1] * page, w)
    try:
        q = queries(pool, L, Hq, seed=case, scale=2.0)
        out, lse = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        check(out, lse, oracle_decode(pool, q.double().cpu().numpy(), lmap, w), f"case {case}")
        # the same call again: the same bits, counters back at zero
        out2, lse2 = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, out2, lse2)
        assert torch_mod().equal(out, out2) and torch_mod().equal(lse, lse2)
    finally:
        K.kvshare_destroy(h)


def test_decode_agrees_with_the_dense_decode(K):
    """The same tokens in a dense store: kvshare_decode rounds its weights to bf16 (2^-9 each)."""
    torch = torch_mod()
    B, Hkv, g, d, T, page = 3, 2, 4, 64, 192, 64
    pool = Pool(K, "bf16", 1, Hkv, page, d, [T] * B, seed=7)
    k = pool.k[0][pool.block_table.long()].transpose(1, 2).reshape(1, B, Hkv, T, d).contiguous()
    v = pool.v[0][pool.block_table.long()].transpose(1, 2).reshape(1, B, Hkv, T, d).contiguous()
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], Hkv * g, Hkv, d, B, T)
    try:
        q = queries(pool, 1, Hkv * g, seed=3)
        out, lse = outputs(q)
        dense, dlse = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse)
        K.kvshare_decode(h, K.Cache(batch=B, context=T, k=k, v=v, slots=1), q, dense, dlse)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        # weights off by 2^-9 relative at most, against their sum rounded alike: 2 * 2^-9 * max |v|
        assert (out - dense).abs().max().item() <= 2 * 2.0 ** -9 * v.float().abs().max().item()
        assert torch.allclose(lse, dlse, atol=1e-5)
    finally:
        K.kvshare_destroy(h)


def test_layers_of_a_range_and_rows_outside_it(K):
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0), (K.KVS_SRC_SINGLE, 1, 0), (K.KVS_SRC_MIX, 1, 0), (K.KVS_SRC_SINGLE, 0, 0)]
    w = np.full((4, 2), 0.25, np.float32)
    pool = Pool(K, "bf16", 2, 2, 32, 128, [70, 5, 0, 33], seed=5)
    h = make(K, "bf16", lmap, 8, 2, 128, 4, 96, w)
    try:
        q = queries(pool, 4, 8, seed=1)
        out, lse = outputs(q)
        K.kvshare_set_layer_order(h, [2, 3, 0, 1])
        n0 = K.kvshare_launch_count(h)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse, 1, 3)
        assert K.kvshare_sync_status(h) == K.KVS_OK and K.kvshare_launch_count(h) == n0 + 2
        assert torch.isnan(out[[0, 3]]).all() and torch.isnan(lse[[0, 3]]).all()
        want = oracle_decode(pool, q.double().cpu().numpy(), lmap, w)
        check(out[1:3], lse[1:3], (want[0][1:3], want[1][1:3], *want[2:]), "layers 1, 2")
        out3, _ = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, out3, None, 1, 3)          # without lse
        assert torch.equal(out3[1:3], out[1:3])
    finally:
        K.kvshare_destroy(h)


def test_pool_larger_than_32_bit_offsets(K):
    """A page whose first byte lies past 2^32 elements of the pool."""
    torch = torch_mod()
    Hkv, page, d, lens = 1, 256, 128, [300]
    N = (1 << 32) // (page * d) + 9                       # elements > 2^32 (8.6 GB a side)
    k = torch.zeros(1, N, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    pool = Pool(K, "bf16", 1, Hkv, page, d, lens, seed=2, spare=0)
    far = torch.tensor([[N - 1, N - 5]], dtype=torch.int32, device="cuda")
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 4, Hkv, d, 1, 512)
    try:
        rows = torch.arange(300, device="cuda")
        slots = (far[0][rows // page].long() * page + rows % page).to(torch.int32)
        take = lambda x: x[0][pool.block_table[0].long()].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[:300].contiguous()  # noqa: E731
        pages = K.Pages(k=k, v=v, block_table=far, lengths=pool.lengths)
        K.kvshare_append_paged(h, pages, 0, take(pool.k), take(pool.v), slots)
        q = queries(pool, 1, 4, seed=9)
        out, lse = outputs(q)
        K.kvshare_decode_paged(h, pages, q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        check(out, lse, oracle_decode(pool, q.double().cpu().numpy(), [(K.KVS_SRC_SINGLE, 0, 0)]), "far pages")
    finally:
        K.kvshare_destroy(h)


# ---------------------------------------------------------------------- bad table entries
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_outside_the_pool_read_as_zeros_and_are_reported(K, dtype):
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)]
    pool = Pool(K, dtype, 1, 2, 16, 64, [50, 40, 16], seed=11)
    table = pool.table.copy()
    table[0, 1], table[1, 2], table[2, 0] = pool.num_pages, -1, 2 ** 31 - 1
    h = make(K, dtype, lmap, 4, 2, 64, 3, 64)
    try:
        q = queries(pool, 1, 4, seed=4)
        out, lse = outputs(q)
        pages = pool.pages(block_table=torch.from_numpy(table).cuda())
        K.kvshare_decode_paged(h, pages, q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_EINVAL
        check(out, lse, oracle_decode(pool, q.double().cpu().numpy(), lmap, table=table), "bad pages")
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse)                  # the context works on
        assert K.kvshare_sync_status(h) == K.KVS_OK
    finally:
        K.kvshare_destroy(h)


def test_lengths_outside_the_table_are_clamped_and_reported(K):
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)]
    pool = Pool(K, "bf16", 1, 2, 16, 64, [48, 48], seed=12)
    h = make(K, "bf16", lmap, 4, 2, 64, 2, 48)
    try:
        q = queries(pool, 1, 4, seed=4)
        out, lse = outputs(q)
        pages = pool.pages(lengths=torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32, device="cuda"))
        K.kvshare_decode_paged(h, pages, q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_EINVAL
        check(out, lse, oracle_decode(pool, q.double().cpu().numpy(), lmap, lens=[48, 0]), "clamped")
    finally:
        K.kvshare_destroy(h)


# ------------------------------------------------------------------------------- append
APPEND = [
    # dtype, d, Hkv, page, (held, new) per sequence
    ("bf16", 64, 4, 64, [(63, 1), (64, 1), (0, 1), (5, 1)]),
    ("bf16", 128, 8, 16, [(0, 100), (7, 1), (15, 2), (16, 33)]),
    ("bf16", 128, 5, 32, [(31, 65), (0, 0), (3, 7)]),
    ("bf16", 64, 1, 256, [(250, 300)]),
    ("f32", 64, 2, 16, [(1, 40), (15, 1)]),
    ("f32", 128, 3, 128, [(100, 60), (0, 128), (127, 1)]),
    ("bf16", 128, 8, 64, [(10, 700), (0, 640)]),
]


@pytest.mark.parametrize("bounds", [False, True], ids=["rows", "bounds"])
@pytest.mark.parametrize("wide", [False, True], ids=["dense", "strided"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_against_the_oracle(K, case, wide, bounds):
    torch = torch_mod()
    dtype, d, Hkv, page, seqs = APPEND[case]
    total = [a + b for a, b in seqs]
    pool = Pool(K, dtype, 2, Hkv, page, d, total, seed=case, bounds=bounds)
    rows = [(b, t) for b, (n, m) in enumerate(seqs) for t in range(n, n + m)]
    pad = 3
    slot_map = [int(pool.table[b, t // page]) * page + t % page for b, t in rows] + [-1] * pad
    n = len(slot_map)
    gen = torch.Generator(device="cuda").manual_seed(case)
    if wide:                                                   # rows of a wider projection
        both = torch.randn(n, 3 + 2 * Hkv, d, generator=gen, device="cuda").to(pool.tdt)
        k_new, v_new = both[:, 3:3 + Hkv], both[:, 3 + Hkv:]
    else:
        k_new, v_new = (torch.randn(n, Hkv, d, generator=gen, device="cuda").to(pool.tdt) for _ in range(2))
    want_k, want_v = pool.host()
    want_c, want_s = (pool.hcodes, pool.hscales) if bounds else (None, None)
    paged.append(want_k[1], want_v[1], want_c[1] if bounds else None, want_s[1] if bounds else None,
                 k_new.double().cpu().numpy(), v_new.double().cpu().numpy(), slot_map, page)
    h = make(K, dtype, [(K.KVS_SRC_SINGLE, 1, 0)], Hkv, Hkv, d, len(seqs), 2048)
    try:
        pages = pool.pages()
        K.kvshare_append_paged(h, pages, 1, k_new, v_new, torch.tensor(slot_map, dtype=torch.int32, device="cuda"))
        assert K.kvshare_sync_status(h) == K.KVS_OK
        got_k, got_v = pool.host()
        assert np.array_equal(got_k, want_k, equal_nan=True) and np.array_equal(got_v, want_v, equal_nan=True)
        if bounds:
            assert np.array_equal(pool.codes.cpu().numpy(), want_c)
            assert np.array_equal(pool.scales.cpu().numpy(), want_s, equal_nan=True)
    finally:
        K.kvshare_destroy(h)


def test_append_skips_slots_outside_the_pool(K):
    torch = torch_mod()
    pool = Pool(K, "bf16", 1, 2, 16, 64, [20], seed=1, bounds=True)
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 2, 2, 64, 1, 64)
    try:
        before = [x.clone() for x in (pool.k, pool.v, pool.codes, pool.scales)]
        x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
        bad = torch.tensor([pool.num_pages * 16, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
        K.kvshare_append_paged(h, pool.pages(), 0, x, x, bad)
        assert K.kvshare_sync_status(h) == K.KVS_EINVAL
        for a, b in zip(before, (pool.k, pool.v, pool.codes, pool.scales)):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))
        n0 = K.kvshare_launch_count(h)
        K.kvshare_append_paged(h, pool.pages(), 0, x[:0], x[:0], bad[:0])       # no token: nothing to do
        assert K.kvshare_launch_count(h) == n0
    finally:
        K.kvshare_destroy(h)


def test_append_zero_keys_and_extremes(K):
    torch = torch_mod()
    pool = Pool(K, "f32", 1, 1, 16, 64, [32, 16], seed=1, bounds=True)
    h = make(K, "f32", [(K.KVS_SRC_SINGLE, 0, 0)], 1, 1, 64, 2, 64)
    try:
        k = torch.zeros(48, 1, 64, device="cuda")
        k[16:32] = torch.linspace(-3e38, 3e38, 64, dtype=torch.float64).float().cuda()   # the largest magnitudes
        k[32:48] = torch.linspace(-1e-41, 2e-41, 64, dtype=torch.float64).float().cuda()  # denormal keys
        slots = [int(pool.table[0, t // 16]) * 16 + t % 16 for t in range(32)] + \
            [int(pool.table[1, 0]) * 16 + t for t in range(16)]
        K.kvshare_append_paged(h, pool.pages(), 0, k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert K.kvshare_sync_status(h) == K.KVS_OK
        hk = k.double().cpu().numpy()
        for i, page in enumerate((pool.table[0, 0], pool.table[0, 1], pool.table[1, 0])):
            c, s = paged.bounds(hk[16 * i:16 * i + 16, 0])
            assert np.array_equal(pool.codes[0, int(page), 0].cpu().numpy(), c)
            assert pool.scales[0, int(page), 0].item() == float(s)
    finally:
        K.kvshare_destroy(h)


# --------------------------------------------------------------------------------- plan
def plan_on_gpu(K, h, lens, new, table, ring, head, count, page, max_tokens, in_place=False):
    torch = torch_mod()
    t = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    B = len(lens)
    lens_d, state, ring_d, table_d = t(lens), t([head, count]), t(ring), t(table)
    lens_o, state_o = (lens_d, state) if in_place else (t([-9] * B), t([-9, -9]))
    start, slots, pos = t([-9] * (B + 1)), t([-9] * max_tokens), t([-9] * max_tokens)
    K.kvshare_plan_pages(h, lens_d, t(new), table_d, ring_d, state, lens_o, state_o, start, slots, pos, page)
    st = K.kvshare_sync_status(h)
    get = lambda x: x.cpu().numpy().tolist()  # noqa: E731
    return dict(block_table=get(table_d), ring=get(ring_d), ring_state=get(state_o), lengths=get(lens_o),
                token_start=get(start), slot_map=get(slots), position=get(pos)), st


@pytest.mark.parametrize("B,blocks,page,tokens,seed", [
    (1, 1, 16, 1, 0), (1, 40, 32, 500, 1), (7, 20, 16, 64, 2), (33, 30, 64, 3000, 3), (300, 12, 16, 9000, 4),
    (1024, 9, 128, 1024, 5), (4096, 5, 16, 20000, 6), (64, 64, 256, 40000, 7)])
def test_plan_against_the_oracle(K, B, blocks, page, tokens, seed):
    rng = np.random.default_rng(seed)
    cap = blocks * page
    N = int(B * blocks * 0.8) + 2
    ids = rng.permutation(N)
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 1, 1, 64, 1, 64)
    try:
        lens, table = [0] * B, np.full((B, blocks), -1).tolist()
        head, count = int(rng.integers(N)), N
        ring = [int(ids[(i - head) % N]) for i in range(N)]
        want_status = {frozenset(): K.KVS_OK, frozenset({"pool"}): K.KVS_ENOMEM, frozenset({"range"}): K.KVS_EINVAL,
                       frozenset({"range", "pool"}): K.KVS_EINVAL}
        for step in range(6):
            new = [int(x) for x in np.where(rng.random(B) < 0.15, -1, rng.integers(0, max(2, 3 * tokens // B), size=B))]
            if step % 2:
                new = [min(m, 1) for m in new]
            new = [m if n + m <= cap or rng.random() < 0.05 else 0 for n, m in zip(lens, new)]
            want, faults = paged.plan(lens, new, table, ring, head, count, page, tokens)
            got, st = plan_on_gpu(K, h, lens, new, table, ring, head, count, page, tokens, in_place=step % 3 == 2)
            for name in want:
                assert got[name] == [list(r) if isinstance(r, list) else int(r) for r in want[name]], (step, name)
            assert st == want_status[frozenset(faults)]
            lens, table, ring, (head, count) = got["lengths"], got["block_table"], got["ring"], got["ring_state"]
    finally:
        K.kvshare_destroy(h)


def test_plan_with_unusable_inputs(K):
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 1, 1, 64, 1, 64)
    try:
        table = [[0, -1], [1, -1]]
        for lens, new, head, count in (([-5, 16], [1, 1], 0, 2), ([16, 2 ** 30], [1, 1], 0, 2), ([16, 16], [2 ** 31 - 1, 1], 0, 2)):
            want, faults = paged.plan(lens, new, table, [2, 3, 0, 0], head, count, 16, 8)
            got, st = plan_on_gpu(K, h, lens, new, table, [2, 3, 0, 0], head, count, 16, 8)
            assert st == K.KVS_EINVAL and "range" in faults
            assert got["lengths"] == want["lengths"] and got["slot_map"] == want["slot_map"]
        for head, count in ((-1, 2), (4, 1), (0, 5), (0, -1)):                   # no free page in a ring like this
            got, st = plan_on_gpu(K, h, [16, 3], [1, 1], table, [2, 3, 0, 0], head, count, 16, 8)
            assert st == K.KVS_EINVAL
            assert got["lengths"] == [16, 4] and got["slot_map"][:2] == [16 + 3, -1] and got["block_table"] == table
        # more pages come back than the pool has room for: dropped
        got, st = plan_on_gpu(K, h, [32, 16], [-1, 0], [[0, 1], [1, -1]], [2, 3, 0, 0], 0, 3, 16, 8)
        assert st == K.KVS_EINVAL and got["ring_state"] == [0, 3] and got["lengths"] == [0, 16]
    finally:
        K.kvshare_destroy(h)


# ----------------------------------------------------------------------------- selection
SELECT = [
    # dtype, d, Hkv, g, page, lens, top, first, last, mix
    ("bf16", 64, 2, 4, 16, [0, 1, 200, 1000, 333], 5, 1, 1, False),
    ("bf16", 128, 2, 16, 32, [640, 2000], 9, 0, 2, True),
    ("bf16", 128, 3, 3, 64, [5000], 17, 2, 3, False),
    ("f32", 64, 1, 1, 16, [4100, 17], 33, 1, 1, True),
    ("f32", 128, 2, 8, 128, [1300, 0, 128], 4, 1, 1, False),
    ("bf16", 64, 1, 2, 16, [40000], 64, 1, 1, False),          # 2500 blocks: 512 threads
    ("bf16", 64, 1, 8, 16, [70000], 7, 1, 1, False),           # 4375 blocks: 1024 threads
    ("bf16", 64, 2, 2, 16, [100, 100], 7, 1, 1, False),        # every block kept: no scores needed
    ("bf16", 128, 1, 4, 128, [200, 0, 17], 3, 1, 1, True),     # lists longer than the block table's rows
    ("f32", 64, 2, 1, 16, [70, 33], 12, 2, 3, False),
]


@pytest.mark.parametrize("case", range(len(SELECT)))
def test_selection_and_sparse_decode_against_the_oracle(K, case):
    torch = torch_mod()
    dtype, d, Hkv, g, page, lens, top, first, last, mix = SELECT[case]
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)] + ([(K.KVS_SRC_MIX, 1, 0)] if mix else [])
    L, Hq, B = len(lmap), Hkv * g, len(lens)
    w = np.linspace(0.1, 0.9, L * Hkv, dtype=np.float32).reshape(L, Hkv) if mix else None
    pool = Pool(K, dtype, 2, Hkv, page, d, lens, seed=50 + case, bounds=True)
    h = make(K, dtype, lmap, Hq, Hkv, d, B, pool.table.shape[1] * page, w)
    try:
        q = queries(pool, L, Hq, seed=case, scale=2.0)
        q[0, 0, 0] = 0                                          # a query without codes
        sel = torch.full((L, B, Hkv, top), -9, dtype=torch.int32, device="cuda")
        pages = pool.pages()
        K.kvshare_select_pages(h, pages, q, sel, first, last)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        got = sel.cpu().numpy()
        hq = q.double().cpu().numpy()
        for l, (kind, s0, s1) in enumerate(lmap):
            for b, n in enumerate(lens):
                for j in range(Hkv):
                    def codes_of(p, src):
                        ph, sl = pool.table[b, p], (s0, s1)[src]
                        return pool.hcodes[sl, ph, j], pool.hscales[sl, ph, j]
                    want = paged.select(hq[l, b, j * g:(j + 1) * g], codes_of, n, page, top, first, last,
                                        w[l][j] if kind == K.KVS_SRC_MIX else None)
                    assert got[l, b, j].tolist() == want + [-1] * (top - len(want)), (l, b, j)
        out, lse = outputs(q)
        K.kvshare_decode_paged(h, pages, q, out, lse, selected=sel)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        check(out, lse, oracle_decode(pool, hq, lmap, w, selected=got), f"case {case}")
    finally:
        K.kvshare_destroy(h)


def test_equal_scores_keep_the_lowest_blocks(K):
    torch = torch_mod()
    pool = Pool(K, "bf16", 1, 2, 16, 64, [16 * 300], seed=1, bounds=True)
    pool.codes[:] = 5                                           # every page scores alike
    pool.scales[:] = 1.0
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 4, 2, 64, 1, 16 * 300)
    try:
        q = queries(pool, 1, 4, seed=1).abs()
        sel = torch.empty(1, 1, 2, 10, dtype=torch.int32, device="cuda")
        K.kvshare_select_pages(h, pool.pages(), q, sel, first=2, last=3)
        assert sel[0, 0].tolist() == [[0, 1, 2, 3, 4, 5, 6, 297, 298, 299]] * 2
    finally:
        K.kvshare_destroy(h)


def test_lists_of_the_callers_own(K):
    """Any order; entries outside a sequence's blocks are skipped and reported."""
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)]
    pool = Pool(K, "bf16", 1, 2, 16, 128, [100, 33, 0], seed=3)
    h = make(K, "bf16", lmap, 4, 2, 128, 3, 112)
    try:
        q = queries(pool, 1, 4, seed=2)
        sel = torch.tensor([[[[6, 0, 3], [2, 6, 5]], [[2, 1, 0], [1, 2, 0]], [[5, 5, 5], [0, 1, 2]]]], dtype=torch.int32, device="cuda")
        out, lse = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse, selected=sel)
        assert K.kvshare_sync_status(h) == K.KVS_OK             # the idle sequence's list is not read
        hq = q.double().cpu().numpy()
        check(out, lse, oracle_decode(pool, hq, lmap, selected=sel.cpu().numpy()), "own lists")
        sel[0, 0, 0] = torch.tensor([7, -1, 2 ** 31 - 1], dtype=torch.int32)
        sel[0, 1, 1] = torch.tensor([3, 1, -5], dtype=torch.int32)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse, selected=sel)
        assert K.kvshare_sync_status(h) == K.KVS_EINVAL
        check(out, lse, oracle_decode(pool, hq, lmap, selected=sel.cpu().numpy()), "bad lists")
    finally:
        K.kvshare_destroy(h)


# ------------------------------------------------------------------- a run of them together
def test_steps_of_a_serving_loop(K):
    """plan -> append -> select -> decode for several steps: prompts, single tokens, leaving and
    returning sequences; every step against a host model that only knows the tokens."""
    torch = torch_mod()
    B, Hq, Hkv, d, page, blocks, M = 5, 8, 2, 64, 16, 12, 160
    lmap = [(K.KVS_SRC_SINGLE, 0, 0), (K.KVS_SRC_SINGLE, 1, 0), (K.KVS_SRC_MIX, 0, 1)]
    w = np.array([[1, 1], [1, 1], [0.3, 0.8]], np.float32)
    N, slots_n, top = 40, 2, 4
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.full((slots_n, N, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    codes = torch.zeros(slots_n, N, Hkv, 2, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(slots_n, N, Hkv, device="cuda")
    table = torch.full((B, blocks), -1, **i32)
    lens = torch.zeros(B, **i32)
    ring, state = torch.arange(N, **i32), torch.tensor([0, N], **i32)
    start, slot_map, pos = torch.zeros(B + 1, **i32), torch.zeros(M, **i32), torch.zeros(M, **i32)
    h = make(K, "bf16", lmap, Hq, Hkv, d, B, blocks * page, w)
    pages = K.Pages(k=k, v=v, block_table=table, lengths=lens, bound_codes=codes, bound_scale=scales)
    gen = torch.Generator(device="cuda").manual_seed(0)
    hist_k = [[[] for _ in range(B)] for _ in range(slots_n)]
    hist_v = [[[] for _ in range(B)] for _ in range(slots_n)]
    steps = [[30, 0, 100, -1, 1], [1, 64, 1, 7, 1], [1, 1, -1, 1, 0], [1, 1, 50, 1, 1], [-1, 1, 1, 20, -1], [17, 1, 1, 1, 90]]
    try:
        for new in steps:
            K.kvshare_plan_pages(h, lens, torch.tensor(new, **i32), table, ring, state, lens, state, start, slot_map, pos, page)
            qkv = torch.randn(slots_n, M, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
            for s in range(slots_n):
                K.kvshare_append_paged(h, pages, s, qkv[s, :, Hq:Hq + Hkv], qkv[s, :, Hq + Hkv:], slot_map)
            q = torch.randn(3, B, Hq, d, generator=gen, device="cuda").to(torch.bfloat16)
            sel = torch.empty(3, B, Hkv, top, **i32)
            out, lse = outputs(q)
            sparse, slse = outputs(q)
            K.kvshare_decode_paged(h, pages, q, out, lse)
            K.kvshare_select_pages(h, pages, q, sel)
            K.kvshare_decode_paged(h, pages, q, sparse, slse, selected=sel)
            assert K.kvshare_sync_status(h) == K.KVS_OK
            at = 0
            for b, m in enumerate(new):
                for s in range(slots_n):
                    if m < 0:
                        hist_k[s][b], hist_v[s][b] = [], []
                    for i in range(max(m, 0)):
                        hist_k[s][b].append(qkv[s, at + i, Hq:Hq + Hkv])
                        hist_v[s][b].append(qkv[s, at + i, Hq + Hkv:])
                at += max(m, 0)
            assert lens.tolist() == [len(x) for x in hist_k[0]]
            hq, chosen = q.double().cpu().numpy(), sel.cpu().numpy()
            for b in range(B):
                n = len(hist_k[0][b])
                if n == 0:
                    assert not out[:, b].any() and torch.isneginf(lse[:, b]).all()
                    continue
                kk = [torch.stack(hist_k[s][b]).double().cpu().numpy() for s in range(slots_n)]
                vv = [torch.stack(hist_v[s][b]).double().cpu().numpy() for s in range(slots_n)]
                for l, (kind, s0, s1) in enumerate(lmap):
                    for j in range(Hkv):
                        def mixed(x):
                            if kind != K.KVS_SRC_MIX:
                                return x[s0][:, j]
                            wj = float(w[l, j])
                            return wj * x[s0][:, j] + float(np.float32(1) - w[l, j]) * x[s1][:, j]
                        h8 = slice(j * 4, j * 4 + 4)
                        rows = np.concatenate([np.arange(c * page, min(n, c * page + page)) for c in chosen[l, b, j] if c >= 0])
                        for got, glse, pick in ((out, lse, np.arange(n)), (sparse, slse, rows)):
                            o, z = paged.attend(hq[l, b, h8], mixed(kk)[pick], mixed(vv)[pick], d ** -0.5)
                            # scores below 2^5 in magnitude, values below 2^3: 20 steps of 2^-22 of either, twice
                            assert np.abs(got[l, b, h8].cpu().numpy() - o).max() < 2 * 20 * 2.0 ** -22 * 2 ** 8
                            assert np.abs(glse[l, b, h8].cpu().numpy() - z).max() < 20 * 2.0 ** -22 * 2 ** 5
            if max(len(x) for x in hist_k[0]) <= top * page:
                assert torch.equal(out, sparse)
    finally:
        K.kvshare_destroy(h)


def test_a_captured_step_follows_its_inputs(K):
    """plan, append, select and decode in one CUDA graph, replayed as the sequences grow."""
    torch = torch_mod()
    B, Hq, Hkv, d, page, blocks = 3, 4, 2, 64, 16, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)]
    h = make(K, "bf16", lmap, Hq, Hkv, d, B, blocks * page)

    def fresh():
        z = torch.full((1, 24, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        return dict(k=z.clone(), v=z.clone(), codes=torch.zeros(1, 24, Hkv, 2, d, dtype=torch.int8, device="cuda"),
                    scales=torch.zeros(1, 24, Hkv, device="cuda"), table=torch.full((B, blocks), -1, **i32),
                    lens=torch.zeros(B, **i32), ring=torch.arange(24, **i32), state=torch.tensor([0, 24], **i32),
                    start=torch.zeros(B + 1, **i32), slots=torch.zeros(B, **i32), pos=torch.zeros(B, **i32),
                    new=torch.ones(B, **i32), kv=torch.zeros(2, B, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                    q=torch.zeros(1, B, Hq, d, dtype=torch.bfloat16, device="cuda"),
                    sel=torch.zeros(1, B, Hkv, 3, **i32), out=torch.zeros(1, B, Hq, d, device="cuda"),
                    lse=torch.zeros(1, B, Hq, device="cuda"))

    def step(s, stream=None):
        pages = K.Pages(k=s["k"], v=s["v"], block_table=s["table"], lengths=s["lens"], bound_codes=s["codes"],
                        bound_scale=s["scales"])
        K.kvshare_plan_pages(h, s["lens"], s["new"], s["table"], s["ring"], s["state"], s["lens"], s["state"],
                             s["start"], s["slots"], s["pos"], page)
        K.kvshare_append_paged(h, pages, 0, s["kv"][0], s["kv"][1], s["slots"])
        K.kvshare_select_pages(h, pages, s["q"], s["sel"])
        K.kvshare_decode_paged(h, pages, s["q"], s["out"], s["lse"], selected=s["sel"])

    try:
        a, b = fresh(), fresh()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(fresh())                                       # first launches outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(a)
        gen = torch.Generator(device="cuda").manual_seed(5)
        for i in range(70):
            kv = torch.randn(2, B, Hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
            q = torch.randn(1, B, Hq, d, generator=gen, device="cuda").to(torch.bfloat16)
            new = torch.tensor([1, 1 if i % 3 else 0, -1 if i == 40 else 1], **i32)
            for s in (a, b):
                s["kv"].copy_(kv), s["q"].copy_(q), s["new"].copy_(new)
            g.replay()
            step(b)
            assert K.kvshare_sync_status(h) == K.KVS_OK
            for name in ("lens", "table", "ring", "state", "slots", "sel", "out", "lse", "codes", "scales"):
                assert torch.equal(a[name], b[name]), (i, name)
        assert a["lens"].tolist()[0] == 70
    finally:
        K.kvshare_destroy(h)


def test_two_contexts_on_two_streams(K):
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0)]
    pools = [Pool(K, "bf16", 1, 2, 32, 128, [3000, 5, 700], seed=s) for s in (1, 2)]
    hs = [make(K, "bf16", lmap, 8, 2, 128, 3, 3008) for _ in pools]
    try:
        qs = [queries(p, 1, 8, seed=s) for s, p in enumerate(pools)]
        alone = []
        for h, p, q in zip(hs, pools, qs):
            out, lse = outputs(q)
            K.kvshare_decode_paged(h, p.pages(), q, out, lse)
            alone.append(out)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in pools]
        outs = [[outputs(q) for _ in range(20)] for q in qs]
        pages = [p.pages() for p in pools]
        torch.cuda.synchronize()
        for i in range(20):
            for h, p, q, s, o in zip(hs, pages, qs, streams, outs):
                K.kvshare_decode_paged(h, p, q, o[i][0], o[i][1], stream=s)
        for h, s in zip(hs, streams):
            assert K.kvshare_sync_status(h, s) == K.KVS_OK
        for o, want in zip(outs, alone):
            assert all(torch.equal(x[0], want) for x in o)
    finally:
        for h in hs:
            K.kvshare_destroy(h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_wait_that_runs_out_is_reported_and_the_context_works_on(K, dtype):
    torch = torch_mod()
    pool = Pool(K, dtype, 1, 2, 16, 64, [300, 40], seed=1)
    h = make(K, dtype, [(K.KVS_SRC_SINGLE, 0, 0)], 4, 2, 64, 2, 304)
    try:
        q = queries(pool, 1, 4, seed=1)
        out, lse = outputs(q)
        K.kvshare_debug_stall_next(h, True)
        K.kvshare_decode_paged(h, pool.pages(), q, out, lse)
        assert K.kvshare_sync_status(h) == K.KVS_ETIMEOUT
        again, alse = outputs(q)
        K.kvshare_decode_paged(h, pool.pages(), q, again, alse)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        assert torch.equal(out, again) and torch.equal(lse, alse)              # only the spare barrier was waited on
    finally:
        K.kvshare_destroy(h)


def test_sizes_past_the_counters_are_refused(K):
    import ctypes
    torch = torch_mod()
    pool = Pool(K, "bf16", 1, 2, 16, 64, [40, 3], seed=1)
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 4, 2, 64, 2, 48)
    try:
        lib, p = K._lib, pool.pages()
        q = queries(pool, 1, 4, seed=1)
        out, lse = outputs(q)
        sel = torch.zeros(64, dtype=torch.int32, device="cuda")
        n0 = K.kvshare_launch_count(h)

        def call(f, **kw):
            c = K.kvshare_pages.from_buffer_copy(p._c)
            for k, x in kw.items():
                setattr(c, k, x)
            r = ctypes.byref(c)
            if f == "decode":
                return lib.kvshare_decode_paged(h, r, q.data_ptr(), out.data_ptr(), lse.data_ptr(), None, 0, 0, 1, None)
            if f == "append":
                return lib.kvshare_append_paged(h, r, 0, q.data_ptr(), q.data_ptr(), 128, 128, sel.data_ptr(), 1, None)
            return lib.kvshare_select_pages(h, r, q.data_ptr(), sel.data_ptr(), 4, 1, 1, 0, 1, None)
        for f in ("decode", "append", "select"):
            for kw in (dict(page_size=24), dict(page_size=8), dict(page_size=512), dict(num_pages=0), dict(slots=0),
                       dict(num_pages=1 << 27), dict(slots=1 << 30), dict(k=None), dict(v=p._c.v + 2)):
                assert call(f, **kw) == K.KVS_EINVAL, (f, kw)
        for f in ("decode", "select"):
            for kw in (dict(batch=0), dict(batch=3), dict(max_blocks=0), dict(max_blocks=4), dict(max_blocks=1 << 27),
                       dict(block_table=None), dict(lengths=p._c.lengths + 1)):
                assert call(f, **kw) == K.KVS_EINVAL, (f, kw)
        i = sel.data_ptr()
        plan = lambda B=2, P=2, ps=16, N=4, M=4: lib.kvshare_plan_pages(h, *[i] * 10, B, P, ps, N, M, None)  # noqa: E731
        for kw in (dict(B=0), dict(P=0), dict(ps=17), dict(N=0), dict(M=0), dict(P=1 << 27), dict(N=1 << 27),
                   dict(M=(1 << 30) + 1)):
            assert plan(**kw) == K.KVS_EINVAL, kw
        assert plan(B=4097) == K.KVS_EUNSUPPORTED
        assert K.kvshare_launch_count(h) == n0 and K.kvshare_sync_status(h) == K.KVS_OK
    finally:
        K.kvshare_destroy(h)


# ------------------------------------------------------------------------------- refusals
def test_refusals_launch_nothing(K):
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0), (K.KVS_SRC_MIX, 0, 1)]
    pool = Pool(K, "bf16", 2, 2, 16, 64, [40, 3], seed=1, bounds=True)
    h = make(K, "bf16", lmap, 4, 2, 64, 2, 48, np.full((2, 2), 0.5, np.float32))
    try:
        pages = pool.pages()
        q = queries(pool, 2, 4, seed=1)
        out, lse = outputs(q)
        sel = torch.zeros(2, 2, 2, 2, dtype=torch.int32, device="cuda")
        n0 = K.kvshare_launch_count(h)
        dec = lambda *a, **k: K.kvshare_decode_paged(h, *a, check=False, **k)  # noqa: E731
        assert dec(pages, q.float(), out) == K.KVS_EINVAL                      # type
        assert dec(pages, q, out.bfloat16()) == K.KVS_EINVAL
        assert dec(pages, q.transpose(1, 2), out) == K.KVS_EINVAL              # shape, strides
        assert dec(pages, q, out[..., :32]) == K.KVS_EINVAL
        assert dec(pages, q.cpu(), out) == K.KVS_EINVAL                        # host memory
        assert dec(pages, q, out, lse[:1]) == K.KVS_EINVAL                     # too few layers
        assert dec(pages, q, out, lse, 0, 3) == K.KVS_EINVAL
        assert dec(pages, q, out, lse, 1, 0) == K.KVS_EINVAL
        assert dec(pages, q, out, lse, selected=sel.long()) == K.KVS_EINVAL
        assert dec(pages, q, out, lse, selected=sel[..., :0].contiguous()) == K.KVS_EINVAL
        s = lambda *a, **k: K.kvshare_select_pages(h, *a, check=False, **k)  # noqa: E731
        assert s(pages, q, sel, first=2, last=1) == K.KVS_EINVAL               # first + last > top
        assert s(pages, q, sel, first=-1, last=1) == K.KVS_EINVAL
        assert s(pages, q, sel, first=0, last=0) == K.KVS_EINVAL
        assert s(pool.pages(bound_codes=None, bound_scale=None), q, sel) == K.KVS_EINVAL
        x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
        slots = torch.zeros(2, dtype=torch.int32, device="cuda")
        ap = lambda *a: K.kvshare_append_paged(h, *a, check=False)  # noqa: E731
        assert ap(pages, 2, x, x, slots) == K.KVS_EINVAL                       # no such slot
        assert ap(pages, -1, x, x, slots) == K.KVS_EINVAL
        assert ap(pages, 0, x[:, :1], x, slots) == K.KVS_EINVAL
        assert ap(pages, 0, x.float(), x, slots) == K.KVS_EINVAL
        assert ap(pages, 0, x, x.transpose(1, 2).contiguous().transpose(1, 2), slots) == K.KVS_EINVAL
        odd = torch.zeros(2, 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, :128].view(2, 2, 64)
        assert ap(pages, 0, odd, x, slots) == K.KVS_EINVAL                     # rows not 16-byte aligned
        assert ap(pages, 0, x, x, slots.long()) == K.KVS_EINVAL
        # a pool of other heads, a table longer than the context, a slot the pool lacks
        other = Pool(K, "bf16", 2, 1, 16, 64, [40, 3], seed=1)
        assert dec(other.pages(), q, out) == K.KVS_EINVAL
        longer = Pool(K, "bf16", 2, 2, 16, 64, [65, 3], seed=1)
        assert dec(longer.pages(), q, out) == K.KVS_EINVAL
        one = Pool(K, "bf16", 1, 2, 16, 64, [40, 3], seed=1)
        assert dec(one.pages(), q, out) == K.KVS_EINVAL
        big = Pool(K, "bf16", 2, 2, 16, 64, [1, 1, 1], seed=1)                 # more sequences than max_batch
        assert dec(big.pages(), torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.zeros(2, 3, 4, 64, device="cuda")) == K.KVS_EINVAL
        with pytest.raises(K.KVShareError):
            pool.pages(lengths=pool.lengths[:1])
        with pytest.raises(K.KVShareError):
            pool.pages(v=pool.v[:, :-1])
        with pytest.raises(K.KVShareError):
            pool.pages(bound_scale=None)
        with pytest.raises(K.KVShareError):
            K.kvshare_decode_paged(h, pages, q, out, lse, 0, 3)
        assert K.kvshare_launch_count(h) == n0
        K.kvshare_set_map(h, [(K.KVS_SRC_LOWRANK, 0, 0), (K.KVS_SRC_SINGLE, 0, 0)])
        assert dec(pages, q, out) == K.KVS_EUNSUPPORTED
        assert s(pages, q, sel) == K.KVS_EUNSUPPORTED
        assert K.kvshare_launch_count(h) == n0 and K.kvshare_sync_status(h) == K.KVS_OK
    finally:
        K.kvshare_destroy(h)


# -------------------------------------------------------------------------------- example
def test_the_readme_example_of_a_paged_cache_runs():
    import os
    import re
    torch = torch_mod()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    paged_block = [b for b in blocks if "kvshare_plan_pages" in b]
    assert len(paged_block) == 1
    names = {}
    torch.manual_seed(0)
    exec(compile(paged_block[0], "README.md", "exec"), names)      # noqa: S102  (the repository's own text)
    # one token each: every head's output is its kv head's value v. The one weight p divides itself
    # out: (p v) (1 / p) with p's three parts and their sum off by at most 6 half steps together
    # (remainder 1, tensor-core sums 4, joining sum 1), reciprocal and product 1 each: 2^-21
    out, v = names["out"], names["v"]
    assert names["lens"].tolist() == [1] * 32
    want = v[10, names["table"][:, 0].long(), :, 0].repeat_interleave(8, dim=1).float()
    assert ((out[21] - want).abs() <= want.abs() * 2.0 ** -21).all()

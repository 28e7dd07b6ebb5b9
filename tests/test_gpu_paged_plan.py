"""Planning with pages that do not exist, and what is reported of a step: against the oracle."""
import numpy as np
import pytest

import oracle.paged_ref as paged
from test_gpu_paged import make, plan_on_gpu
from paged_helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from cross_layer_kv_shared_b200 import kvshare
    return kvshare


@pytest.fixture
def ctx(K):
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 2, 2, 64, 8, 4096)
    yield h
    K.kvshare_destroy(h)


def agree(got, want):
    for name in want:
        assert got[name] == [list(r) if isinstance(r, list) else int(r) for r in want[name]], name


# pages whose slot numbers wrap in 32 bits to rows of pages 0, 1 and 3 at 16 tokens a page among them
BAD = [-1, 12, 1 << 28, 0x10000001, (1 << 28) + 3, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("bad", BAD)
def test_pages_outside_the_pool_get_no_slot_and_are_reported(K, ctx, bad, page):
    N, lens, new = 12, [page + 3, 5, 2 * page, 0], [2, 1, page + 1, 3]
    good = [[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, -1, -1], [-1] * 4]
    free = [5, 6, 7, 8, 9, 10, 11, 0, 0, 0, 0, 0]
    for where in ("table", "ring"):
        table, ring = [list(r) for r in good], list(free)
        if where == "table":
            table[0][1] = bad                  # the page the next tokens of sequence 0 continue in
        else:
            ring[1] = bad                      # the second page that sequence 2 takes
        want, faults = paged.plan(lens, new, table, ring, 0, 7, page, 2 * page, num_pages=N)
        got, st = plan_on_gpu(K, ctx, lens, new, table, ring, 0, 7, page, 2 * page)
        assert st == K.KVS_EINVAL and faults == {"range"}
        agree(got, want)
        live = [s for s in got["slot_map"] if s >= 0]
        assert len(set(live)) == len(live) and all(s < N * page for s in live)
    got, st = plan_on_gpu(K, ctx, lens, new, good, free, 0, 7, page, 2 * page)        # nothing is left behind
    assert st == K.KVS_OK and min(got["slot_map"][:sum(new)]) >= 0


@pytest.mark.parametrize("bad", BAD)
def test_pages_outside_the_pool_are_reported_where_they_return(K, ctx, bad):
    table = [[3, bad, 5], [1, -1, -1]]
    ring = [9, 8, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0]
    want, faults = paged.plan([40, 4], [-1, 1], table, ring, 0, 2, 16, 8, num_pages=12)
    got, st = plan_on_gpu(K, ctx, [40, 4], [-1, 1], table, ring, 0, 2, 16, 8)
    assert st == K.KVS_EINVAL and faults == {"range"}
    agree(got, want)


def test_no_other_row_is_written_for_a_page_outside_the_pool(K, ctx):
    """plan and append together: the rows of the other sequences stay as they were, bit for bit."""
    torch = torch_mod()
    i32 = dict(dtype=torch.int32, device="cuda")
    N, page = 12, 16
    k = torch.randn(1, N, 2, page, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn(1, N, 2, page, 64, device="cuda").to(torch.bfloat16)
    before = k.clone(), v.clone()
    table = torch.tensor([[0, 0x10000001], [1, -1]], **i32)
    lens, state = torch.tensor([20, 7], **i32), torch.tensor([0, 3], **i32)
    ring = torch.tensor([5, 6, 7] + [0] * 9, **i32)
    start, slots, pos = torch.zeros(3, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32)
    K.kvshare_plan_pages(ctx, lens, torch.tensor([2, 1], **i32), table, ring, state, lens, state, start, slots, pos, page)
    new = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pages = K.Pages(k=k, v=v, block_table=table, lengths=lens)
    K.kvshare_append_paged(ctx, pages, 0, new, new, slots)
    assert K.kvshare_sync_status(ctx) == K.KVS_EINVAL
    assert slots.tolist() == [-1, -1, page + 7, -1] and lens.tolist() == [22, 8]
    for x, was in zip((k, v), before):
        was[0, 1, :, 7] = 7.0
        assert torch.equal(x.view(torch.int16), was.view(torch.int16))


@pytest.mark.parametrize("length", [33, 2 ** 31 - 1, -1, -2 ** 31])
def test_a_leaving_sequence_of_unknown_length_returns_no_page(K, ctx, length):
    """Clamped to its row of the table it would put whatever the row holds into the ring, pages of others too."""
    table = [[3, 1], [1, -1]]                          # the second entry of row 0 is stale: page 1 is row 1's
    ring = [9, 8, 0, 0, 0, 0, 0, 0, 0, 0]
    want, faults = paged.plan([length, 4], [-1, 1], table, ring, 0, 2, 16, 8, num_pages=10)
    got, st = plan_on_gpu(K, ctx, [length, 4], [-1, 1], table, ring, 0, 2, 16, 8)
    assert st == K.KVS_EINVAL and faults == {"range"}
    assert got["ring_state"] == [0, 2] and got["ring"] == ring and got["lengths"] == [0, 5]
    agree(got, want)


def test_two_kinds_of_fault_are_both_reported(K, ctx):
    """One sequence past its row of the table, another without pages: neither report is lost."""
    table, ring = [[0, -1], [1, -1]], [2, 3, 0, 0]
    want, faults = paged.plan([16, 16], [17, 1], table, ring, 0, 0, 16, 32, num_pages=4)
    got, st = plan_on_gpu(K, ctx, [16, 16], [17, 1], table, ring, 0, 0, 16, 32)
    assert faults == {"range", "pool"}
    agree(got, want)
    assert st == K.KVS_EINVAL
    assert K.kvshare_sync_status(ctx) == K.KVS_ENOMEM
    assert K.kvshare_sync_status(ctx) == K.KVS_OK
    # a time-out on top of both: all three, one a call
    K.kvshare_debug_stall_next(ctx, True)
    torch = torch_mod()
    i32 = dict(dtype=torch.int32, device="cuda")
    t = lambda x: torch.tensor(x, **i32)  # noqa: E731
    state, start, slots = t([0, 0]), torch.zeros(3, **i32), torch.zeros(32, **i32)
    K.kvshare_plan_pages(ctx, t([16, 16]), t([17, 1]), t(table), t(ring), state, torch.zeros(2, **i32),
                         torch.zeros(2, **i32), start, slots, torch.zeros(32, **i32), 16)
    kv = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    K.kvshare_decode_paged(ctx, K.Pages(k=kv, v=kv, block_table=t([[0, 1], [2, 3]]), lengths=t([3, 0])), q,
                           torch.zeros(q.shape, device="cuda"))
    seen = [K.kvshare_sync_status(ctx) for _ in range(4)]
    assert seen == [K.KVS_ETIMEOUT, K.KVS_EINVAL, K.KVS_ENOMEM, K.KVS_OK]

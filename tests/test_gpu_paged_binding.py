"""The paged entry points take what the others take: a handle by value, sizes as numpy integers."""
import numpy as np
import pytest

from paged_helpers import Pool, torch_mod
from test_gpu_paged import make, outputs, queries

pytestmark = pytest.mark.gpu


def test_handles_by_value_and_numpy_sizes():
    from cross_layer_kv_shared_b200 import kvshare as K
    torch = torch_mod()
    lmap = [(K.KVS_SRC_SINGLE, 0, 0), (K.KVS_SRC_SINGLE, 1, 0)]
    pool = Pool(K, "bf16", 2, 2, 16, 64, [40, 3], seed=1, bounds=True)
    h = make(K, "bf16", lmap, 4, 2, 64, 2, 48)
    i32 = dict(dtype=torch.int32, device="cuda")
    i = np.int64
    try:
        pages, q = pool.pages(), queries(pool, 2, 4, seed=1)
        kv = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
        slot = torch.tensor([int(pool.table[0, 2]) * 16 + 7], **i32)
        results = []
        for handle in (h, h.value):
            (out, lse), sel = outputs(q), torch.full((2, 2, 2, 2), -9, **i32)
            state, start, slots, pos = torch.tensor([0, 4], **i32), *(torch.zeros(n, **i32) for n in (3, 4, 4))
            table, lens = torch.zeros(2, 3, **i32), torch.zeros(2, **i32)
            K.kvshare_plan_pages(handle, lens, torch.ones(2, **i32), table, torch.arange(4, **i32), state, lens, state,
                                 start, slots, pos, i(16))
            K.kvshare_append_paged(handle, pages, i(1), kv, kv, slot)
            K.kvshare_select_pages(handle, pages, q, sel, i(1), i(1), i(0), i(2))
            K.kvshare_decode_paged(handle, pages, q, out, lse, i(1), i(2), selected=sel)
            assert K.kvshare_sync_status(handle) == K.KVS_OK
            assert slots.tolist() == [0, 16, -1, -1] and torch.isnan(out[0]).all()
            results.append((out[1], lse[1], sel, pool.codes.clone()))
        for a, b in zip(*results):
            assert torch.equal(a, b)
    finally:
        K.kvshare_destroy(h)
    assert K.kvshare_decode_paged(None, pages, q, out, lse, check=False) == K.KVS_EINVAL
    assert K.kvshare_select_pages(None, pages, q, sel, check=False) == K.KVS_EINVAL
    assert K.kvshare_append_paged(None, pages, 0, kv, kv, slot, check=False) == K.KVS_EINVAL


@pytest.mark.parametrize("bounds", [False, True], ids=["rows", "bounds"])
def test_rows_in_any_order_are_written(bounds):
    """Skipped entries, gaps and a shuffled order: the rows are right whether or not bounds are kept; a page
    whose entries are in order has right bounds beside one whose entries are not."""
    from cross_layer_kv_shared_b200 import kvshare as K
    import oracle.paged_ref as paged
    torch = torch_mod()
    pool = Pool(K, "bf16", 1, 2, 16, 64, [48, 16], seed=4, bounds=True)
    p0, p1, p2, p3 = (int(pool.table[b, i]) * 16 for b, i in ((0, 0), (0, 1), (0, 2), (1, 0)))
    slots = [p0 + 3, -1, p0 + 5, p0 + 4, p2 + 9, p0 + 15, p3, p3 + 1, p3 + 2, -1, p1 + 15, p0 + 1, p2 + 8]
    new = torch.randn(len(slots), 2, 64, device="cuda").to(torch.bfloat16)
    want_k, want_v = pool.host()
    paged.append(want_k[0], want_v[0], None, None, new.double().cpu().numpy(), (-new).double().cpu().numpy(), slots, 16)
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)], 2, 2, 64, 2, 48)
    try:
        pages = pool.pages() if bounds else pool.pages(bound_codes=None, bound_scale=None)
        K.kvshare_append_paged(h, pages, 0, new, -new, torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert K.kvshare_sync_status(h) == K.KVS_OK
        got_k, got_v = pool.host()
        assert np.array_equal(got_k, want_k, equal_nan=True) and np.array_equal(got_v, want_v, equal_nan=True)
        if bounds:
            for slot, rows in ((p1, 16), (p3, 3)):
                for j in range(2):
                    c, s = paged.bounds(got_k[0, slot // 16, j, :rows])
                    assert np.array_equal(pool.codes[0, slot // 16, j].cpu().numpy(), c)
                    assert pool.scales[0, slot // 16, j].item() == float(s)
    finally:
        K.kvshare_destroy(h)


def test_a_layer_uses_a_copy_of_another_layers_selection():
    from cross_layer_kv_shared_b200 import kvshare as K
    torch = torch_mod()
    pool = Pool(K, "bf16", 1, 2, 16, 128, [400, 90, 0], seed=5, bounds=True)
    h = make(K, "bf16", [(K.KVS_SRC_SINGLE, 0, 0)] * 3, 8, 2, 128, 3, 400)
    try:
        q = queries(pool, 3, 8, seed=1)
        sel = torch.full((3, 3, 2, 4), -9, dtype=torch.int32, device="cuda")
        (out, lse), (alone, alse) = outputs(q), outputs(q)
        pages = pool.pages()
        K.kvshare_select_pages(h, pages, q, sel, l0=0, l1=1)
        assert (sel[1:] == -9).all()
        sel[1:] = sel[0]
        K.kvshare_decode_paged(h, pages, q, out, lse, selected=sel)
        for l in range(3):                              # each layer against the same list, by itself
            K.kvshare_decode_paged(h, pages, q, alone, alse, l, l + 1, selected=sel)
        assert K.kvshare_sync_status(h) == K.KVS_OK
        assert torch.equal(out, alone) and torch.equal(lse, alse) and torch.isfinite(out).all()
    finally:
        K.kvshare_destroy(h)

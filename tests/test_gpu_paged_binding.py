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

"""Argument checks of the paged entry points that need no GPU."""
import ctypes


def test_null_and_shape_checks_run_before_any_cuda_call():
    from cross_layer_kv_shared_b200 import kvshare as K
    lib = K._lib
    assert lib.kvshare_plan_pages(*[None] * 11, 1, 1, 16, 1, 1, None) == K.KVS_EINVAL
    assert lib.kvshare_append_paged(None, None, 0, None, None, 0, 0, None, 1, None) == K.KVS_EINVAL
    assert lib.kvshare_decode_paged(None, None, None, None, None, None, 0, 0, 0, None) == K.KVS_EINVAL
    assert lib.kvshare_select_pages(None, None, None, None, 1, 0, 1, 0, 0, None) == K.KVS_EINVAL


def test_struct_layout_matches_the_header():
    from cross_layer_kv_shared_b200 import kvshare as K
    p = K.kvshare_pages
    assert [p.k.offset, p.v.offset, p.bound_codes.offset, p.bound_scale.offset] == [0, 8, 16, 24]
    assert [p.slots.offset, p.num_pages.offset, p.page_size.offset] == [32, 36, 40]
    assert [p.block_table.offset, p.lengths.offset, p.batch.offset, p.max_blocks.offset] == [48, 56, 64, 68]
    assert ctypes.sizeof(p) == 72


def test_host_tensors_are_refused():
    import pytest
    import torch
    from cross_layer_kv_shared_b200 import kvshare as K
    k = torch.zeros(1, 2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(K.KVShareError):
        K.Pages(k=k, v=k, block_table=torch.zeros(1, 1, dtype=torch.int32), lengths=torch.zeros(1, dtype=torch.int32))
    i = torch.zeros(1, dtype=torch.int32)
    st = K.kvshare_plan_pages(ctypes.c_void_p(), i, i, i.view(1, 1), i, i, i, i, i, i, i, 16, check=False)
    assert st == K.KVS_EINVAL

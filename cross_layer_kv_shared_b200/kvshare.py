"""ctypes binding of libkvshare (include/kvshare.h): argument marshalling only.

Every function keeps the C name. Tensors are torch tensors on the CUDA device
(torch is used for device memory and streams only); every step of the
computation runs in the library's kernels. A missing library raises at import:
there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvshare.so")

KVS_OK, KVS_EINVAL, KVS_EUNSUPPORTED, KVS_ENOMEM, KVS_ECUDA, KVS_ETIMEOUT = range(6)
KVS_F32, KVS_BF16 = 0, 1
KVS_SRC_SINGLE, KVS_SRC_MIX, KVS_SRC_LOWRANK = 0, 1, 2


class kvshare_config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("softmax_scale", ctypes.c_float),
                ("basis_rank", ctypes.c_int), ("max_resid_rank", ctypes.c_int), ("max_batch", ctypes.c_int),
                ("max_context", ctypes.c_int)]


class kvshare_layer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("src0", ctypes.c_int), ("src1", ctypes.c_int)]


class kvshare_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("slots", ctypes.c_int),
                ("coef_k", ctypes.c_void_p), ("coef_v", ctypes.c_void_p),
                ("basis_k", ctypes.c_void_p), ("basis_v", ctypes.c_void_p),
                ("u_k", ctypes.c_void_p), ("u_v", ctypes.c_void_p),
                ("s_k", ctypes.c_void_p), ("s_v", ctypes.c_void_p),
                ("r_k", ctypes.c_void_p), ("r_v", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("pairs", ctypes.c_int),
                ("batch", ctypes.c_int), ("context", ctypes.c_int),
                ("lengths", ctypes.c_void_p)]


class kvshare_pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("bound_codes", ctypes.c_void_p),
                ("bound_scale", ctypes.c_void_p), ("slots", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("block_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("batch", ctypes.c_int), ("max_blocks", ctypes.c_int)]


class KVShareError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kvshare_status_string(status)} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m cross_layer_kv_shared_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, V = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    sig = {
        "kvshare_create": ([ctypes.POINTER(kvshare_config), ctypes.POINTER(ctypes.c_void_p)], I),
        "kvshare_destroy": ([P], I),
        "kvshare_set_map": ([P, ctypes.POINTER(kvshare_layer), P], I),
        "kvshare_decode": ([P, ctypes.POINTER(kvshare_cache), P, P, P, I, I, V], I),
        "kvshare_decode_host": ([P, ctypes.POINTER(kvshare_cache), P, P, P, I, I, V], I),
        "kvshare_decode_stats": ([P, ctypes.POINTER(kvshare_cache), P, P, P, P, P, P, P, I, I, V], I),
        "kvshare_prefill": ([P, ctypes.POINTER(kvshare_cache), P, P, P, I, I, I, V], I),
        "kvshare_pack_residual": ([P, P, P, P, P, P, P, P, P, I, I, V], I),
        "kvshare_append_lowrank": ([P, ctypes.POINTER(kvshare_cache), P, P, P, P, V], I),
        "kvshare_plan_pages": ([P] * 11 + [I, I, I, I, I, V], I),
        "kvshare_append_paged": ([P, ctypes.POINTER(kvshare_pages), I, P, P, ctypes.c_longlong, ctypes.c_longlong, P,
                                  I, V], I),
        "kvshare_decode_paged": ([P, ctypes.POINTER(kvshare_pages), P, P, P, P, I, I, I, V], I),
        "kvshare_select_pages": ([P, ctypes.POINTER(kvshare_pages), P, P, I, I, I, I, I, V], I),
        "kvshare_sync_status": ([P, V], I),
        "kvshare_set_splits": ([P, I], I),
        "kvshare_set_kv_overlap": ([P, I], I),
        "kvshare_set_layer_order": ([P, P], I),
        "kvshare_debug_stall_next": ([P, I], I),
        "kvshare_debug_set_grid": ([P, I], I),
        "kvshare_launch_count": ([P], ctypes.c_uint64),
        "kvshare_status_string": ([I], ctypes.c_char_p),
        "kvshare_decode_layer_noalloc": ([P, P, P, P, P, P, I, I, I, I, I, I, I, I, V], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def kvshare_status_string(status: int) -> str:
    return _lib.kvshare_status_string(int(status)).decode()


def _check(status: int, where: str) -> int:
    if status != KVS_OK:
        raise KVShareError(status, where)
    return status


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return int(t.data_ptr()) if hasattr(t, "data_ptr") else int(t)


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


# (query heads, (kv heads, head dim, dtype)) of each live context: what the paged entry points
# check their tensors against
_configs = {}


def kvshare_create(num_layers: int, num_q_heads: int, num_kv_heads: int, head_dim: int, dtype: int,
                   max_batch: int, max_context: int, softmax_scale: float = 0.0, basis_rank: int = 32,
                   max_resid_rank: int = 16, check: bool = True):
    """Returns (status, handle); raises KVShareError on failure when ``check``."""
    cfg = kvshare_config(num_layers, num_q_heads, num_kv_heads, head_dim, dtype, softmax_scale, basis_rank,
                         max_resid_rank, max_batch, max_context)
    h = ctypes.c_void_p()
    st = _lib.kvshare_create(ctypes.byref(cfg), ctypes.byref(h))
    if check:
        _check(st, "kvshare_create")
    if st == KVS_OK:
        _configs[h.value] = (num_q_heads, (num_kv_heads, head_dim, dtype))
    return st, h


def _config(h):
    """The sizes of a live context, by its handle (the c_void_p or its value), or None."""
    return _configs.get(getattr(h, "value", h))


def kvshare_destroy(h) -> int:
    _configs.pop(getattr(h, "value", h), None)
    return _lib.kvshare_destroy(h)


def kvshare_set_map(h, layer_map: Sequence, w=None, check: bool = True) -> int:
    """layer_map: (kind, src0, src1) per layer; w: host float32 array [L][Hkv] or None."""
    arr = (kvshare_layer * len(layer_map))(*[kvshare_layer(int(k), int(a), int(b)) for k, a, b in layer_map])
    wp = None
    keep = None
    if w is not None:
        import numpy as np
        keep = np.ascontiguousarray(np.asarray(w, dtype=np.float32))
        wp = keep.ctypes.data
    st = _lib.kvshare_set_map(h, arr, wp)
    if check:
        _check(st, "kvshare_set_map")
    return st


@dataclass
class Cache:
    """Device tensors of a shared cache (fields as in kvshare_cache)."""
    batch: int
    context: int
    k: object = None
    v: object = None
    slots: int = 0
    coef_k: object = None
    coef_v: object = None
    basis_k: object = None
    basis_v: object = None
    u_k: object = None
    u_v: object = None
    s_k: object = None
    s_v: object = None
    r_k: object = None
    r_v: object = None
    rank: object = None
    pairs: int = 0
    lengths: object = None      # [batch] int32 device tensor of per-sequence token counts

    def as_c(self) -> kvshare_cache:
        p = lambda t: _ptr(t) or None  # noqa: E731
        return kvshare_cache(p(self.k), p(self.v), self.slots, p(self.coef_k), p(self.coef_v), p(self.basis_k),
                             p(self.basis_v), p(self.u_k), p(self.u_v), p(self.s_k), p(self.s_v), p(self.r_k),
                             p(self.r_v), p(self.rank), self.pairs, self.batch, self.context, p(self.lengths))


def kvshare_decode(h, cache: Cache, q, out, lse=None, l0: int = 0, l1: int = None, stream=None,
                   check: bool = True) -> int:
    c = cache.as_c()
    st = _lib.kvshare_decode(h, ctypes.byref(c), _ptr(q), _ptr(out), _ptr(lse), int(l0),
                             int(l1 if l1 is not None else q.shape[0]), _stream(stream))
    if check:
        _check(st, "kvshare_decode")
    return st


def kvshare_decode_stats(h, cache: Cache, q, out, lse, mass=None, score=None, entropy=None, peak=None,
                         l0: int = 0, l1: int = None, stream=None, check: bool = True) -> int:
    c = cache.as_c()
    st = _lib.kvshare_decode_stats(h, ctypes.byref(c), _ptr(q), _ptr(out), _ptr(lse), _ptr(mass), _ptr(score),
                                   _ptr(entropy), _ptr(peak), int(l0), int(l1 if l1 is not None else q.shape[0]),
                                   _stream(stream))
    if check:
        _check(st, "kvshare_decode_stats")
    return st


def kvshare_decode_host(h, cache: Cache, q_host, out_host, lse_host=None, l0: int = 0, l1: int = None,
                        stream=None, check: bool = True) -> int:
    c = cache.as_c()
    st = _lib.kvshare_decode_host(h, ctypes.byref(c), _ptr(q_host), _ptr(out_host), _ptr(lse_host), int(l0),
                                  int(l1 if l1 is not None else q_host.shape[0]), _stream(stream))
    if check:
        _check(st, "kvshare_decode_host")
    return st


def kvshare_prefill(h, cache: Cache, q, out, lse=None, l0: int = 0, l1: int = None, seqlen: int = None,
                    stream=None, check: bool = True) -> int:
    c = cache.as_c()
    st = _lib.kvshare_prefill(h, ctypes.byref(c), _ptr(q), _ptr(out), _ptr(lse), int(l0),
                              int(l1 if l1 is not None else q.shape[0]),
                              int(seqlen if seqlen is not None else q.shape[3]), _stream(stream))
    if check:
        _check(st, "kvshare_prefill")
    return st


def kvshare_pack_residual(h, score, u_k, u_v, rank, u_k8, u_v8, s_k, s_v, batch: int, context: int,
                          stream=None, check: bool = True) -> int:
    st = _lib.kvshare_pack_residual(h, _ptr(score), _ptr(u_k), _ptr(u_v), _ptr(rank), _ptr(u_k8), _ptr(u_v8),
                                    _ptr(s_k), _ptr(s_v), int(batch), int(context), _stream(stream))
    if check:
        _check(st, "kvshare_pack_residual")
    return st


def kvshare_append_lowrank(h, cache: Cache, k_new, v_new, score, pos, stream=None, check: bool = True) -> int:
    c = cache.as_c()
    st = _lib.kvshare_append_lowrank(h, ctypes.byref(c), _ptr(k_new), _ptr(v_new), _ptr(score), _ptr(pos),
                                     _stream(stream))
    if check:
        _check(st, "kvshare_append_lowrank")
    return st


# ---- paged cache. A pool's sizes are not known to the C side, so these entry points check
# their tensors' shapes, types and strides here (EINVAL) before the call; that the memory is
# the context's device's is checked there.
_torch = None   # torch, imported with the first tensor


def _use_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _dense(t, dtype, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _device_stream(stream, device: int) -> Optional[int]:
    """The given stream, or torch's current one on the tensors' own device."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return int(getattr(stream, "cuda_stream", stream))


@dataclass(frozen=True)
class Pages:
    """Device tensors of a paged cache (fields as in kvshare_pages); sizes are the tensors' own.

    k, v [slots][num_pages][Hkv][page_size][d]; block_table [batch][max_blocks] int32;
    lengths [batch] int32; bound_codes [slots][num_pages][Hkv][2][d] int8 and bound_scale
    [slots][num_pages][Hkv] float32 where block selection is used. The tensors' contents may
    change between calls, the tensors may not (make another Pages for others).
    """
    k: object
    v: object
    block_table: object
    lengths: object
    bound_codes: object = None
    bound_scale: object = None

    def __post_init__(self):
        torch = _torch or _use_torch()
        types = {torch.bfloat16: KVS_BF16, torch.float32: KVS_F32}
        k, t = self.k, self.block_table
        ok = k.dtype in types and k.dim() == 5 and t.dim() == 2
        ok = ok and _dense(k, k.dtype, k.shape) and _dense(self.v, k.dtype, k.shape) and \
            _dense(t, torch.int32, t.shape) and _dense(self.lengths, torch.int32, (t.shape[0],))
        if self.bound_codes is not None or self.bound_scale is not None:
            ok = ok and self.bound_codes is not None and self.bound_scale is not None and \
                _dense(self.bound_codes, torch.int8, (*k.shape[:3], 2, k.shape[4])) and \
                _dense(self.bound_scale, torch.float32, k.shape[:3])
        used = [x for x in (k, self.v, t, self.lengths, self.bound_codes, self.bound_scale) if x is not None]
        if not ok or not all(x.is_cuda and x.get_device() == k.get_device() for x in used):
            raise KVShareError(KVS_EINVAL, "Pages")
        c = kvshare_pages(_ptr(k), _ptr(self.v), _ptr(self.bound_codes), _ptr(self.bound_scale), k.shape[0],
                          k.shape[1], k.shape[3], _ptr(t), _ptr(self.lengths), t.shape[0], t.shape[1])
        keep = lambda name, x: object.__setattr__(self, name, x)  # noqa: E731
        keep("_c", c)
        keep("_ref", ctypes.byref(c))
        # what a context must have been created with
        keep("_model", (k.shape[2], k.shape[4], types[k.dtype]))
        keep("_dtype", k.dtype)
        keep("_device", k.get_device())


def _layer_range(pages: Pages, cfg, q, l1):
    """(query shape [L][batch][Hq][d] expected, l1), or None if q does not hold layers up to l1."""
    L = q.shape[0] if q.dim() == 4 else 0
    l1 = L if l1 is None else int(l1)
    shape = (L, pages._c.batch, cfg[0], cfg[1][1])
    return (shape, l1) if 0 <= l1 <= L and _dense(q, pages._dtype, shape) else None


def kvshare_plan_pages(h, lengths, new_tokens, block_table, ring, ring_state, lengths_out, ring_state_out,
                       token_start, slot_map, position, page_size: int, stream=None, check: bool = True) -> int:
    """Sizes are the tensors': batch and max_blocks of block_table, num_pages of ring, max_tokens of slot_map."""
    int32, st = (_torch or _use_torch()).int32, KVS_EINVAL
    if block_table.dim() == 2:
        (B, P), N, M = block_table.shape, ring.numel(), slot_map.numel()
        for t, n in ((lengths, B), (new_tokens, B), (block_table, B * P), (ring, N), (ring_state, 2), (lengths_out, B),
                     (ring_state_out, 2), (token_start, B + 1), (slot_map, M), (position, M)):
            if t.dtype is not int32 or t.numel() != n or not t.is_contiguous():
                break
        else:
            if lengths.is_cuda:
                st = _lib.kvshare_plan_pages(
                    h, lengths.data_ptr(), new_tokens.data_ptr(), block_table.data_ptr(), ring.data_ptr(),
                    ring_state.data_ptr(), lengths_out.data_ptr(), ring_state_out.data_ptr(), token_start.data_ptr(),
                    slot_map.data_ptr(), position.data_ptr(), B, P, page_size, N, M,
                    _device_stream(stream, lengths.get_device()))
    if check and st != KVS_OK:
        raise KVShareError(st, "kvshare_plan_pages")
    return st


def kvshare_append_paged(h, pages: Pages, slot: int, k_new, v_new, slot_map, stream=None, check: bool = True) -> int:
    """k_new, v_new: [tokens][Hkv][d], each token's heads dense; the tokens may be rows of a wider tensor."""
    st, cfg, model = KVS_EINVAL, _config(h), pages._model
    if cfg is not None and cfg[1] == model:
        n, H, d = slot_map.numel(), model[0], model[1]
        dt, shape = pages._dtype, (n, H, d)
        if slot_map.dtype is _torch.int32 and slot_map.is_contiguous() and k_new.dtype is dt and v_new.dtype is dt and \
                k_new.shape == shape and v_new.shape == shape:
            (kr, kh, ke), (vr, vh, ve) = k_new.stride(), v_new.stride()
            if ke == 1 and ve == 1 and (H == 1 or (kh == d and vh == d)):
                if n <= 1:                      # one token's stride says nothing about its row
                    kr = vr = H * d
                st = _lib.kvshare_append_paged(h, pages._ref, slot, k_new.data_ptr(), v_new.data_ptr(), kr, vr,
                                               slot_map.data_ptr(), n, _device_stream(stream, pages._device))
    if check and st != KVS_OK:
        raise KVShareError(st, "kvshare_append_paged")
    return st


def kvshare_decode_paged(h, pages: Pages, q, out, lse=None, l0: int = 0, l1: int = None, selected=None, stream=None,
                         check: bool = True) -> int:
    st, cfg = KVS_EINVAL, _config(h)
    got = _layer_range(pages, cfg, q, l1) if cfg is not None and cfg[1] == pages._model else None
    if got is not None:
        (shape, l1), float32, top, sp = got, _torch.float32, 0, None
        ok = _dense(out, float32, shape) and (lse is None or _dense(lse, float32, shape[:3]))
        if selected is not None:
            # an empty list has no address, which would ask for every block
            top, sp = selected.shape[-1], selected.data_ptr()
            ok = ok and top > 0 and _dense(selected, _torch.int32, (shape[0], shape[1], pages._model[0], top))
        if ok:
            st = _lib.kvshare_decode_paged(h, pages._ref, q.data_ptr(), out.data_ptr(),
                                           None if lse is None else lse.data_ptr(), sp, top, l0, l1,
                                           _device_stream(stream, pages._device))
    if check and st != KVS_OK:
        raise KVShareError(st, "kvshare_decode_paged")
    return st


def kvshare_select_pages(h, pages: Pages, q, selected, first: int = 1, last: int = 1, l0: int = 0, l1: int = None,
                         stream=None, check: bool = True) -> int:
    st, cfg = KVS_EINVAL, _config(h)
    got = _layer_range(pages, cfg, q, l1) if cfg is not None and cfg[1] == pages._model else None
    if got is not None:
        (shape, l1), top = got, selected.shape[-1]
        if _dense(selected, _torch.int32, (shape[0], shape[1], pages._model[0], top)):
            st = _lib.kvshare_select_pages(h, pages._ref, q.data_ptr(), selected.data_ptr(), top, first, last, l0, l1,
                                           _device_stream(stream, pages._device))
    if check and st != KVS_OK:
        raise KVShareError(st, "kvshare_select_pages")
    return st


def kvshare_sync_status(h, stream=None) -> int:
    return _lib.kvshare_sync_status(h, _stream(stream))


def kvshare_set_splits(h, splits: int) -> int:
    return _check(_lib.kvshare_set_splits(h, int(splits)), "kvshare_set_splits")


def kvshare_set_kv_overlap(h, on: bool = True) -> int:
    return _check(_lib.kvshare_set_kv_overlap(h, 1 if on else 0), "kvshare_set_kv_overlap")


def kvshare_set_layer_order(h, order=None, check: bool = True) -> int:
    """order: sequence of num_layers distinct layer indices, or None for model order."""
    keep = None
    if order is not None:
        keep = (ctypes.c_int * len(order))(*[int(x) for x in order])
    st = _lib.kvshare_set_layer_order(h, keep)
    if check:
        _check(st, "kvshare_set_layer_order")
    return st


def kvshare_debug_set_grid(h, ctas: int) -> int:
    return _check(_lib.kvshare_debug_set_grid(h, int(ctas)), "kvshare_debug_set_grid")


def kvshare_debug_stall_next(h, on: bool = True) -> int:
    return _check(_lib.kvshare_debug_stall_next(h, 1 if on else 0), "kvshare_debug_stall_next")


def kvshare_launch_count(h) -> int:
    return int(_lib.kvshare_launch_count(h))


def kvshare_decode_layer_noalloc(q, k, v, w, out, lse, batch: int, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int, context: int, slots: int, src0: int, src1: int = -1,
                                 stream=None, check: bool = True) -> int:
    """One bf16 decode layer whose scratch lives in the library's fixed device array (no allocation)."""
    st = _lib.kvshare_decode_layer_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(out), _ptr(lse), int(batch),
                                           int(num_q_heads), int(num_kv_heads), int(head_dim), int(context),
                                           int(slots), int(src0), int(src1), _stream(stream))
    if check:
        _check(st, "kvshare_decode_layer_noalloc")
    return st

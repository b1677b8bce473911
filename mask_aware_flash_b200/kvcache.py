"""Serving over a paged K/V cache held in 8 bits.

A decode step of one layer is ``fm_cache_append`` (quantises the new tokens' K and V into the cache) and
``fm_cache_attn`` (their attention over it, under the same four mask vectors as the prompt's attention).  With
``accumulate=True`` the cache also keeps the attention weight that every key has received;
``fm_attn_key_weight`` starts it from a prompt, and ``fm_cache_evict`` keeps the heaviest keys of a cache that
has grown over its budget.

    cache = fm_cache_alloc(B, H_kv, D, slots)                  # int8 codes, one scale per 64 tokens and head
    o, lse = fm_attn_fwd(q, k, v, meta, vecs, scale)            # the prompt
    fm_cache_append(cache, k, v, start=zeros)                   # its tokens (clears their weights)
    fm_attn_key_weight(q, k, lse, meta, vecs, scale, weight=cache.weight)
    new_len = fm_cache_evict(cache, smaller, length, budget, recent=128)
    ...
    fm_cache_append(smaller, k1, v1, start=new_len, row=position)   # one token
    o1, lse1 = fm_cache_attn(smaller, q1, new_len + 1, scale, row=position, vecs=vecs, accumulate=True)

As everywhere in the package the caller owns the buffers; work runs on the current stream of the cache's device, or on the
one given.  What a call allocates itself belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import sys

import torch

from . import (FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, AttnArgs, CacheAttnArgs, FmError, KVCacheC,
               MaskMeta, VecArray, _check, _check_tensors, _vecs)
from . import __name__ as _pkg_name

CACHE_PAGE = 64  # slots of a page, and tokens that share a scale
_CODE_TYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_NO_VECS = VecArray(None, None, None, None)
_VEC_NAMES = ("vecs[0]", "vecs[1]", "vecs[2]", "vecs[3]")


def _lib():
    return sys.modules[_pkg_name].lib()


def _call(fn, what, device, stream, *args):
    """Calls `fn` with the stream's handle last: `stream`, or the current stream of the tensors' device, which is made
    the current device for the call (a launch goes to the current device)."""
    if stream is not None and not torch.cuda.is_available():
        return _check(fn(*args, stream.cuda_stream), what)
    index = device.index
    # (the raw handles: a Stream object per call would cost more than the launch it is for)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            code = fn(*args, raw)
    if code:
        _check(code, what)


def _allocating(stream):
    """What a call allocates belongs to the stream it runs on: memory that this stream's allocator hands out has no work of
    another stream pending, and what is dropped (a workspace) is handed out again in this stream's order only."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _expect(what, device, name, t, dtype, shape):
    """One tensor of a call: on `device`, contiguous, of that type and shape (_check_tensors words the error)."""
    if not (t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous()):
        _check_tensors(what, device, [(name, t, dtype, shape)])


class KVCache:
    """The tensors of one layer's cache, checked once and fixed: their addresses are taken here, so an attribute set later
    is refused (make another KVCache for other tensors; what the tensors hold may change at any time).

    k_codes, v_codes: int8 or float8_e4m3fn [n_pages, H_kv, 64, D]; k_scale, v_scale: float32 [n_pages, H_kv];
    page_table: int32 [B, max_pages]; weight: float32, pos: int32, both [B, H_kv, max_pages * 64] or None.
    Slot s of sequence b is slot s % 64 of page page_table[b, s // 64]; a key's value is its code times the scale of
    its (page, head).  pos is the row index of each slot's token (None: the slot itself)."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, page_table, weight=None, pos=None):
        what = "KVCache"
        if k_codes.dim() != 4 or page_table.dim() != 2:
            raise FmError(FM_ERR_INVALID_ARG, f"{what}: k_codes must be [n_pages, H_kv, 64, D], page_table [B, max_pages]")
        if k_codes.dtype not in _CODE_TYPES:
            raise FmError(FM_ERR_UNSUPPORTED, f"{what}: codes must be int8 or float8_e4m3fn, not {k_codes.dtype}")
        n_pages, H_kv, page, D = k_codes.shape
        B, max_pages = page_table.shape
        if page != CACHE_PAGE:
            raise FmError(FM_ERR_INVALID_ARG, f"{what}: a page holds {CACHE_PAGE} slots, not {page}")
        if D not in (64, 128, 256):
            raise FmError(FM_ERR_UNSUPPORTED, f"{what}: D must be 64, 128 or 256, not {D}")
        slots = (B, H_kv, max_pages * CACHE_PAGE)
        _check_tensors(what, k_codes.device,
                       [("k_codes", k_codes, None, None), ("v_codes", v_codes, k_codes.dtype, k_codes.shape),
                        ("k_scale", k_scale, torch.float32, (n_pages, H_kv)),
                        ("v_scale", v_scale, torch.float32, (n_pages, H_kv)),
                        ("page_table", page_table, torch.int32, None), ("weight", weight, torch.float32, slots),
                        ("pos", pos, torch.int32, slots)])
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.page_table, self.weight, self.pos = page_table, weight, pos
        self.B, self.H_kv, self.D, self.n_pages, self.max_pages = B, H_kv, D, n_pages, max_pages
        self.device = k_codes.device
        self.batch = (B,)
        self.c = KVCacheC(B, H_kv, D, n_pages, max_pages, _CODE_TYPES[k_codes.dtype], k_codes.data_ptr(),
                          v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
                          None if weight is None else weight.data_ptr(), None if pos is None else pos.data_ptr())
        self._ref = ctypes.byref(self.c)

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"KVCache: {name} cannot be set: calls use the tensors that the cache was made with")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise AttributeError(f"KVCache: {name} cannot be deleted: calls use the tensors that the cache was made with")

    @property
    def slots(self) -> int:
        """Slots that the page table holds per sequence."""
        return self.max_pages * CACHE_PAGE


def fm_cache_alloc(B, H_kv, D, slots, codes=torch.int8, weight=True, pos=True, device="cuda") -> KVCache:
    """A cache of its own pages for `slots` slots per sequence (rounded up to whole pages), zeroed."""
    max_pages = -(-int(slots) // CACHE_PAGE)
    if max_pages < 1:
        raise FmError(FM_ERR_INVALID_ARG, "fm_cache_alloc: slots must be >= 1")
    pool = (B * max_pages, H_kv, CACHE_PAGE, D)
    table = torch.arange(B * max_pages, dtype=torch.int32, device=device).view(B, max_pages)
    return KVCache(*(torch.zeros(pool, dtype=torch.uint8, device=device).view(codes) for _ in range(2)),
                   *(torch.zeros(pool[:2], dtype=torch.float32, device=device) for _ in range(2)), table,
                   weight=torch.zeros((B, H_kv, max_pages * CACHE_PAGE), device=device) if weight else None,
                   pos=torch.zeros((B, H_kv, max_pages * CACHE_PAGE), dtype=torch.int32, device=device) if pos else None)


def _ptr(t):
    return None if t is None else t.data_ptr()


def fm_cache_append(cache: KVCache, k, v, start, count=None, row=None, stream=None):
    """Writes tokens k, v [B, n_new, H_kv, D] (bf16 or fp32) into the cache: token t < count[b] (None: all) of sequence b
    to slot start[b] + t, with weight 0 and pos row[b] + t (None: the slot).  start, count, row: int32 [B] on the
    device.  Tokens that do not fit the page table are left out."""
    what = "fm_cache_append"
    if k.dim() != 4 or k.dtype not in _DTYPES:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: k must be bfloat16 or float32 [B, n_new, H_kv, D]")
    dev, batch, shape = cache.device, cache.batch, (cache.B, k.shape[1], cache.H_kv, cache.D)
    _expect(what, dev, "k", k, k.dtype, shape)
    _expect(what, dev, "v", v, k.dtype, shape)
    _expect(what, dev, "start", start, torch.int32, batch)
    if count is not None:
        _expect(what, dev, "count", count, torch.int32, batch)
    if row is not None:
        _expect(what, dev, "row", row, torch.int32, batch)
    _call(_lib().fm_cache_append, what, cache.device, stream, cache._ref, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype],
          shape[1], start.data_ptr(), _ptr(count), _ptr(row))


def _attn_args(what, cache, q, cache_len, scale, row, vecs, causal, accumulate):
    if q.dim() != 4 or q.dtype != torch.bfloat16:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: q must be bfloat16 [B, n_q, H, D]")
    Hm = n_k = 0
    vec = _NO_VECS
    if vecs is not None:
        ref = next((x for x in vecs if x is not None), None)
        if ref is not None:
            if ref.dim() != 3:
                raise FmError(FM_ERR_INVALID_ARG, f"{what}: vectors must be [B, Hm, n_k]")
            Hm, n_k = ref.shape[1], ref.shape[2]
            for c in range(4):
                if vecs[c] is not None:
                    _expect(what, cache.device, _VEC_NAMES[c], vecs[c], torch.int32, (cache.B, Hm, n_k))
            vec = _vecs(vecs)
    return CacheAttnArgs(q.shape[2], q.shape[1], 0, scale, q.data_ptr(), _ptr(cache_len), _ptr(row), vec, Hm, n_k,
                         1 if causal else 0, 1 if accumulate else 0)


def fm_cache_attn_workspace_bytes(cache: KVCache, q, accumulate=False) -> int:
    """Bytes of workspace fm_cache_attn needs for queries of q's shape."""
    a = _attn_args("fm_cache_attn", cache, q, None, 1.0, None, None, False, accumulate)
    return int(_lib().fm_cache_attn_workspace_bytes(cache._ref, ctypes.byref(a)))


def fm_cache_attn(cache: KVCache, q, cache_len, scale, row=None, vecs=None, causal=False, accumulate=False, o=None,
                  lse=None, ws=None, stream=None):
    """Attention of q [B, n_q, H, D] (bf16; H % H_kv == 0) over the first cache_len[b] slots -> o (bf16, q's shape),
    lse [B, H, n_q] fp32.

    row: int32 [B], row index of each sequence's first query (needed with vecs or causal).  vecs: the four mask vectors
    int32 [B, Hm, n_k] (None = empty), read at each key's pos; causal also masks a key for the rows before its pos.
    accumulate adds the weight each key receives to cache.weight.  ws: optional uint8 workspace of
    fm_cache_attn_workspace_bytes (allocated here when None); calls that may overlap need one each."""
    what = "fm_cache_attn"
    a = _attn_args(what, cache, q, cache_len, scale, row, vecs, causal, accumulate)
    dev, batch = cache.device, cache.batch
    _, n_q, H, _ = q.shape
    shape, rows = (cache.B, n_q, H, cache.D), (cache.B, H, n_q)
    _expect(what, dev, "q", q, torch.bfloat16, shape)
    _expect(what, dev, "cache_len", cache_len, torch.int32, batch)
    if row is not None:
        _expect(what, dev, "row", row, torch.int32, batch)
    if o is not None:
        _expect(what, dev, "o", o, torch.bfloat16, shape)
    if lse is not None:
        _expect(what, dev, "lse", lse, torch.float32, rows)
    if ws is not None:
        _expect(what, dev, "ws", ws, torch.uint8, ws.shape)
    L, ref = _lib(), ctypes.byref(a)
    if o is None or lse is None or ws is None:
        with _allocating(stream):
            if o is None:
                o = torch.empty_like(q)
            if lse is None:
                lse = torch.empty(rows, dtype=torch.float32, device=dev)
            if ws is None:
                ws = torch.empty(max(int(L.fm_cache_attn_workspace_bytes(cache._ref, ref)), 1), dtype=torch.uint8, device=dev)
    _call(L.fm_cache_attn, what, cache.device, stream, cache._ref, ref, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
          ws.numel())
    return o, lse


def fm_attn_key_weight(q, k, lse, meta: MaskMeta, vecs, scale, weight=None, accumulate=False, stream=None):
    """Attention weight that each prompt key receives: for K/V head hk and key j the sum over the query heads that share
    hk and the rows that see j of exp(scale q.k - lse).  q [B, n_q, H, D], k [B, n_k, H_kv, D] bf16; lse, meta, vecs as
    fm_attn_fwd left or took them.  weight: fp32 [B, H_kv, >= n_k] (a cache's weight; allocated [B, H_kv, n_k] when None),
    written over, or added to with accumulate."""
    what = "fm_attn_key_weight"
    if q.dim() != 4 or k.dim() != 4 or q.dtype is not torch.bfloat16:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: q and k must be bfloat16 [B, n, heads, D]")
    if not q.is_cuda:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: q must be a CUDA tensor")
    dev, q_shape = q.device, q.shape
    B, n_q, H, D = q_shape
    _, n_k, H_kv, _ = k.shape
    _expect(what, dev, "q", q, torch.bfloat16, q_shape)
    _expect(what, dev, "k", k, torch.bfloat16, (B, n_k, H_kv, D))
    _expect(what, dev, "lse", lse, torch.float32, (B, H, n_q))
    if weight is not None:
        if weight.dim() != 3 or weight.shape[2] < n_k:
            raise FmError(FM_ERR_INVALID_ARG, f"{what}: weight must be [B, H_kv, >= n_k]")
        stride = weight.shape[2]
        _expect(what, dev, "weight", weight, torch.float32, (B, H_kv, stride))
    elif accumulate:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: accumulate needs a weight to add to")
    d = meta.desc
    vec_shape, vec = (d.B, d.Hm, d.n_k), VecArray()
    for c, x in enumerate(vecs):
        if x is not None:
            _expect(what, dev, _VEC_NAMES[c], x, torch.int32, vec_shape)
            vec[c] = x.data_ptr()
    if weight is None:
        stride = n_k
        if stream is None:
            weight = torch.empty((B, H_kv, n_k), dtype=torch.float32, device=dev)
        else:
            with _allocating(stream):
                weight = torch.empty((B, H_kv, n_k), dtype=torch.float32, device=dev)
    a = AttnArgs(B, H, n_q, n_k, D, 0, scale, q.data_ptr(), k.data_ptr(), None, H_kv, 0)
    _call(_lib().fm_attn_key_weight, what, dev, stream, ctypes.byref(a), ctypes.byref(meta.c), vec, lse.data_ptr(),
          weight.data_ptr(), stride, 1 if accumulate else 0)
    return weight


def fm_cache_evict_workspace_bytes(src: KVCache, budget: int) -> int:
    """Bytes of workspace fm_cache_evict needs."""
    return int(_lib().fm_cache_evict_workspace_bytes(src._ref, int(budget)))


def fm_cache_evict(src: KVCache, dst: KVCache, cache_len, budget: int, recent: int = 0, new_len=None, ws=None, stream=None):
    """Keeps, for every sequence and K/V head, the last `recent` of its cache_len[b] slots and the budget - recent others
    of largest src.weight (ties: the lowest slot), and writes them in slot order to slots 0, 1, ... of dst.  dst may share
    src's pools under a table of other pages.  Returns int32 [B]: min(cache_len, budget)."""
    what = "fm_cache_evict"
    if src.weight is None:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: src has no weight to go by")
    if (src.B, src.H_kv, src.D, src.k_codes.dtype) != (dst.B, dst.H_kv, dst.D, dst.k_codes.dtype):
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: src and dst must agree in B, H_kv, D and code type")
    dev = src.device
    _expect(what, dev, "cache_len", cache_len, torch.int32, src.batch)
    if new_len is not None:
        _expect(what, dev, "new_len", new_len, torch.int32, src.batch)
    if ws is not None:
        _expect(what, dev, "ws", ws, torch.uint8, ws.shape)
    if dst.device != dev:
        raise FmError(FM_ERR_INVALID_ARG, f"{what}: src and dst must be on one device")
    L = _lib()
    with _allocating(stream):
        if new_len is None:
            new_len = torch.empty_like(cache_len)
        if ws is None:
            n = int(L.fm_cache_evict_workspace_bytes(src._ref, int(budget)))
            ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    _call(L.fm_cache_evict, what, src.device, stream, src._ref, dst._ref, cache_len.data_ptr(), int(budget), int(recent),
          new_len.data_ptr(), ws.data_ptr(), ws.numel())
    return new_len

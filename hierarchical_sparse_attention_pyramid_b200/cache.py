"""torch front end of the paged key/value cache (include/lh.h, lh_cache_write,
lh_cache_read, lh_cache_attn): tokens quantised as they are written, sequences
read back, and the attention of single tokens or trees of drafted tokens over
the cache.  Only marshalling, as dense.py."""

from __future__ import annotations

import ctypes
import math
import operator

import torch

from . import _lib
from ._lib import LhCache, LhCacheAttnConfig
from .dense import (_NAMES, _are_tensors, _call, _contiguous_like, _err, _flat, _is_tensor, _keep, _not_tensors,
                    _plans, _ptr, _sig, _tensor, _writable, _written)

_KINDS = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float8_e4m3fn: "e4m3", torch.int8: "int8"}


class KVCache:
    """The tensors of a paged cache: k, v [pages, heads, page, d] of bf16, fp16, float8_e4m3fn or int8 and, for the
    8-bit types, k_scale, v_scale [pages, heads, page] fp32.  KVCache.empty allocates them.  The tensors of a KVCache
    stay the ones it was made of: the library holds their addresses."""

    def __setattr__(self, name, value):
        raise AttributeError(f"{name}: a KVCache is made anew for other tensors")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _is_tensor("k", k)
        sig = ("cache", _sig(k), _sig(v), _sig(k_scale), _sig(v_scale))
        plan = _plans.get(sig)
        if plan is None:
            plan = _keep(sig, self._check(k, v, k_scale, v_scale))
        pages, heads, page, d, kind = plan
        c = LhCache(pages, page, heads, d, _lib.CACHE_KINDS[kind], k.data_ptr(), v.data_ptr(), _ptr(k_scale),
                    _ptr(v_scale))
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, sig=sig, pages=pages, heads=heads, page=page,
                             d=d, kind=kind, device=k.device, c=c, ref=ctypes.byref(c),
                             tensors=tuple(t for t in (k, v, k_scale, v_scale) if t is not None))

    @staticmethod
    def _check(k, v, k_scale, v_scale):
        _tensor("k", k)
        if k.dim() != 4 or k.dtype not in _KINDS:
            raise ValueError(f"k: shape {tuple(k.shape)} of {k.dtype}, expected [pages, heads, page, d] of bf16, fp16, "
                             "float8_e4m3fn or int8")
        _flat("k", k, k.device, k.dtype, k.shape)
        _flat("v", v, k.device, k.dtype, k.shape)
        if k.element_size() == 1:
            _flat("k_scale", k_scale, k.device, torch.float32, k.shape[:3])
            _flat("v_scale", v_scale, k.device, torch.float32, k.shape[:3])
        elif k_scale is not None or v_scale is not None:
            raise ValueError(f"k_scale, v_scale: a cache of {k.dtype} has none")
        return (*k.shape, _KINDS[k.dtype])

    @staticmethod
    def empty(pages: int, heads: int, page: int, d: int, kind: str = "e4m3", device="cuda") -> "KVCache":
        dtype = {n: t for t, n in _KINDS.items()}[kind]
        kv = [torch.empty((pages, heads, page, d), dtype=dtype, device=device) for _ in range(2)]
        if dtype.itemsize > 1:
            return KVCache(*kv)
        return KVCache(*kv, *(torch.empty((pages, heads, page), dtype=torch.float32, device=device) for _ in range(2)))


def _table(cache: KVCache, page_table):
    _tensor("page_table", page_table, cache.device, torch.int32)
    if page_table.dim() != 2 or not page_table.is_contiguous() or page_table.shape[1] < 1:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)}, expected a contiguous [sequences, pages]")
    return page_table.shape


def cache_write(cache: KVCache, k, v, slots) -> None:
    """Write tokens k, v [n, heads, d] (bf16, fp16 or fp32, channels contiguous) at slots (int64 [n]: page id * page +
    row; negative: skipped), quantised as the cache holds them.  A slot may be given once in a call."""
    try:
        key = ("cache_write", cache.sig, _sig(k), _sig(v), _sig(slots))
    except AttributeError:
        _not_tensors(k=k, v=v, slots=slots)
        raise
    plan = _plans.get(key)
    if plan is None:
        _are_tensors(k=k, v=v, slots=slots)
        _tensor("k", k, cache.device)
        if k.dim() != 3 or tuple(k.shape[1:]) != (cache.heads, cache.d) or k.dtype not in _NAMES:
            raise ValueError(f"k: shape {tuple(k.shape)} of {k.dtype}, expected [n, {cache.heads}, {cache.d}] of bf16, "
                             "fp16 or fp32")
        _tensor("v", v, cache.device, k.dtype, k.shape)
        _flat("slots", slots, cache.device, torch.int64, k.shape[:1])
        if k.numel() and (k.stride(-1) != 1 or v.stride(-1) != 1):
            raise ValueError("k, v: channels must be contiguous")
        i2 = ctypes.c_int64 * 2
        plan = _keep(key, (k.shape[0], _lib.DENSE_DTYPES[_NAMES[k.dtype]], i2(*k.stride()[:2]), i2(*v.stride()[:2])))
    n, dtype, k_stride, v_stride = plan
    if cache.k.requires_grad or cache.v.requires_grad:
        _writable("cache.k", cache.k)
        _writable("cache.v", cache.v)
    if n:
        index = cache.device.index
        _call("lh_cache_write", index, cache.ref, n, dtype, k.data_ptr(), v.data_ptr(), k_stride, v_stride,
              slots.data_ptr(), _err(index))
        _written(cache.tensors)


def cache_read(cache: KVCache, page_table, starts, total: int, dtype=torch.bfloat16, out=None):
    """The first starts[s+1] - starts[s] tokens of every sequence s, by its row of page_table (int32 [sequences,
    pages]), in rows starts[s] .. of (k, v) [total, heads, d].  out: (k, v) to write; rows of no sequence are left as
    they are (uninitialised without out)."""
    total = operator.index(total)
    try:
        key = ("cache_read", cache.sig, _sig(page_table), _sig(starts), total, dtype)
    except AttributeError:
        _not_tensors(page_table=page_table, starts=starts)
        raise
    plan = _plans.get(key)
    if plan is None:
        _are_tensors(page_table=page_table, starts=starts)
        seqs, width = _table(cache, page_table)
        _flat("starts", starts, cache.device, torch.int32, (seqs + 1,))
        if total < 0:
            raise ValueError(f"total: {total}, expected 0 or more")
        if dtype not in _NAMES:
            raise ValueError(f"dtype: {dtype}, expected bf16, fp16 or fp32")
        plan = _keep(key, (seqs, width, _lib.DENSE_DTYPES[_NAMES[dtype]], (total, cache.heads, cache.d),
                           (cache.heads * cache.d, cache.d, 1)))
    seqs, width, code, shape, strides = plan
    if out is None:
        out = (torch.empty_strided(shape, strides, dtype=dtype, device=cache.device),
               torch.empty_strided(shape, strides, dtype=dtype, device=cache.device))
    else:
        for name, t in zip(("out[0]", "out[1]"), out):
            _flat(name, t, cache.device, dtype, shape)
            _writable(name, t)
        _written(out)
    if total:
        index = cache.device.index
        _call("lh_cache_read", index, cache.ref, seqs, width, page_table.data_ptr(), starts.data_ptr(), total, code,
              out[0].data_ptr(), out[1].data_ptr(), _err(index))
    return out


def cache_attention(cache: KVCache, q, page_table, lens, q_start=None, max_tokens: int = 1, tree_mask=None,
                    scale: float | None = None, softcap: float = 0.0, slopes=None, out=None):
    """Attention of the newest tokens q [n, Hq, d] (bf16 or fp16) of every sequence over its cache -> [n, Hq, d].

    lens: int32 [sequences], cached tokens, the query tokens among them (the last ones).  q_start: int32
    [sequences + 1], first query token of each sequence, at most max_tokens each; None: one each.  A token sees the
    positions up to its own; with tree_mask (int64 [n]) all positions before the sequence's query tokens, and query
    token u of its sequence where bit u is set.  scale, softcap, slopes: as dense_forward."""
    scale, softcap, max_tokens = None if scale is None else float(scale), float(softcap), operator.index(max_tokens)
    try:
        key = ("cache_attention", cache.sig, _sig(q), _sig(page_table), _sig(lens), _sig(q_start), max_tokens,
               _sig(tree_mask), scale, softcap, _sig(slopes))
    except AttributeError:
        _not_tensors(q=q, page_table=page_table, lens=lens, q_start=q_start, tree_mask=tree_mask, slopes=slopes)
        raise
    plan = _plans.get(key)
    fresh = plan is None
    if fresh:
        _are_tensors(q=q, page_table=page_table, lens=lens)
        cfg = _attention_config(cache, q, page_table, lens, q_start, max_tokens, tree_mask, scale, softcap, slopes)
        plan = cfg, _lib.load().lh_cache_attn_ws_bytes(cache.ref, cfg)
    cfg, need = plan
    if out is None:
        out = _contiguous_like(q)
    else:
        _flat("out", out, q.device, q.dtype, q.shape)
        _writable("out", out)
        _written(out)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    index = cache.device.index
    _call("lh_cache_attn", index, cache.ref, cfg, q.data_ptr(), page_table.data_ptr(), lens.data_ptr(), _ptr(q_start),
          _ptr(tree_mask), _ptr(slopes), out.data_ptr(), _ptr(ws), need, _err(index))
    if fresh:
        _keep(key, plan)  # of a call that it refuses (by a pointer) the library gives no size
    return out


def _attention_config(cache, q, page_table, lens, q_start, max_tokens, tree_mask, scale, softcap, slopes):
    seqs, width = _table(cache, page_table)
    _tensor("q", q, cache.device)
    if (q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16) or q.shape[2] != cache.d
            or not q.shape[1] or q.shape[1] % cache.heads):
        raise ValueError(f"q: shape {tuple(q.shape)} of {q.dtype}, expected [n, a multiple of {cache.heads}, {cache.d}] of "
                         "bf16 or fp16")
    if cache.kind in ("bf16", "fp16") and cache.kind != _NAMES[q.dtype]:
        raise ValueError(f"q: {q.dtype}, expected the cache's {cache.k.dtype}")
    n, Hq, d = q.shape
    if n and (q.stride(-1) != 1 or (n > 1 and q.stride(0) % 8) or (Hq > 1 and q.stride(1) % 8)):
        raise ValueError(f"q: strides {q.stride()}, expected contiguous channels in 16-byte rows")
    _flat("lens", lens, cache.device, torch.int32, (seqs,))
    if q_start is not None:
        _flat("q_start", q_start, cache.device, torch.int32, (seqs + 1,))
    elif n != seqs:
        raise ValueError(f"q: {n} tokens, expected {seqs} without q_start")
    if tree_mask is not None:
        _flat("tree_mask", tree_mask, cache.device, torch.int64, (n,))
    if slopes is not None:
        _flat("slopes", slopes, cache.device, torch.float32, (Hq,))
    return ctypes.byref(LhCacheAttnConfig(seqs, width, Hq, _lib.DENSE_DTYPES[_NAMES[q.dtype]], max_tokens, n,
                                          1.0 / math.sqrt(d) if scale is None else scale, softcap,
                                          (ctypes.c_int64 * 2)(q.stride(0), q.stride(1) if Hq > 1 else d)))

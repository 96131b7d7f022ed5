"""torch front end of the paged key/value cache (include/lh.h, lh_cache_write,
lh_cache_read, lh_cache_attn): tokens quantised as they are written, sequences
read back, and the attention of single tokens or trees of drafted tokens over
the cache.  Only marshalling, as dense.py."""

from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import LhCache, LhCacheAttnConfig
from .dense import _NAMES, _call, _err, _flat, _ptr, _tensor

_KINDS = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float8_e4m3fn: "e4m3", torch.int8: "int8"}


class KVCache:
    """The tensors of a paged cache: k, v [pages, heads, page, d] of bf16, fp16, float8_e4m3fn or int8 and, for the
    8-bit types, k_scale, v_scale [pages, heads, page] fp32.  KVCache.empty allocates them."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
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
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page, self.d = k.shape
        self.kind = _KINDS[k.dtype]
        self.c = LhCache(self.pages, self.page, self.heads, self.d, _lib.CACHE_KINDS[self.kind], k.data_ptr(),
                         v.data_ptr(), *(None if t is None else t.data_ptr() for t in (k_scale, v_scale)))

    @staticmethod
    def empty(pages: int, heads: int, page: int, d: int, kind: str = "e4m3", device="cuda") -> "KVCache":
        dtype = {n: t for t, n in _KINDS.items()}[kind]
        kv = [torch.empty((pages, heads, page, d), dtype=dtype, device=device) for _ in range(2)]
        if dtype.itemsize > 1:
            return KVCache(*kv)
        return KVCache(*kv, *(torch.empty((pages, heads, page), dtype=torch.float32, device=device) for _ in range(2)))

    @property
    def device(self):
        return self.k.device


def _table(cache: KVCache, page_table):
    _tensor("page_table", page_table, cache.device, torch.int32)
    if page_table.dim() != 2 or not page_table.is_contiguous() or page_table.shape[1] < 1:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)}, expected a contiguous [sequences, pages]")
    return page_table.shape


def cache_write(cache: KVCache, k, v, slots) -> None:
    """Write tokens k, v [n, heads, d] (bf16, fp16 or fp32, channels contiguous) at slots (int64 [n]: page id * page +
    row; negative: skipped), quantised as the cache holds them.  A slot may be given once in a call."""
    _tensor("k", k, cache.device)
    if k.dim() != 3 or tuple(k.shape[1:]) != (cache.heads, cache.d) or k.dtype not in _NAMES:
        raise ValueError(f"k: shape {tuple(k.shape)} of {k.dtype}, expected [n, {cache.heads}, {cache.d}] of bf16, fp16 "
                         "or fp32")
    _tensor("v", v, cache.device, k.dtype, k.shape)
    _flat("slots", slots, cache.device, torch.int64, k.shape[:1])
    if k.numel() == 0:
        return
    if k.stride(-1) != 1 or v.stride(-1) != 1:
        raise ValueError("k, v: channels must be contiguous")
    i2 = ctypes.c_int64 * 2
    _call("lh_cache_write", cache.device, ctypes.byref(cache.c), k.shape[0], _lib.DENSE_DTYPES[_NAMES[k.dtype]],
          _ptr(k), _ptr(v), i2(*k.stride()[:2]), i2(*v.stride()[:2]), _ptr(slots), _err(cache.device))


def cache_read(cache: KVCache, page_table, starts, total: int, dtype=torch.bfloat16, out=None):
    """The first starts[s+1] - starts[s] tokens of every sequence s, by its row of page_table (int32 [sequences,
    pages]), in rows starts[s] .. of (k, v) [total, heads, d].  out: (k, v) to write; rows of no sequence are left as
    they are (uninitialised without out)."""
    seqs, width = _table(cache, page_table)
    _flat("starts", starts, cache.device, torch.int32, (seqs + 1,))
    if dtype not in _NAMES:
        raise ValueError(f"dtype: {dtype}, expected bf16, fp16 or fp32")
    shape = (total, cache.heads, cache.d)
    if out is None:
        out = tuple(torch.empty(shape, dtype=dtype, device=cache.device) for _ in range(2))
    else:
        for name, t in zip(("out[0]", "out[1]"), out):
            _flat(name, t, cache.device, dtype, shape)
    if total:
        _call("lh_cache_read", cache.device, ctypes.byref(cache.c), seqs, width, _ptr(page_table), _ptr(starts), total,
              _lib.DENSE_DTYPES[_NAMES[dtype]], _ptr(out[0]), _ptr(out[1]), _err(cache.device))
    return out


def cache_attention(cache: KVCache, q, page_table, lens, q_start=None, max_tokens: int = 1, tree_mask=None,
                    scale: float | None = None, softcap: float = 0.0, slopes=None, out=None):
    """Attention of the newest tokens q [n, Hq, d] (bf16 or fp16) of every sequence over its cache -> [n, Hq, d].

    lens: int32 [sequences], cached tokens, the query tokens among them (the last ones).  q_start: int32
    [sequences + 1], first query token of each sequence, at most max_tokens each; None: one each.  A token sees the
    positions up to its own; with tree_mask (int64 [n]) all positions before the sequence's query tokens, and query
    token u of its sequence where bit u is set.  scale, softcap, slopes: as dense_forward."""
    seqs, width = _table(cache, page_table)
    _tensor("q", q, cache.device)
    if (q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16) or q.shape[2] != cache.d
            or not q.shape[1] or q.shape[1] % cache.heads):
        raise ValueError(f"q: shape {tuple(q.shape)} of {q.dtype}, expected [n, a multiple of {cache.heads}, {cache.d}] of "
                         "bf16 or fp16")
    if cache.kind in ("bf16", "fp16") and cache.kind != _NAMES[q.dtype]:
        raise ValueError(f"q: {q.dtype}, expected the cache's {cache.k.dtype}")
    n, Hq, d = q.shape
    if n and (q.stride(-1) != 1 or q.data_ptr() % 16 or (n > 1 and q.stride(0) % 8) or (Hq > 1 and q.stride(1) % 8)):
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
    if out is None:
        out = torch.empty((n, Hq, d), dtype=q.dtype, device=q.device)
    else:
        _flat("out", out, q.device, q.dtype, q.shape)
    cfg = LhCacheAttnConfig(seqs, width, Hq, _lib.DENSE_DTYPES[_NAMES[q.dtype]], max_tokens, n,
                            1.0 / math.sqrt(d) if scale is None else scale, softcap,
                            (ctypes.c_int64 * 2)(q.stride(0), q.stride(1) if Hq > 1 else d))
    need = _lib.load().lh_cache_attn_ws_bytes(ctypes.byref(cache.c), ctypes.byref(cfg))
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _call("lh_cache_attn", q.device, ctypes.byref(cache.c), ctypes.byref(cfg), _ptr(q), _ptr(page_table), _ptr(lens),
          _ptr(q_start), _ptr(tree_mask), _ptr(slopes), _ptr(out), _ptr(ws), need, _err(q.device))
    return out

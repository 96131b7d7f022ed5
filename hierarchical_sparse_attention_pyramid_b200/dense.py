"""torch front end of the dense attention around the layer (include/lh.h,
lh_rotary, lh_mask_spans, lh_dense_fwd, lh_dense_bwd): rotary positions, masks
over packed documents, and the masked attention with its gradient that a model
trained with the Lighthouse layer resumes on.  Only marshalling: outputs are
allocated with torch and every step runs in the library's kernels.

Tensors are [B, H, N, d] with any batch, head and token strides that the
kernels can address (channels contiguous; the attention: multiples of 8
elements), so views of token-major projections need no copy.  The `*_forward`
and `*_backward` calls and `rotary` refuse other tensors; `dense_attention` and
`apply_rotary`, the autograd forms, copy them first.  The others record no
gradient: their results are detached, tensors that they are given to write
must not require one while gradients are recorded, and count as modified in
place.
"""

from __future__ import annotations

import ctypes
import math
import threading
from dataclasses import dataclass
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import LhDenseConfig, LhRotaryConfig

_NAMES = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
_err_words: dict = {}
_err_lock = threading.Lock()

# Host plans of the calls (checked configurations), by the tensors' shapes,
# strides, types and devices and the call's options: a program calls each
# operator with a handful of those, and checking and filling a configuration
# takes longer than the smallest kernels run.
_plans: dict = {}
_PLANS_MOST = 4096


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _keep(key, plan):
    if len(_plans) >= _PLANS_MOST:
        _plans.clear()
    _plans[key] = plan
    return plan


def _err(index: int):
    """Address of a device's error word: the calls below report into it (lh_check_error
    clears it), see check_dense_error.  One a device for good: kernels in flight hold its address."""
    t = _err_words.get(index)
    if t is None:
        with _err_lock, torch.cuda.device(index):
            t = _err_words.get(index)
            if t is None:
                if torch.cuda.is_current_stream_capturing():
                    return None  # the first call on a device is a captured one: not reported
                t = torch.zeros(_lib.ERR_WORD_BYTES, dtype=torch.uint8, device="cuda")
                torch.cuda.current_stream().synchronize()
                t = _err_words[index] = (t.data_ptr(), t)
    return t[0]


def check_dense_error(device=None) -> None:
    """Synchronise the current stream and raise if a dense attention, rotary or
    cache call on this device reported a timeout or a bad index.  No call looks
    by itself, dense_attention and its backward included: an output whose kernel
    gave up a wait is unfinished, and only this tells.  Calls captured into a
    graph report too if an eager one ran on the device before."""
    index = torch.device("cuda" if device is None else device).index
    index = torch.cuda.current_device() if index is None else index
    if index in _err_words:
        _call("lh_check_error", index, _err(index))


def _call(name: str, index: int, *args) -> None:
    """A library call on a device's current stream (also when another device is current)."""
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        _lib.call(name, *args, stream)
    else:
        with torch.cuda.device(index):
            _lib.call(name, *args, stream)


def _writable(name: str, t) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, and none is recorded for what is written into it")


# what a call wrote through pointers counts as modified in place: a graph that saved it says so
_written = torch.autograd.graph.increment_version


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tensor(name: str, t, device=None, dtype=None, shape=None):
    """Host check of an argument before its pointer reaches the library, which cannot see sizes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name}: liblh takes CUDA tensors")
    return t


def _is_tensor(name: str, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")


def _are_tensors(**ts):
    for name, t in ts.items():
        _is_tensor(name, t)


def _not_tensors(**ts):
    """The error for arguments (None: not given) that a call's key could not be made of."""
    _are_tensors(**{name: t for name, t in ts.items() if t is not None})


def _flat(name: str, t, device, dtype, shape):
    _tensor(name, t, device, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t


def _addressable(t) -> bool:
    """Rows of 16-byte units: what the attention kernels can load without a copy (the library checks the pointer)."""
    return (t.stride(-1) == 1
            and all(n == 1 or (s > 0 and s % 8 == 0) for n, s in zip(t.shape[:3], t.stride()[:3])))


def _strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


# ------------------------------------------------------------------ rotary positions

def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original: int = 8192, fast_turns: float = 32.0, slow_turns: float = 1.0, device="cuda"):
    """-> (frequencies [rot/2] float64, amplitude): radians a position of each rotated pair, base^(-2i/rot), for a
    context stretched by `factor` over the `original` length with scaling
    - "linear": positions divided by the factor;
    - "ntk": the base raised to base * factor^(rot / (rot - 2)), which stretches the slowest pair by the factor and
      leaves the fastest;
    - "yarn": pairs that make more than fast_turns turns in the original length are left, those that make fewer than
      slow_turns are divided by the factor, with a linear blend between; the amplitude is 0.1 ln(factor) + 1."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot: {rot}, expected an even number of channels")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'ntk' or 'yarn'")
    if not base > 1 or not factor >= 1 or original < 1:
        raise ValueError("expected base > 1, factor >= 1 and original >= 1")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = float(base) ** (-i / max(rot, 1))
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn" and factor > 1:
        at = [rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
              for turns in (fast_turns, slow_turns)]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        amplitude = 0.1 * math.log(factor) + 1.0
    return f.to(device), amplitude


@dataclass(frozen=True)
class Rotary:
    """Rotary positions of a model: what `rotary` takes beside the tensors."""
    frequencies: torch.Tensor  # [rot/2] float64
    layout: str = "half"
    amplitude: float = 1.0

    @staticmethod
    def make(rot: int, base: float = 10000.0, layout: str = "half", device="cuda", **scaling) -> "Rotary":
        frequencies, amplitude = rotary_frequencies(rot, base, device=device, **scaling)
        return Rotary(frequencies, layout, amplitude)


def rotary(q, k, frequencies, positions=None, layout: str = "half", amplitude: float = 1.0, inverse: bool = False,
           out=None):
    """Rotary positions of q [B, Hq, N, d] and k [B, Hk, N, d] (k None: q alone) -> (q', k').

    The first 2 * len(frequencies) channels of each head are turned: pairs (i, i + rot/2) with layout "half",
    (2i, 2i + 1) with "interleaved".  positions: int32 [B, N], or None for 0 .. N-1.  inverse turns back: the
    gradient of a call is the inverse call on the output's gradient.  out: (q', k') to write, which may be (q, k) and
    overlap them and each other in no other way."""
    ts = (q,) if k is None else (q, k)
    amplitude, inverse = float(amplitude), bool(inverse)
    try:
        outs = [torch.empty_like(t) for t in ts] if out is None else list(out)[:len(ts)]
        key = ("rotary", _sig(q), _sig(k), _sig(frequencies), _sig(positions), layout, amplitude, inverse,
               None if out is None else tuple(_sig(o) for o in outs))
    except (AttributeError, TypeError):
        _are_tensors(q=q, frequencies=frequencies)
        _not_tensors(k=k, positions=positions)
        raise
    if len(outs) < len(ts):
        raise ValueError(f"out: {len(outs)} tensors, expected {len(ts)}")
    if out is not None:
        for i, o in enumerate(outs):
            _writable(f"out[{i}]", o)
            for j, t in enumerate(ts + tuple(outs[:i])):  # the calls' own check: what begins at one place
                if o.data_ptr() == t.data_ptr() and o.numel() and (i != j or not _same_places(o, t)):
                    raise ValueError(f"out[{i}]: overlaps another tensor of the call")
    cfg = _plans.get(key)
    if cfg is None:
        cfg = _keep(key, _rotary_config(q, k, frequencies, positions, layout, amplitude, inverse, ts, outs))
    if q.numel() or (k is not None and k.numel()):
        _call("lh_rotary", q.device.index, cfg, q.data_ptr(), _ptr(k), frequencies.data_ptr(), _ptr(positions),
              outs[0].data_ptr(), outs[1].data_ptr() if k is not None else None)
        if out is not None:
            _written(outs)
    return outs[0], (outs[1] if k is not None else None)


def _same_places(a, b) -> bool:
    """Of two tensors that begin at one place: whether an index is the same place in both."""
    return a.shape == b.shape and all(n == 1 or s == t for n, s, t in zip(a.shape, a.stride(), b.stride()))


def _rotary_config(q, k, frequencies, positions, layout, amplitude, inverse, ts, outs):
    _are_tensors(q=q, frequencies=frequencies)
    _tensor("q", q)
    if q.dim() != 4 or q.dtype not in _NAMES:
        raise ValueError(f"q: shape {tuple(q.shape)} of {q.dtype}, expected [B, H, N, d] of bf16, fp16 or fp32")
    B, Hq, N, d = q.shape
    if k is not None:
        _tensor("k", k, q.device, q.dtype)
        if k.dim() != 4 or (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d):
            raise ValueError(f"k: shape {tuple(k.shape)}, expected ({B}, H, {N}, {d})")
    if layout not in _lib.ROTARY_LAYOUTS:
        raise ValueError(f"layout: {layout!r}, expected 'half' or 'interleaved'")
    _tensor("frequencies", frequencies, q.device, torch.float64)
    if frequencies.dim() != 1 or not frequencies.is_contiguous() or 2 * frequencies.numel() > d:
        raise ValueError(f"frequencies: shape {tuple(frequencies.shape)}, expected at most {d // 2} in one row")
    if positions is not None:
        _flat("positions", positions, q.device, torch.int32, (B, N))
    for name, o, t in zip(("out[0]", "out[1]"), outs, ts):
        _tensor(name, o, q.device, q.dtype, t.shape)
        if any(n > 1 and s == 0 for n, s in zip(o.shape, o.stride())):
            raise ValueError(f"{name}: an expanded tensor cannot be written")
    for name, t in zip(("q", "out[0]", "k", "out[1]"), (t for pair in zip(ts, outs) for t in pair)):
        if d > 1 and t.stride(-1) != 1 and t.numel():
            raise ValueError(f"{name}: channels must be contiguous")
    return ctypes.byref(LhRotaryConfig(B, N, Hq, 0 if k is None else k.shape[1], d, 2 * frequencies.numel(),
                                       _lib.ROTARY_LAYOUTS[layout], _lib.DENSE_DTYPES[_NAMES[q.dtype]], int(inverse),
                                       amplitude, _strides(q), _strides(ts[-1]), _strides(outs[0]),
                                       _strides(outs[-1])))


class _RotaryFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rope, positions):
        ctx.layout, ctx.amplitude = rope.layout, float(rope.amplitude)  # one number for both directions
        ctx.save_for_backward(rope.frequencies, positions)  # changed in place before the backward: refused by torch
        q, k = (t if t is None or t.stride(-1) == 1 else t.contiguous() for t in (q, k))
        out = rotary(q, k, rope.frequencies, positions, rope.layout, ctx.amplitude)
        return out if k is not None else out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        frequencies, positions = ctx.saved_tensors
        dq, dk = (t if t is None or t.stride(-1) == 1 else t.contiguous() for t in (dq, dk))
        gq, gk = rotary(dq, dk, frequencies, positions, ctx.layout, ctx.amplitude, inverse=True)
        return gq, gk, None, None


def apply_rotary(q, k, rope: Rotary, positions=None):
    """`rotary` with its gradient in q and k.  k None: q alone (one tensor is returned)."""
    for name, t in (("frequencies", rope.frequencies), ("amplitude", rope.amplitude)):
        if isinstance(t, torch.Tensor) and t.requires_grad:
            raise ValueError(f"{name}: no gradient is computed for them")
    return _RotaryFn.apply(q, k, rope, positions)


# ------------------------------------------------------------------ masks

class AttentionMask(NamedTuple):
    """A mask of the dense attention over B rows of N tokens; attention_mask makes it, every layer shares it."""
    B: int
    N: int
    spans: torch.Tensor


def attention_mask(docs=None, prefix=None, causal: bool = True) -> AttentionMask:
    """The mask of packed rows.  docs: int32 [B, N], a document being a run of equal ids and a negative id padding
    (None: a row is one document).  prefix: bool or uint8 [B, N]; the prefix tokens that lead a document are seen by
    all of it.  causal: beyond that a token sees its document up to itself; otherwise all of it."""
    some = docs if docs is not None else prefix
    if some is None:
        raise ValueError("attention_mask: docs or prefix needed (a plain causal mask needs none)")
    try:
        key = ("mask", _sig(docs), _sig(prefix))
    except AttributeError:
        _not_tensors(docs=docs, prefix=prefix)
        raise
    nbytes = _plans.get(key)
    if nbytes is None:
        _tensor("docs" if docs is not None else "prefix", some)
        if some.dim() != 2 or some.numel() == 0:
            raise ValueError(f"docs: shape {tuple(some.shape)}, expected a non-empty [B, N]")
        if docs is not None:
            _flat("docs", docs, some.device, torch.int32, some.shape)
        if prefix is not None:
            if prefix.dtype not in (torch.bool, torch.uint8):
                raise ValueError(f"prefix: dtype {prefix.dtype}, expected bool or uint8")
            _flat("prefix", prefix, some.device, prefix.dtype, some.shape)
        nbytes = _keep(key, _lib.load().lh_mask_spans_bytes(*some.shape))
    B, N = some.shape
    spans = torch.empty(nbytes, dtype=torch.uint8, device=some.device)
    _call("lh_mask_spans", some.device.index, B, N, int(bool(causal)), _ptr(docs), _ptr(prefix), spans.data_ptr())
    return AttentionMask(B, N, spans)


# ------------------------------------------------------------------ attention

class AttentionSaved(NamedTuple):
    """What dense_forward leaves for dense_backward beside the output."""
    lse: torch.Tensor           # [B, Hq, N] fp32, log of the row's sum of exponentials
    o_low: torch.Tensor | None  # [B, Hq, N, d] in the inputs' type: what rounding the output took off


def _dense_config(q, k, v, mask, causal, scale, softcap, slopes):
    _tensor("q", q)
    if q.dim() != 4 or q.dtype not in (torch.bfloat16, torch.float16) or q.shape[3] not in (64, 128) or not q.shape[1]:
        raise ValueError(f"q: shape {tuple(q.shape)} of {q.dtype}, expected [B, H, N, 64 or 128] of bf16 or fp16")
    B, Hq, N, d = q.shape
    _tensor("k", k, q.device, q.dtype)
    if k.dim() != 4 or (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d) or not k.shape[1] or Hq % k.shape[1]:
        raise ValueError(f"k: shape {tuple(k.shape)}, expected ({B}, a divisor of {Hq}, {N}, {d})")
    _tensor("v", v, q.device, q.dtype, k.shape)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not _addressable(t):
            raise ValueError(f"{name}: strides {t.stride()}, expected contiguous channels in 16-byte rows")
    if mask is not None:
        if (mask.B, mask.N) != (B, N):
            raise ValueError(f"mask: of {mask.B} x {mask.N} tokens, expected {B} x {N}")
        _flat("mask.spans", mask.spans, q.device, torch.uint8, (_lib.load().lh_mask_spans_bytes(B, N),))
    if slopes is not None:
        _flat("slopes", slopes, q.device, torch.float32, (Hq,))
    return LhDenseConfig(B, N, Hq, k.shape[1], d, _lib.DENSE_DTYPES[_NAMES[q.dtype]], int(bool(causal)),
                         1.0 / math.sqrt(d) if scale is None else scale, softcap, _strides(q), _strides(k),
                         _strides(v))


def dense_forward(q, k, v, mask: AttentionMask | None = None, causal: bool = True, scale: float | None = None,
                  softcap: float = 0.0, slopes=None, for_backward: bool = True):
    """Masked attention of q [B, Hq, N, d] over k, v [B, Hkv, N, d], bf16 or fp16 -> (o as q, AttentionSaved).

    mask: from attention_mask (causal is then the mask's); None: causal or full.  scale: 1/sqrt(d) unless given.
    softcap > 0: scores x become softcap * tanh(x / softcap).  slopes: fp32 [Hq], scores get -slope |i - j|.
    A query without keys gets o = 0, lse = -inf.  for_backward False leaves o_low out: dense_backward then takes its
    row sums from the rounded output, which costs accuracy where few keys carry a row."""
    scale, softcap, causal = None if scale is None else float(scale), float(softcap), bool(causal)
    try:
        key = ("dense_forward", _sig(q), _sig(k), _sig(v), None if mask is None else (mask.B, mask.N, _sig(mask.spans)),
               causal, scale, softcap, _sig(slopes))
    except AttributeError:
        _not_tensors(q=q, k=k, v=v, slopes=slopes)
        raise
    plan = _plans.get(key)
    if plan is None:
        _are_tensors(q=q, k=k, v=v)
        cfg = _dense_config(q, k, v, mask, causal, scale, softcap, slopes)
        make_o = _maker(q)
        cfg.o_stride = _strides(make_o(q))
        B, Hq, N, d = q.shape
        plan = _keep(key, (ctypes.byref(cfg), make_o, (B, Hq, N), (Hq * N, N, 1)))
    cfg, make_o, rows, rows_stride = plan
    o = make_o(q)
    lse = torch.empty_strided(rows, rows_stride, dtype=torch.float32, device=q.device)
    low = _contiguous_like(q) if for_backward else None
    if not rows[0] or not rows[2]:
        return o, AttentionSaved(lse, low)
    index = q.device.index
    _call("lh_dense_fwd", index, cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          None if mask is None else mask.spans.data_ptr(), _ptr(slopes), o.data_ptr(), _ptr(low), lse.data_ptr(),
          _err(index))
    return o, AttentionSaved(lse, low)


def dense_backward(do, q, k, v, o, saved: AttentionSaved, mask: AttentionMask | None = None, causal: bool = True,
                   scale: float | None = None, softcap: float = 0.0, slopes=None):
    """Gradients of dense_forward's o with its inputs and both of its results -> (dq, dk, dv)."""
    lse, low = saved
    scale, softcap, causal = None if scale is None else float(scale), float(softcap), bool(causal)
    try:
        key = ("dense_backward", _sig(do), _sig(q), _sig(k), _sig(v), _sig(o), _sig(lse), _sig(low),
               None if mask is None else (mask.B, mask.N, _sig(mask.spans)), causal, scale, softcap, _sig(slopes))
    except AttributeError:
        _not_tensors(do=do, q=q, k=k, v=v, o=o, lse=lse, o_low=low, slopes=slopes)
        raise
    plan = _plans.get(key)
    if plan is None:
        _are_tensors(do=do, q=q, k=k, v=v, o=o, lse=lse)
        cfg = _dense_config(q, k, v, mask, causal, scale, softcap, slopes)
        for name, t in (("do", do), ("o", o)):
            _tensor(name, t, q.device, q.dtype, q.shape)
            if not _addressable(t):
                raise ValueError(f"{name}: strides {t.stride()}, expected contiguous channels in 16-byte rows")
        _flat("lse", lse, q.device, torch.float32, q.shape[:3])
        if low is not None:
            _flat("o_low", low, q.device, q.dtype, q.shape)
        make = [_maker(t) for t in (q, k, v)]
        cfg.o_stride, cfg.do_stride = _strides(o), _strides(do)
        cfg.dq_stride, cfg.dk_stride, cfg.dv_stride = (_strides(m(t)) for m, t in zip(make, (q, k, v)))
        plan = _keep(key, (ctypes.byref(cfg), *make))
    cfg, make_q, make_k, make_v = plan
    dq, dk, dv = make_q(q), make_k(k), make_v(v)
    if lse.numel() == 0:
        return dq, dk, dv
    delta = torch.empty_like(lse)
    index = q.device.index
    _call("lh_dense_bwd", index, cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(low),
          do.data_ptr(), lse.data_ptr(), None if mask is None else mask.spans.data_ptr(), _ptr(slopes), delta.data_ptr(),
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _err(index))
    return dq, dk, dv


def _contiguous_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _maker(t):
    """What allocates an output like t: with its strides where the kernels can write them."""
    return torch.empty_like if _addressable(torch.empty_like(t)) else _contiguous_like


def _usable(t):
    if _addressable(t) and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _DenseAttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, slopes, mask, for_backward, opt):
        q, k, v = _usable(q), _usable(k), _usable(v)
        o, saved = dense_forward(q, k, v, mask, slopes=slopes, for_backward=for_backward, **opt)
        ctx.save_for_backward(q, k, v, o, *saved, slopes, None if mask is None else mask.spans)
        ctx.mask, ctx.opt = mask, opt
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, low, slopes, _ = ctx.saved_tensors
        dq, dk, dv = dense_backward(_usable(do), q, k, v, o, AttentionSaved(lse, low), ctx.mask, slopes=slopes,
                                    **ctx.opt)
        return dq, dk, dv, None, None, None, None


def dense_attention(q, k, v, mask: AttentionMask | None = None, causal: bool = True, scale: float | None = None,
                    softcap: float = 0.0, slopes=None, rotary: Rotary | None = None, positions=None):
    """Masked attention with its gradient in q, k and v (arguments as dense_forward).  rotary: positions are applied
    to q and k first.

    Forward and backward may be captured in a CUDA graph.  While an eager graph of the same leaves is alive, capture
    over other ones (`q.detach().requires_grad_()`): torch makes a leaf's accumulation wait on the stream that it was
    first used on, which a capture does not allow."""
    for name, t in (("slopes", slopes), ("scale", scale), ("softcap", softcap)):
        if isinstance(t, torch.Tensor) and t.requires_grad:
            raise ValueError(f"{name}: no gradient is computed for them")
    # read once for both directions: a tensor may hold another number by the backward
    scale, softcap, causal = None if scale is None else float(scale), float(softcap), bool(causal)
    if rotary is not None:
        q, k = apply_rotary(q, k, rotary, positions)
    elif positions is not None:
        raise ValueError("positions: they need rotary")
    for_backward = torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v))
    return _DenseAttentionFn.apply(q, k, v, slopes, mask, for_backward,
                                   dict(causal=causal, scale=scale, softcap=softcap))

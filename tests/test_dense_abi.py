"""Host checks of the dense attention, rotary and cache calls: every refusal
returns before any CUDA work (no GPU needed)."""

import ctypes
import os

import pytest
import torch

import hierarchical_sparse_attention_pyramid_b200 as lh
from hierarchical_sparse_attention_pyramid_b200 import _lib

FAKE, ODD = 1 << 40, (1 << 40) + 4  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from hierarchical_sparse_attention_pyramid_b200.build import build
        build()
    return _lib.load()


def i3(*x):
    return (ctypes.c_int64 * len(x))(*x)


def rotary_config(**kw):
    c = dict(B=1, N=4, Hq=2, Hk=2, d=64, rot=64, layout=0, dtype=0, inverse=0, amplitude=1.0)
    s = {n: i3(512, 256, 64) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")}
    return _lib.LhRotaryConfig(**{**c, **s, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(Hq=0, Hk=0), 1), (dict(rot=63), 1), (dict(rot=66), 1), (dict(layout=2), 1),
    (dict(dtype=3), 1), (dict(inverse=2), 1), (dict(Hq=70000), 2), (dict(B=1 << 40, N=2), 2),
])
def test_rotary_refusals(lib, kw, status):
    assert lib.lh_rotary(ctypes.byref(rotary_config(**kw)), FAKE, FAKE, FAKE, None, FAKE, FAKE, None) == status
    assert lib.lh_last_error_message()


def test_rotary_pointers_and_empty_calls(lib):
    c = ctypes.byref(rotary_config())
    assert lib.lh_rotary(c, None, FAKE, FAKE, None, FAKE, FAKE, None) == 1
    assert lib.lh_rotary(c, FAKE, FAKE, None, None, FAKE, FAKE, None) == 1
    assert lib.lh_rotary(c, FAKE + 1, FAKE, FAKE, None, FAKE, FAKE, None) == 1
    assert lib.lh_rotary(c, FAKE, FAKE, ODD, None, FAKE, FAKE, None) == 1
    assert lib.lh_rotary(None, FAKE, FAKE, FAKE, None, FAKE, FAKE, None) == 1
    assert lib.lh_rotary(ctypes.byref(rotary_config(N=0)), None, None, None, None, None, None, None) == 0


def dense_config(**kw):
    c = dict(B=2, N=100, Hq=4, Hkv=2, d=64, dtype=0, causal=1, scale=0.125, softcap=0.0)
    s = {f"{n}_stride": i3(25600, 6400, 64) for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    return _lib.LhDenseConfig(**{**c, **s, **kw})


DENSE_BAD = [
    (dict(N=0), 1), (dict(Hq=3), 1), (dict(d=96), 2), (dict(dtype=1), 2), (dict(dtype=9), 1), (dict(causal=2), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("inf")), 1),
    (dict(q_stride=i3(25600, 6400, 60)), 1), (dict(k_stride=i3(25600, 0, 64)), 1), (dict(v_stride=i3(-8, 6400, 64)), 1),
    (dict(o_stride=i3(25600, 6401, 64)), 1), (dict(B=1 << 21), 2), (dict(N=(1 << 30) + 1), 2),
    (dict(B=1 << 16, N=1 << 20), 2),
]


@pytest.mark.parametrize("kw,status", DENSE_BAD)
def test_dense_refusals(lib, kw, status):
    c = ctypes.byref(dense_config(**kw))
    assert lib.lh_dense_fwd(c, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, None, None) == status
    assert lib.lh_dense_bwd(c, *[FAKE] * 4, None, FAKE, FAKE, None, None, *[FAKE] * 4, None, None) == status
    assert lib.lh_last_error_message()


def test_dense_pointers(lib):
    c = ctypes.byref(dense_config())
    args = [FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, None]
    for i in (0, 1, 2, 5, 7):
        for bad in (None, ODD):
            assert lib.lh_dense_fwd(c, *args[:i], bad, *args[i + 1:], None) == 1
    assert lib.lh_dense_fwd(c, *args[:3], ODD, *args[4:], None) == 1  # spans
    assert lib.lh_dense_fwd(c, *args[:6], ODD, *args[7:], None) == 1  # o_low
    back = [FAKE] * 4 + [None] + [FAKE] * 2 + [None, None] + [FAKE] * 4 + [None]
    assert lib.lh_dense_bwd(c, *back[:4], ODD, *back[5:], None) == 1
    for i in (0, 1, 2, 3, 5, 6, 9, 10, 11, 12):
        for bad in (None, ODD):
            assert lib.lh_dense_bwd(c, *back[:i], bad, *back[i + 1:], None) == 1
    for n in ("do", "dq", "dk", "dv"):
        odd = ctypes.byref(dense_config(**{f"{n}_stride": i3(25600, 6400, 63)}))
        assert lib.lh_dense_bwd(odd, *back, None) == 1


def test_mask_refusals(lib):
    assert lib.lh_mask_spans_bytes(0, 5) == 0 and lib.lh_mask_spans_bytes(2, -1) == 0
    # two tables of tiles, two of spans, scratch, a word a row
    assert lib.lh_mask_spans_bytes(2, 129) == 2 * 2 * 2 * 16 + 2 * 129 * 20 + 2 * 4
    for args in ((0, 5, 1, None, None, FAKE), (1, 0, 1, None, None, FAKE), (1, 5, 2, None, None, FAKE),
                 (1, 5, 1, None, None, None), (1, 5, 1, None, None, ODD), (1, 5, 1, FAKE + 2, None, FAKE)):
        assert lib.lh_mask_spans(*args, None) == 1
    assert lib.lh_mask_spans(1, (1 << 30) + 1, 1, None, None, FAKE, None) == 2


def cache_of(**kw):
    c = dict(pages=4, page=16, heads=2, d=64, kind=2, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)
    return _lib.LhCache(**{**c, **kw})


def attn_config(**kw):
    c = dict(seqs=3, width=2, Hq=8, dtype=0, max_tokens=1, n_tok=3, scale=0.1, softcap=0.0)
    return _lib.LhCacheAttnConfig(**{**c, "q_stride": i3(512, 64), **kw})


CACHE_BAD = [(dict(pages=0), 1), (dict(d=32), 2), (dict(page=12), 2), (dict(page=4), 2), (dict(page=8192), 2),
             (dict(kind=4), 1), (dict(k=None), 1), (dict(v=ODD), 1), (dict(k_scale=None), 1), (dict(heads=70000), 2),
             (dict(pages=1 << 30), 2)]


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_cache_refusals(lib, kw, status):
    c = ctypes.byref(cache_of(**kw))
    s = i3(128, 64)
    assert lib.lh_cache_write(c, 5, 0, FAKE, FAKE, s, s, FAKE, None, None) == status
    assert lib.lh_cache_read(c, 1, 1, FAKE, FAKE, 5, 0, FAKE, FAKE, None, None) == status
    a = ctypes.byref(attn_config())
    assert lib.lh_cache_attn_ws_bytes(c, a) == 0
    assert lib.lh_cache_attn(c, a, FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE, 1 << 40, None, None) == status
    assert lib.lh_last_error_message()


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), 1), (dict(width=0), 1), (dict(max_tokens=0), 1), (dict(Hq=7), 1), (dict(dtype=1), 2),
    (dict(dtype=5), 1), (dict(scale=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(width=1 << 28), 2),
    (dict(n_tok=1 << 31), 2), (dict(q_stride=i3(500, 64)), 1), (dict(n_tok=4), 1), (dict(max_tokens=2), 1),
])
def test_cache_attention_refusals(lib, kw, status):
    a = ctypes.byref(attn_config(**kw))
    assert lib.lh_cache_attn(ctypes.byref(cache_of()), a, FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE, 1 << 40,
                             None, None) == status


def test_cache_attention_arguments(lib):
    c, a = ctypes.byref(cache_of()), ctypes.byref(attn_config(width=64))
    need = lib.lh_cache_attn_ws_bytes(c, a)
    # 3 sequences x 2 heads x 8 units of 128 keys at most: 48 blocks, two places of 8 rows each
    assert need == 48 * 2 * 8 * (64 * 4 + 8)
    args = [FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE]
    for i in (0, 1, 2, 6, 7):
        assert lib.lh_cache_attn(c, a, *args[:i], None, *args[i + 1:], need, None, None) == 1
    assert lib.lh_cache_attn(c, a, *args, need - 1, None, None) == 3
    # a tree with slopes, or of more than 64 tokens; an unquantised cache of another type
    assert lib.lh_cache_attn(c, a, *args[:3], FAKE, FAKE, FAKE, *args[6:], need, None, None) == 2
    many = ctypes.byref(attn_config(max_tokens=65))
    assert lib.lh_cache_attn(c, many, *args[:3], FAKE, FAKE, None, *args[6:], 1 << 40, None, None) == 2
    half = ctypes.byref(cache_of(kind=1))
    assert lib.lh_cache_attn(half, a, *args, need, None, None) == 2
    # nothing to do
    none = ctypes.byref(attn_config(seqs=0, n_tok=0))
    assert lib.lh_cache_attn(c, none, None, None, None, None, None, None, None, None, 0, None, None) == 0
    s = i3(128, 64)
    assert lib.lh_cache_write(c, 0, 0, None, None, None, None, None, None, None) == 0
    assert lib.lh_cache_write(c, -1, 0, FAKE, FAKE, s, s, FAKE, None, None) == 1
    assert lib.lh_cache_write(c, 5, 7, FAKE, FAKE, s, s, FAKE, None, None) == 1
    assert lib.lh_cache_write(c, 5, 0, FAKE, FAKE, s, s, None, None, None) == 1
    assert lib.lh_cache_write(c, 1 << 31, 0, FAKE, FAKE, s, s, FAKE, None, None) == 2
    assert lib.lh_cache_read(c, 1, 0, FAKE, FAKE, 5, 0, FAKE, FAKE, None, None) == 1
    assert lib.lh_cache_read(c, 1, 1, FAKE, FAKE, 0, 0, None, None, None, None) == 0
    assert lib.lh_cache_read(c, 1, 1, FAKE, FAKE, 5, 0, ODD, FAKE, None, None) == 1


def test_fp16_stays_outside_the_layer(lib):
    cfg = _lib.LhConfig(1, 1, 4096, 64, 3, 2, 256, 0, _lib.DENSE_DTYPES["fp16"], 0, 0)
    info = _lib.LhPlanInfo()
    assert lib.lh_plan(ctypes.byref(cfg), ctypes.byref(info)) == 1


def test_python_front_end_refuses_what_it_cannot_pass():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f, _ = lh.rotary_frequencies(64, device="cpu")
    for call in (lambda: lh.rotary(x, x, f), lambda: lh.dense_forward(x, x, x), lambda: lh.KVCache(x, x),
                 lambda: lh.attention_mask(torch.zeros(1, 4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: lh.rotary([1], x, f), lambda: lh.dense_forward(x, None, x), lambda: lh.KVCache(3, x),
                 lambda: lh.attention_mask([0, 1])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="docs or prefix"):
        lh.attention_mask()
    for kw in (dict(rot=7), dict(rot=8, scaling="cubic"), dict(rot=8, base=0.5), dict(rot=8, factor=0.5)):
        with pytest.raises(ValueError):
            lh.rotary_frequencies(device="cpu", **kw)
    with pytest.raises(ValueError, match="no gradient"):
        lh.dense_attention(x, x, x, slopes=torch.zeros(2, requires_grad=True))


def test_options_that_require_a_gradient_are_refused():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    one = torch.ones((), requires_grad=True)
    f, _ = lh.rotary_frequencies(64, device="cpu")
    for call in (lambda: lh.dense_attention(x, x, x, scale=one), lambda: lh.dense_attention(x, x, x, softcap=one),
                 lambda: lh.apply_rotary(x, x, lh.Rotary(f.clone().requires_grad_())),
                 lambda: lh.apply_rotary(x, x, lh.Rotary(f, amplitude=one))):
        with pytest.raises(ValueError, match="no gradient is computed"):
            call()


def test_positions_without_rotary_are_refused():
    x = torch.zeros(1, 2, 256, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 256, dtype=torch.int32)
    with pytest.raises(ValueError, match="positions: they need rotary"):
        lh.dense_attention(x, x, x, positions=pos)
    with pytest.raises(ValueError, match="positions: they need rotary"):
        lh.lighthouse_attention(x, x, x, 1, 2, 64, positions=pos)

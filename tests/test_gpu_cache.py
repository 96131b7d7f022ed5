"""The paged cache on the GPU: writing (quantised), reading back, and the
attention of single tokens and trees over it, against plain fp64 forms."""

import pytest
import torch

import hierarchical_sparse_attention_pyramid_b200 as lh
from tests import dense_util as du

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp16", "e4m3", "int8"]


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def paging(lens, page, seed=0, spare=2):
    """-> page_table [seqs, width] (unused entries -1), number of pages, slots of all positions in sequence order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at, slots = 0, []
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n].int()
        at += n
        p = torch.arange(lens[s])
        slots.append(table[s].long()[p // page] * page + p % page)
    return table.cuda(), sum(need) + spare, torch.cat(slots).cuda()


def starts_of(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).int().cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,d,page,lens", [(2, 128, 16, (1, 40, 0, 17)), (3, 64, 8, (9, 8, 100)), (1, 128, 256, (300,))])
def test_write_and_read(kind, dtype, heads, d, page, lens):
    table, pages, slots = paging(lens, page)
    cache = lh.KVCache.empty(pages, heads, page, d, kind)
    n = sum(lens)
    k, v = randn((n, heads, d), dtype, 1, 3.0), randn((n, heads, d), dtype, 2, 1e-3)
    k[0, 0] = 0
    lh.cache_write(cache, k, v, slots)
    got = lh.cache_read(cache, table, starts_of(lens), n, dtype=dtype)
    lh.check_dense_error()
    u = du.half_step(dtype)
    for x, y in zip((k, v), got):
        if kind in ("bf16", "fp16"):
            held = x.to(torch.bfloat16 if kind == "bf16" else torch.float16)
            assert torch.equal(y, held.to(dtype))
            continue
        # each held value nearest, but for borders that the fp32 multiplier and scale (2^-22) may cross
        want, step = du.quantise64(x, kind)
        err = (y.double() - want).abs()
        # half a step of the output: relative for its normal numbers, and half of the one step that subnormal ones
        # have (fp16: values of this test around 1e-5 are below its 2^-14, where steps are 2^-24)
        near = u * want.abs() + torch.finfo(dtype).smallest_normal * u + 2.0 ** -21 * want.abs() + 1e-30
        crossed = err > near
        assert (err <= step + near).all()
        assert crossed.float().mean() <= 1e-3
        # and never further from x than half a step of the held type
        assert ((y.double() - x.double()).abs() <= step / 2 * (1 + 2.0 ** -12) + near + 2.0 ** -20 * x.abs().amax(-1, keepdim=True).double()).all()


def test_write_takes_strides_skips_and_keeps_the_rest():
    heads, d, page = 2, 64, 16
    cache = lh.KVCache.empty(4, heads, page, d, "e4m3")
    for t in (cache.k, cache.v):
        t.view(torch.int8).fill_(17)
    cache.k_scale.fill_(2.0)
    cache.v_scale.fill_(3.0)
    qkv = randn((10, 6, d), torch.bfloat16, 1)
    k, v = qkv[:, 2:4], qkv[:, 4:6]
    slots = torch.arange(10, device="cuda") * 5
    slots[3] = -1
    lh.cache_write(cache, k, v, slots)
    want = lh.KVCache.empty(4, heads, page, d, "e4m3")
    for t in (want.k, want.v):
        t.view(torch.int8).fill_(17)
    want.k_scale.fill_(2.0)
    want.v_scale.fill_(3.0)
    live = slots >= 0
    lh.cache_write(want, k[live].contiguous(), v[live].contiguous(), slots[live].contiguous())
    for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (want.k, want.v, want.k_scale, want.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    touched = (cache.k.view(torch.int8) != 17).any(-1).any(1).flatten().nonzero().flatten().tolist()
    assert set(touched) <= set(slots[live].tolist())
    # rows that 16-byte loads cannot take
    odd = torch.empty(10 * heads * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(10, heads, d)
    odd.copy_(k)
    lh.cache_write(want, odd, odd, slots.clamp_min(0) + (slots < 0) * 63)
    lh.cache_write(cache, k, k, slots.clamp_min(0) + (slots < 0) * 63)
    assert torch.equal(cache.k.view(torch.uint8), want.k.view(torch.uint8))
    # nothing to write
    lh.cache_write(cache, k[:0], v[:0], slots[:0])


def test_rows_that_are_not_finite():
    cache = lh.KVCache.empty(1, 1, 8, 64, "int8")
    k = torch.ones(3, 1, 64, device="cuda")
    k[0, 0, 5], k[1, 0, 6] = float("nan"), float("inf")
    k[2] = 1e-42  # subnormal: kept to what fp32 can scale
    table, starts = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    lh.cache_write(cache, k, k, torch.arange(3, device="cuda"))
    got, _ = lh.cache_read(cache, table, starts, 3, dtype=torch.float32)
    assert got[:2].isnan().all() and got[2].isfinite().all() and (got[2] <= 1e-41).all()


def test_read_leaves_other_rows_and_reports_bad_pages():
    lens = (20, 5)
    table, pages, slots = paging(lens, 8)
    cache = lh.KVCache.empty(pages, 1, 8, 64, "bf16")
    x = randn((25, 1, 64), torch.bfloat16, 1)
    lh.cache_write(cache, x, -x, slots)
    out = tuple(torch.full((40, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    starts = torch.tensor([3, 23, 28], dtype=torch.int32, device="cuda")
    lh.cache_read(cache, table, starts, 40, out=out)
    assert torch.equal(out[0][3:28], x) and torch.equal(out[1][3:28], -x)
    assert (out[0][:3] == 7).all() and (out[0][28:] == 7).all()
    lh.check_dense_error()
    bad = table.clone()
    bad[0, 1] = pages
    bad[1, 0] = -5
    lh.cache_read(cache, bad, starts, 40, out=out)
    with pytest.raises(lh._lib.LhError, match="LH_ERR_DEVICE"):
        lh.check_dense_error()
    lh.check_dense_error()
    lh.cache_write(cache, x[:1], x[:1], torch.tensor([pages * 8], device="cuda"))
    with pytest.raises(lh._lib.LhError, match="LH_ERR_DEVICE"):
        lh.check_dense_error()


def filled(kind, lens, heads, d, page, seed=0, v_scale=1.0):
    """A cache with random sequences; what it stands for, per sequence, in fp64."""
    table, pages, slots = paging(lens, page, seed)
    cache = lh.KVCache.empty(pages, heads, page, d, kind)
    cache.k.view(torch.uint8).fill_(0xff)  # NaN (or -1) wherever nothing is written
    cache.v.view(torch.uint8).fill_(0xff)
    if cache.k_scale is not None:
        cache.k_scale.fill_(float("nan"))
        cache.v_scale.fill_(float("nan"))
    n = sum(lens)
    k, v = randn((n, heads, d), torch.float32, seed + 1), randn((n, heads, d), torch.float32, seed + 2, v_scale)
    v *= torch.exp(randn((n, 1, 1), torch.float32, seed + 3))  # rows of different size
    lh.cache_write(cache, k, v, slots)
    ks, vs = (t.double() for t in lh.cache_read(cache, table, starts_of(lens), n, dtype=torch.float32))
    cut = [0] + torch.tensor(lens).cumsum(0).tolist()
    return cache, table, [ks[a:b] for a, b in zip(cut, cut[1:])], [vs[a:b] for a, b in zip(cut, cut[1:])]


ATTN = [
    # kind, dtype, G, heads, d, page, lens, tokens of each sequence, softcap, alibi, tree
    ("bf16", torch.bfloat16, 4, 2, 128, 16, (1, 7, 16, 300), None, 0.0, 0, 0),
    ("fp16", torch.float16, 1, 3, 64, 8, (9, 129, 0), None, 30.0, 1, 0),
    ("e4m3", torch.bfloat16, 8, 1, 128, 64, (1000, 128, 127), None, 50.0, 0, 0),
    ("e4m3", torch.float16, 5, 2, 64, 32, (64, 31, 33), None, 0.0, 1, 0),
    ("int8", torch.bfloat16, 16, 1, 128, 128, (257, 1), None, 0.0, 0, 0),
    ("int8", torch.float16, 2, 2, 64, 16, (513, 40), (3, 0), 20.0, 0, 0),
    ("bf16", torch.bfloat16, 4, 1, 64, 16, (90, 33, 2), (5, 1, 2), 0.0, 1, 0),
    ("e4m3", torch.bfloat16, 4, 2, 128, 16, (200, 24, 70), (24, 24, 10), 0.0, 0, 1),
    ("fp16", torch.float16, 8, 1, 128, 32, (65, 300), (64, 13), 10.0, 0, 1),
    ("int8", torch.bfloat16, 3, 2, 128, 4096, (4200,), (2,), 0.0, 0, 0),
    # 17 to 32 query rows a key head, and more: tiles of 128 on the tensor cores
    ("int8", torch.float16, 1, 2, 64, 8, (700, 18, 40), (18, 17, 0), 0.0, 0, 1),
    ("bf16", torch.bfloat16, 32, 1, 64, 64, (1, 130, 129, 0), None, 15.0, 0, 0),
    ("bf16", torch.bfloat16, 33, 1, 64, 64, (1, 130, 129, 0), None, 15.0, 0, 0),
    ("int8", torch.bfloat16, 48, 1, 128, 16, (700, 129), None, 0.0, 1, 0),
    ("e4m3", torch.float16, 8, 1, 128, 16, (500, 60), (40, 33), 0.0, 1, 0),
    ("fp16", torch.float16, 20, 2, 128, 32, (1000, 3), None, 0.0, 0, 0),
    ("e4m3", torch.bfloat16, 5, 1, 64, 128, (3000, 64, 2), (64, 64, 2), 0.0, 0, 1),
]


def random_tree(tokens, seed):
    g = torch.Generator().manual_seed(seed)
    out = []
    for T in tokens:
        seen = []
        for t in range(T):
            parent = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << t))
        out += [m - (1 << 64) if m >= 1 << 63 else m for m in seen]
    return torch.tensor(out, dtype=torch.int64)


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_cache_attention(case):
    kind, dtype, G, heads, d, page, lens, tokens, cap, alibi, tree = case
    cache, table, ks, vs = filled(kind, lens, heads, d, page)
    T = [1] * len(lens) if tokens is None else list(tokens)
    n, Hq = sum(T), G * heads
    q = randn((n, Hq, d), dtype, 5, 1.5)
    slopes = torch.tensor([2.0 ** -(i % 8 + 1) for i in range(Hq)], device="cuda") if alibi else None
    masks = random_tree(T, 3).cuda() if tree else None
    cut = [0] + torch.tensor(T).cumsum(0).tolist()
    opt = dict(softcap=cap, slopes=slopes, tree_mask=masks)
    if tokens is not None:
        opt |= dict(q_start=torch.tensor(cut, dtype=torch.int32, device="cuda"), max_tokens=max(T))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = lh.cache_attention(cache, q, table, ln, **opt)
    lh.check_dense_error()
    value, bound = du.cache_attention64(q, ks, vs, cut, lens, None if masks is None else
                                        [x & (1 << 64) - 1 for x in masks.tolist()], None, cap, slopes)
    du.check("o", got, (value, bound))
    assert torch.equal(got, lh.cache_attention(cache, q, table, ln, **opt))
    # strided queries, another stream, an output given
    wide = torch.zeros(n, Hq + 2, d, dtype=dtype, device="cuda")
    wide[:, 1:-1] = q
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lh.cache_attention(cache, wide[:, 1:-1], table, ln, out=out, **opt)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, got)


def test_cache_attention_long_and_many():
    """One long sequence over all SMs, and many short ones beside it: parts that end inside others."""
    for lens, G in (((20000,), 4), (tuple([3] * 200 + [9000] + [130] * 60), 4), ((20000, 1), 24), ((20000, 1), 40),
                    (tuple([3] * 200 + [9000] + [130] * 60), 40)):
        cache, table, ks, vs = filled("int8", lens, 2, 64, 64)
        q = randn((len(lens), 2 * G, 64), torch.bfloat16, 5, 1.5)
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = lh.cache_attention(cache, q, table, ln)
        value, bound = du.cache_attention64(q, ks, vs, list(range(len(lens) + 1)), lens)
        du.check("o", got, (value, bound))


@pytest.mark.parametrize("kind,d", [("bf16", 64), ("int8", 128)])
def test_rows_of_a_tile_at_different_pace(kind, d):
    """Tiles of 128 rows whose first 32 rows keep one maximum while the others' grows with every 128 keys, so that the
    first warp of a tile is ahead of the others (which rescale their outputs each time) when the keys end."""
    heads, G, lens = 2, 128, (2048, 250, 384, 1, 129)
    table, pages, slots = paging(lens, 64)
    cache = lh.KVCache.empty(pages, heads, 64, d, kind)
    n = sum(lens)
    k, v = randn((n, heads, d), torch.float32, 1, 0.1), randn((n, heads, d), torch.float32, 2)
    k[:, :, 0] = torch.cat([torch.arange(m) // 128 for m in lens]).cuda()[:, None].float()
    lh.cache_write(cache, k, v, slots)
    ks, vs = (t.double() for t in lh.cache_read(cache, table, starts_of(lens), n, dtype=torch.float32))
    cut = [0] + torch.tensor(lens).cumsum(0).tolist()
    ks, vs = ([t[a:b] for a, b in zip(cut, cut[1:])] for t in (ks, vs))
    q = randn((len(lens), heads * G, d), torch.bfloat16, 5, 0.3)
    q.view(len(lens), heads, G, d)[:, :, :32, 0] = 0
    q.view(len(lens), heads, G, d)[:, :, 32:, 0] = 160.0  # the maximum moves by about 14 (20) with each unit of 128 keys
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = lh.cache_attention(cache, q, table, ln)
    du.check("o", got, du.cache_attention64(q, ks, vs, list(range(len(lens) + 1)), lens))
    for _ in range(50):
        assert torch.equal(got, lh.cache_attention(cache, q, table, ln))
    lh.check_dense_error()


@pytest.mark.parametrize("kind,dtype,G,d,tree", [("e4m3", torch.bfloat16, 40, 64, 0), ("int8", torch.float16, 33, 128, 0),
                                                 ("bf16", torch.bfloat16, 48, 64, 0), ("fp16", torch.float16, 33, 128, 0),
                                                 ("e4m3", torch.bfloat16, 6, 64, 1), ("bf16", torch.bfloat16, 5, 128, 1),
                                                 ("int8", torch.bfloat16, 4, 64, 0)])
def test_empty_sequences_between_others(kind, dtype, G, d, tree):
    """Query tokens of sequences of length 0 (unused places of a batch) get zeros and leave the other sequences alone:
    empty ones first, last, alone and several in a row, in stretches of several sequences and heads a block."""
    some = [0, 0, 130, 1, 0, 257, 0, 0, 0, 64, 300, 0, 129, 128, 0]
    lens = tuple(some[i % len(some)] if i % 7 else 0 for i in range(210)) + (700, 0, 0, 0)
    cache, table, ks, vs = filled(kind, lens, 4, d, 16)
    T = [8] * len(lens) if tree else [1] * len(lens)
    masks = None
    if tree:
        masks = random_tree(T, 3).cuda()
        # a tree has its tokens in the cache: short sequences have as many as they have positions
        T = [8 if n == 0 or n >= 8 else n for n in lens]
        keep = torch.cat([torch.arange(8) < t for t in T])
        masks = masks[keep.cuda()].contiguous()
    n, Hq = sum(T), 4 * G
    q = randn((n, Hq, d), dtype, 5, 1.5)
    cut = [0] + torch.tensor(T).cumsum(0).tolist()
    opt = dict(q_start=torch.tensor(cut, dtype=torch.int32, device="cuda"), max_tokens=max(T), tree_mask=masks)
    got = lh.cache_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), **opt)
    lh.check_dense_error()
    for s, length in enumerate(lens):
        if length == 0:
            assert (got[cut[s]:cut[s + 1]] == 0).all(), s
    value, bound = du.cache_attention64(q, ks, vs, cut, lens, None if masks is None else
                                        [x & (1 << 64) - 1 for x in masks.tolist()])
    du.check("o", got, (value, bound))


@pytest.mark.parametrize("G", [1, 12, 20, 40])
def test_distances_of_positions_past_2_to_the_24(G):
    """A distance bias over 33 million positions (all columns of the table but the last on one page): the weights of the
    newest keys go by their exact distances, which positions in fp32 would not give."""
    d, page, width = 64, 4096, 8194
    n = (width - 2) * page + page + 37  # 2^25 + 4133
    cache = lh.KVCache.empty(3, 1, page, d, "int8")
    k, v = randn((3 * page, 1, d), torch.float32, 1), randn((3 * page, 1, d), torch.float32, 2)
    lh.cache_write(cache, k, v, torch.arange(3 * page, device="cuda"))
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    q = randn((1, G, d), torch.bfloat16, 5)
    slopes = torch.tensor([1.0 + 0.125 * (h % 8) for h in range(G)], device="cuda")
    got = lh.cache_attention(cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), slopes=slopes)
    lh.check_dense_error()
    near = page + 37  # the keys of the last two pages; the others' weights are below e^-4000
    ks, vs = (t.double() for t in lh.cache_read(cache, table[:, -2:].contiguous(), starts_of((near,)), near,
                                                dtype=torch.float32))
    du.check("o", got, du.cache_attention64(q, [ks], [vs], [0, 1], (near,), slopes=slopes))


@pytest.mark.parametrize("kind", ["fp16", "int8"])
@pytest.mark.parametrize("G", [2, 12, 20, 40])
def test_scores_far_below_a_large_cap(kind, G):
    lens = (300, 40)
    cache, table, ks, vs = filled(kind, lens, 1, 64, 16)
    q = randn((2, G, 64), torch.float16, 5, 1.5)
    got = lh.cache_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), softcap=2.0 ** 20)
    du.check("o", got, du.cache_attention64(q, ks, vs, [0, 1, 2], lens, softcap=2.0 ** 20))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [4, 17, 40])
def test_values_near_the_ends_of_fp32(kind, G):
    """Value rows of 1e35 and of 1e-34, sizes that an 8-bit cache can hold in steps of its type."""
    lens = (20, 5)
    for size in (1e35, 1e-34):
        table, pages, slots = paging(lens, 16)
        cache = lh.KVCache.empty(pages, 1, 16, 64, kind)
        k, v = randn((25, 1, 64), torch.float32, 1), randn((25, 1, 64), torch.float32, 2) * size
        lh.cache_write(cache, k, v, slots)
        ks, vs = (t.double() for t in lh.cache_read(cache, table, starts_of(lens), 25, dtype=torch.float32))
        q = randn((2, G, 64), torch.bfloat16, 5)
        got = lh.cache_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        du.check("o", got, du.cache_attention64(q, [ks[:20], ks[20:]], [vs[:20], vs[20:]], [0, 1, 2], lens))


def test_cache_attention_values_of_any_size():
    """Value rows of very different size in one 8-bit cache, and tiny ones: none underflows on the way."""
    lens = (70,)
    for size, G in ((1e-18, 4), (1e12, 4), (1e-18, 17), (1e12, 17), (1e-18, 40), (1e12, 40)):
        cache, table, ks, vs = filled("e4m3", lens, 1, 64, 16, v_scale=size)
        q = randn((1, G, 64), torch.bfloat16, 5)
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        value, bound = du.cache_attention64(q, ks, vs, [0, 1], lens)
        du.check("o", lh.cache_attention(cache, q, table, ln), (value, bound))


@pytest.mark.parametrize("G", [2, 20, 40])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_lengths_and_pages_are_cut_and_reported(kind, G):
    lens = (40, 20)
    cache, table, ks, vs = filled(kind, lens, 1, 64, 8)
    q = randn((2, G, 64), torch.bfloat16, 5)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    good = lh.cache_attention(cache, q, table, ln)
    lh.check_dense_error()
    bad = table.clone()
    bad[0, 2] = 1 << 20  # keys 16-23 of sequence 0 are not seen
    got = lh.cache_attention(cache, q, bad, ln)
    with pytest.raises(lh._lib.LhError, match="LH_ERR_DEVICE"):
        lh.check_dense_error()
    assert torch.equal(got[1], good[1])
    keep = torch.tensor([i for i in range(40) if not 16 <= i < 24], device="cuda")
    # 32 keys at their places: no distance bias, so that only the set matters
    value, bound = du.cache_attention64(q[:1], [ks[0][keep]], [vs[0][keep]], [0, 1], (32,))
    du.check("o", got[:1], (value, bound))
    for wrong in ((1 << 30, 20), (-3, 20)):
        lh.cache_attention(cache, q, table, torch.tensor(wrong, dtype=torch.int32, device="cuda"))
        with pytest.raises(lh._lib.LhError, match="LH_ERR_DEVICE"):
            lh.check_dense_error()
    # more tokens than the call allows
    start = torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda")
    lh.cache_attention(cache, q, table, ln, q_start=start, max_tokens=1)
    with pytest.raises(lh._lib.LhError, match="LH_ERR_DEVICE"):
        lh.check_dense_error()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_then_steps_as_served(kind):
    """The operators as they are used together: a prompt's queries and keys are turned, its keys and values written,
    and the dense attention runs on what the cache stands for; then single tokens are turned, written and attended,
    captured in one graph that is replayed for each step.  Each step's output is the last row of the dense attention
    over all tokens so far."""
    heads, G, d, page, prompt, steps = 2, 4, 128, 16, 45, 6
    total = prompt + steps
    rope = lh.Rotary.make(d, base=5e5)
    table, pages, slots = paging((total,), page)
    cache = lh.KVCache.empty(pages, heads, page, d, kind)
    q = randn((1, total, heads * G, d), torch.bfloat16, 1).transpose(1, 2)
    k, v = (randn((1, total, heads, d), torch.bfloat16, s).transpose(1, 2) for s in (2, 3))
    qr, kr = lh.rotary(q[:, :, :prompt], k[:, :, :prompt], rope.frequencies)
    lh.cache_write(cache, kr[0].transpose(0, 1), v[0, :, :prompt].transpose(0, 1), slots[:prompt].contiguous())
    kc, vc = lh.cache_read(cache, table, starts_of((prompt,)), prompt)
    first = lh.dense_attention(qr, kc.transpose(0, 1)[None], vc.transpose(0, 1)[None])

    at = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ln, slot = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    qs, ks, vs = (torch.zeros(1, h, 1, d, dtype=torch.bfloat16, device="cuda") for h in (heads * G, heads, heads))

    def step():
        a, b = lh.rotary(qs, ks, rope.frequencies, at)
        lh.cache_write(cache, b[0].transpose(0, 1), vs[0].transpose(0, 1), slot)
        return lh.cache_attention(cache, a[0].transpose(0, 1), table, ln)

    def feed(t):
        at.fill_(t)
        ln.fill_(t + 1)
        slot.copy_(slots[t:t + 1])
        for dst, src in ((qs, q), (ks, k), (vs, v)):
            dst.copy_(src[:, :, t:t + 1])

    feed(prompt)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in range(prompt, total):
        feed(t)
        graph.replay()
        kc, vc = lh.cache_read(cache, table, starts_of((t + 1,)), t + 1)
        q_all = lh.rotary(q[:, :, :t + 1], None, rope.frequencies)[0]
        value, bound = du.cache_attention64(q_all[0, :, t][None], [kc.double()], [vc.double()], [0, 1], (t + 1,))
        du.check("step", out, (value, bound))
        dense = lh.dense_attention(q_all, kc.transpose(0, 1)[None], vc.transpose(0, 1)[None])
        du.check("dense", dense[0, :, t][None], (value, bound))
        # earlier rows see the same keys: the prompt's outputs again
        du.check("prompt", dense[:, :, :prompt], (first.double(), 2 * du.half_step(torch.bfloat16) * (1 + first.double().abs())))
    lh.check_dense_error()

"""The dense attention's and the cache's operators as programs call them: inputs
changed between the directions, captured training steps beside eager graphs,
buffers past 32-bit offsets, and many sequences at once."""

import math
import time
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import hierarchical_sparse_attention_pyramid_b200 as lh
from tests import dense_util as du
from tests.test_gpu_cache import filled, paging, randn, starts_of

pytestmark = pytest.mark.gpu


def test_inputs_changed_before_the_backward_are_refused():
    x = [randn((1, 2, 40, 64), torch.bfloat16, s).requires_grad_() for s in (1, 2, 3)]
    rope = lh.Rotary.make(64)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[None].contiguous()
    slopes = torch.tensor([0.5, 0.25], device="cuda")
    for changed in (pos, slopes, rope.frequencies):
        y = lh.dense_attention(*x, slopes=slopes, rotary=rope, positions=pos)
        changed += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_options_of_tensor_type_are_those_of_the_forward():
    """Numbers given as tensors and changed before the backward: the gradient is that of the forward's numbers."""
    def grads(change):
        x = [randn((1, 2, 40, 64), torch.bfloat16, s).requires_grad_() for s in (1, 2, 3)]
        scale, cap, amplitude = torch.tensor(0.125), torch.tensor(5.0), torch.tensor(1.25)
        rope = lh.Rotary(lh.rotary_frequencies(64)[0], amplitude=amplitude)
        y = lh.dense_attention(*x, scale=scale, softcap=cap, rotary=rope)
        if change:
            for t in (scale, cap, amplitude):
                t *= 2
        return torch.autograd.grad(y.float().square().sum(), x)

    assert all(torch.equal(a, b) for a, b in zip(grads(False), grads(True)))


def test_first_calls_of_two_threads_share_the_error_word(monkeypatch):
    monkeypatch.setattr(lh.dense, "_err_words", {})
    zeros = torch.zeros

    def slow(*args, **kw):
        time.sleep(0.3)  # both threads have found no word by now
        return zeros(*args, **kw)

    monkeypatch.setattr(torch, "zeros", slow)
    with ThreadPoolExecutor(2) as pool:
        a, b = pool.map(lh.dense._err, [0, 0])
    assert a == b == lh.dense._err(0)


def test_a_refused_call_leaves_no_plan():
    """A cache at an address that the library refuses, then one of the same shapes that it takes."""
    lens = (300, 40)
    cache, table, ks, vs = filled("bf16", lens, 2, 64, 32)
    q = randn((2, 6, 64), torch.bfloat16, 5)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    odd = torch.zeros(cache.k.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view(cache.k.shape)
    with pytest.raises(lh._lib.LhError, match="16-byte"):
        lh.cache_attention(lh.KVCache(odd, cache.v), q, table, ln)
    got = lh.cache_attention(cache, q, table, ln)
    du.check("o", got, du.cache_attention64(q, ks, vs, [0, 1, 2], lens))


def test_rotary_refuses_outputs_over_other_tensors():
    q, k = randn((1, 2, 6, 64), torch.bfloat16, 1), randn((1, 2, 6, 64), torch.bfloat16, 2)
    f, _ = lh.rotary_frequencies(64)
    want = lh.rotary(q, k, f)
    o = torch.empty_like(q)
    for out in ((k, q), (o, q), (k, o), (o, o), (q, q), (q.view(1, 6, 2, 64).transpose(1, 2), k)):
        with pytest.raises(ValueError, match="overlaps"):
            lh.rotary(q, k, f, out=out)
    with pytest.raises(ValueError, match="overlaps"):
        lh.rotary(q, None, f, out=(q.view(1, 6, 2, 64).transpose(1, 2),))
    lh.rotary(q, k, f, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # in place, by a view whose strides differ only where there is one index
    one = randn((3, 1, 2, 64), torch.bfloat16, 4)
    want = lh.rotary(one.transpose(1, 2), None, f)[0]
    lh.rotary(one.transpose(1, 2), None, f, out=(one.view(3, 2, 1, 64),))
    assert torch.equal(one.transpose(1, 2), want)
    # the same tensor for both, turned into two others
    a, b = lh.rotary(q, q, f)
    assert torch.equal(a, b)


def test_written_tensors_count_as_modified():
    """What the calls that record no gradient write is news to graphs that saved it, and they write no tensor that a
    gradient is recorded for."""
    f, _ = lh.rotary_frequencies(64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ln = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    slots = torch.arange(8, device="cuda")
    cache = lh.KVCache.empty(1, 2, 8, 64, "bf16")
    x = randn((8, 2, 64), torch.bfloat16, 1)
    lh.cache_write(cache, x, x, slots)
    q = randn((1, 2, 64), torch.bfloat16, 2)
    starts = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    calls = [
        ((1, 2, 5, 64), lambda t: lh.rotary(t, None, f, out=(t,))),
        ((1, 2, 5, 64), lambda t: lh.rotary(t.clone(), t, f, out=(torch.empty_like(t), t))),
        ((1, 2, 8, 64), lambda t: lh.cache_write(lh.KVCache(t, torch.zeros_like(t)), x, x, slots)),
        ((1, 2, 8, 64), lambda t: lh.cache_write(lh.KVCache(torch.zeros_like(t), t), x, x, slots)),
        ((8, 2, 64), lambda t: lh.cache_read(cache, table, starts, 8, out=(t, torch.empty_like(t)))),
        ((8, 2, 64), lambda t: lh.cache_read(cache, table, starts, 8, out=(torch.empty_like(t), t))),
        ((1, 2, 64), lambda t: lh.cache_attention(cache, q, table, ln, out=t)),
    ]
    for shape, call in calls:
        leaf = randn(shape, torch.bfloat16, 3).requires_grad_()
        t = leaf * 1
        loss = (t * t).sum()
        with pytest.raises(ValueError, match="requires a gradient"):
            call(t)
        with torch.no_grad():
            call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        with torch.inference_mode():
            call(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    kept = lh.KVCache.empty(1, 2, 8, 64, "int8")
    leaf = torch.ones(1, 2, 8, device="cuda", requires_grad=True)
    loss = (leaf * kept.v_scale).sum()
    lh.cache_write(kept, x, x, slots)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_second_derivatives_are_refused():
    x = [randn((1, 2, 40, 64), torch.bfloat16, s).requires_grad_() for s in (1, 2, 3)]
    for y in (lh.dense_attention(*x), lh.apply_rotary(x[0], None, lh.Rotary.make(64))):
        g, = torch.autograd.grad(y.float().square().sum(), x[0], create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.float().sum().backward()


def test_options_of_tensor_type_are_read_at_each_call():
    q = randn((1, 2, 40, 64), torch.bfloat16, 1)
    scale = torch.tensor(0.125)
    a = lh.dense_forward(q, q, q, scale=scale)[0]
    scale *= 2
    b = lh.dense_forward(q, q, q, scale=scale)[0]
    assert torch.equal(a, lh.dense_forward(q, q, q, scale=0.125)[0])
    assert torch.equal(b, lh.dense_forward(q, q, q, scale=0.25)[0])


def test_a_cache_keeps_its_tensors():
    cache = lh.KVCache.empty(2, 1, 8, 64, "int8")
    with pytest.raises(AttributeError, match="made anew"):
        cache.k = cache.k.clone()
    with pytest.raises(AttributeError, match="made anew"):
        cache.v_scale = None


def test_captured_training_step_beside_an_eager_graph():
    """A step's forward and backward captured over detached leaves while an eager graph of the leaves lives."""
    leaves = [randn((1, h, 150, 64), torch.bfloat16, s).requires_grad_() for h, s in ((4, 1), (2, 2), (2, 3))]
    docs = torch.repeat_interleave(torch.arange(3, dtype=torch.int32), 50)[None].contiguous().cuda()
    rope = lh.Rotary.make(64)

    def step(q, k, v):
        y = lh.dense_attention(q, k, v, lh.attention_mask(docs), softcap=20.0, rotary=rope)
        return (y, *torch.autograd.grad(y.float().square().sum(), (q, k, v)))

    eager = lh.dense_attention(*leaves, rotary=rope)  # alive throughout
    static = [t.detach().clone().requires_grad_() for t in leaves]
    want = [t.detach().clone() for t in step(*(t.detach().clone().requires_grad_() for t in leaves))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static)
    for shift in (0.0, 0.5):
        fresh = [(t.detach() + shift).requires_grad_() for t in leaves]
        want = step(*fresh)
        with torch.no_grad():
            for a, b in zip(static, fresh):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    eager.float().sum().backward()
    assert all(t.grad is not None for t in leaves)


def test_two_streams_at_once():
    """The same calls on two streams with no wait between them: workspaces are a call's own."""
    lens = (900, 300, 5000)
    cache, table, ks, vs = filled("e4m3", lens, 2, 128, 16)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [randn((3, 16, 128), torch.bfloat16, s) for s in (1, 2)]
    want = [lh.cache_attention(cache, q, table, ln) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(lh.cache_attention(cache, qs[i], table, ln))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("G,tokens", [(2, 1), (4, 3), (8, 4), (30, 2)])
def test_many_sequences(G, tokens):
    """Hundreds of sequences of one to a few units of work: every block ends inside some row of some sequence."""
    g = torch.Generator().manual_seed(G)
    lens = tuple(int(x) for x in torch.randint(tokens, 700, (333,), generator=g))
    cache, table, ks, vs = filled("e4m3", lens, 2, 64, 32)
    q = randn((333 * tokens, 2 * G, 64), torch.bfloat16, 5, 1.5)
    cut = torch.arange(334, dtype=torch.int32) * tokens
    got = lh.cache_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q_start=cut.cuda(),
                             max_tokens=tokens)
    du.check("o", got, du.cache_attention64(q, ks, vs, cut.tolist(), lens))
    lh.check_dense_error()


def test_cache_rows_past_32_bit_offsets():
    """A cache of 5 GiB a tensor whose sequence lies in its last pages."""
    pages, heads, page, d = 20480, 4, 512, 128
    cache = lh.KVCache.empty(pages, heads, page, d, "e4m3")
    assert cache.k.numel() > 1 << 32
    n = 700
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    p = torch.arange(n, device="cuda")
    slots = table[0].long()[p // page] * page + p % page
    k, v = randn((n, heads, d), torch.bfloat16, 1), randn((n, heads, d), torch.bfloat16, 2)
    lh.cache_write(cache, k, v, slots)
    kc, vc = lh.cache_read(cache, table, starts_of((n,)), n, dtype=torch.float32)
    for got, want in ((kc, k), (vc, v)):
        value, step = du.quantise64(want, "e4m3")
        assert ((got.double() - want.double()).abs() <= 0.5 * step * (1 + 2.0 ** -18) + 1e-30).all()
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    for G in (1, 4, 40):
        q = randn((1, heads * G, d), torch.bfloat16, 5)
        du.check("o", lh.cache_attention(cache, q, table, ln),
                 du.cache_attention64(q, [kc.double()], [vc.double()], [0, 1], (n,)))
    lh.check_dense_error()


def test_attention_and_rotary_past_32_bit_offsets():
    """Batch rows 2^31 elements apart, as views of one buffer, give what contiguous ones give."""
    B, N, d, far = 2, 130, 64, (1 << 31) + 64
    big = torch.empty(far + (1 << 18), dtype=torch.bfloat16, device="cuda")

    def view(H, at):
        return big.as_strided((B, H, N, d), (far, N * d, d, 1), at)

    views, plain, at = [], [], 0
    for s, H in enumerate((4, 2, 2, 4)):  # q, k, v, do
        views.append(view(H, at))
        plain.append(randn((B, H, N, d), torch.bfloat16, s))
        views[-1].copy_(plain[-1])
        at += H * N * d
    outs = []
    for q, k, v, do in (views, plain):
        o, saved = lh.dense_forward(q, k, v, softcap=20.0)
        outs.append((o, saved.lse, *lh.dense_backward(do, q, k, v, o, saved, softcap=20.0)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    f, _ = lh.rotary_frequencies(d)
    want = lh.rotary(plain[0], plain[1], f)
    lh.rotary(views[0], views[1], f, out=(views[0], views[1]))
    assert torch.equal(views[0], want[0]) and torch.equal(views[1], want[1])


def test_long_documents_of_one_token_and_one_long_one():
    """65 thousand documents of one token see themselves alone: o = v, dq = dk = 0, dv = do; beside one document that
    fills the other batch row."""
    N, d = 65537, 64
    q, k, v, do = (randn((2, 1, N, d), torch.bfloat16, s) for s in (1, 2, 3, 4))
    docs = torch.zeros((2, N), dtype=torch.int32, device="cuda")
    docs[0] = torch.arange(N, device="cuda")
    mask = lh.attention_mask(docs)
    o, saved = lh.dense_forward(q, k, v, mask)
    dq, dk, dv = lh.dense_backward(do, q, k, v, o, saved, mask)
    assert torch.equal(o[0], v[0]) and torch.equal(dv[0], do[0])
    # P (dP - P dP) with P = 2^x off 1 by the fp32 rounding of LSE: nothing that 2^-12 of the sizes would not cover
    size = (do[0].double() * v[0].double()).sum(-1).abs().max().item() * 8 / math.sqrt(d)
    assert dq[0].abs().max() <= 2.0 ** -12 * size and dk[0].abs().max() <= 2.0 ** -12 * size
    rows = torch.tensor([0, 1, 127, 128, 40000, N - 1], device="cuda")
    s = (q[1, 0, rows].double() @ k[1, 0].double().T) / math.sqrt(d)
    s = s.masked_fill(torch.arange(N, device="cuda") > rows[:, None], -math.inf)
    p = torch.softmax(s, -1)
    value, u = p @ v[1, 0].double(), du.half_step(torch.bfloat16)
    du.check("o", o[1, 0, rows], (value, u * value.abs() + (u + du.F) * (p @ v[1, 0].double().abs()) + 1e-30))


def test_no_rows_and_no_tokens():
    """Empty batches and rows pass through every operator, with their gradients."""
    for B, N in ((0, 5), (2, 0)):
        q, k, v = (torch.empty(B, h, N, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True) for h in (4, 2, 2))
        y = lh.dense_attention(q, k, v, rotary=lh.Rotary.make(64))
        y.sum().backward()
        assert y.shape == q.shape and q.grad.shape == q.shape and k.grad.shape == v.grad.shape == k.shape
    cache = lh.KVCache.empty(1, 2, 8, 64, "e4m3")
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, zero = torch.zeros(0, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lh.cache_write(cache, none[:, :2], none[:, :2], torch.empty(0, dtype=torch.int64, device="cuda"))
    assert lh.cache_read(cache, table, zero, 0)[0].shape == (0, 2, 64)
    assert lh.cache_attention(cache, none, table, zero[:0]).shape == none.shape
    assert lh.cache_attention(cache, none, table, zero[:0], q_start=zero).shape == none.shape
    lh.check_dense_error()


def test_front_end_refusals():
    """Shapes, types, strides and devices that the library cannot see are refused before a pointer reaches it."""
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    q, k = t(2, 4, 8, 64), t(2, 2, 8, 64)
    f, _ = lh.rotary_frequencies(64)
    o, saved = lh.dense_forward(q, k, k)
    cache = lh.KVCache.empty(4, 2, 8, 64, "int8")
    plain = lh.KVCache.empty(4, 2, 8, 64, "bf16")
    x, table, ln = t(3, 2, 64), i32(3, 2), i32(3)
    bad = [
        lambda: lh.rotary(q, t(2, 2, 9, 64), f), lambda: lh.rotary(q, k.float(), f), lambda: lh.rotary(q, k, f.float()),
        lambda: lh.rotary(q, k, f, i32(2, 9)), lambda: lh.rotary(q, k, f, i32(2, 8).long()),
        lambda: lh.rotary(q, k, f, layout="pairs"), lambda: lh.rotary(q, k, f, out=(q,)),
        lambda: lh.rotary(q, k, f, out=(q, k[:1].expand(2, 2, 8, 64))), lambda: lh.rotary(q.transpose(2, 3), k, f),
        lambda: lh.rotary(q[..., :32], None, f), lambda: lh.rotary(q, k.cpu(), f),
        lambda: lh.dense_forward(q, k, t(2, 2, 9, 64)), lambda: lh.dense_forward(q, t(2, 3, 8, 64), t(2, 3, 8, 64)),
        lambda: lh.dense_forward(q.float(), k.float(), k.float()), lambda: lh.dense_forward(q, k.half(), k),
        lambda: lh.dense_forward(q[..., :32], k[..., :32], k[..., :32]),
        lambda: lh.dense_forward(q, k, k[:, :, :, :].transpose(2, 3).contiguous().transpose(2, 3)),
        lambda: lh.dense_forward(q, k, k, lh.attention_mask(i32(2, 9))), lambda: lh.dense_forward(q, k, k, slopes=t(4)),
        lambda: lh.dense_forward(q, k, k, slopes=t(3, dtype=torch.float32)),
        lambda: lh.dense_backward(o[:1], q, k, k, o, saved), lambda: lh.dense_backward(o, q, k, k, o.half(), saved),
        lambda: lh.dense_backward(o, q, k, k, o, saved._replace(lse=saved.lse[:, :2])),
        lambda: lh.dense_backward(o, q, k, k, o, saved._replace(o_low=saved.o_low.transpose(1, 2))),
        lambda: lh.dense_backward(o[:, :, :1].expand(2, 4, 8, 64), q, k, k, o, saved),
        lambda: lh.attention_mask(i32(2, 8).long()), lambda: lh.attention_mask(i32(2, 8), t(2, 8)),
        lambda: lh.attention_mask(i32(2, 8), torch.zeros(2, 7, dtype=torch.bool, device="cuda")),
        lambda: lh.attention_mask(i32(2, 8).T), lambda: lh.attention_mask(i32(0, 8)),
        lambda: lh.KVCache(cache.k, cache.v), lambda: lh.KVCache(plain.k, plain.v[:2]),
        lambda: lh.KVCache(plain.k, plain.v, cache.k_scale, cache.v_scale), lambda: lh.KVCache(plain.k[:, :1], plain.v[:, :1]),
        lambda: lh.KVCache(plain.k.float(), plain.v.float()),
        lambda: lh.cache_write(cache, x, x, i32(3)), lambda: lh.cache_write(cache, x, x[:2], i32(3).long()),
        lambda: lh.cache_write(cache, x, x.half(), i32(3).long()), lambda: lh.cache_write(cache, t(3, 3, 64), t(3, 3, 64), i32(3).long()),
        lambda: lh.cache_read(cache, table, ln, 3), lambda: lh.cache_read(cache, table.long(), i32(4), 3),
        lambda: lh.cache_read(cache, table, i32(4), 3, dtype=torch.float64), lambda: lh.cache_read(cache, table, i32(4), -1),
        lambda: lh.cache_read(cache, table, i32(4), 3, out=(x, x[:2])),
        lambda: lh.cache_attention(cache, t(2, 4, 64), table, ln), lambda: lh.cache_attention(cache, t(3, 3, 64), table, ln),
        lambda: lh.cache_attention(plain, t(3, 4, 64).half(), table, ln),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, i32(2)), lambda: lh.cache_attention(cache, t(3, 4, 64), table.T, ln),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, q_start=i32(3)),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, tree_mask=i32(3)),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, out=t(3, 4, 64).half()),
        lambda: lh.cache_attention(cache, t(3, 4, 72)[..., 4:68], table, ln, slopes=t(3, dtype=torch.float32)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {n} was not refused")
    late = [  # what only the library sees
        lambda: lh.dense_forward(q, k, k, scale=-1.0), lambda: lh.dense_forward(q, k, k, softcap=float("nan")),
        lambda: lh.dense_forward(t(2 * 4 * 8 * 64 + 8)[4:-4].view(2, 4, 8, 64), k, k),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, max_tokens=2),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, q_start=i32(4), max_tokens=0),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, q_start=i32(4), max_tokens=65, tree_mask=i32(3).long()),
        lambda: lh.cache_attention(cache, t(3, 4, 64), table, ln, slopes=t(4, dtype=torch.float32), q_start=i32(4),
                                   tree_mask=i32(3).long()),
        lambda: lh.cache_write(lh.KVCache.empty(2, 2, 12, 64, "bf16"), x, x, i32(3).long()),
    ]
    for n, call in enumerate(late):
        with pytest.raises(lh._lib.LhError):
            call()
            raise AssertionError(f"late call {n} was not refused")
    torch.cuda.synchronize()

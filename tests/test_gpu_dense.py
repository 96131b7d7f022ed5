"""Rotary positions, masks and the masked dense attention with its gradient on
the GPU, against plain fp64 forms with bounds that count roundings
(dense_util)."""

import math

import pytest
import torch

import hierarchical_sparse_attention_pyramid_b200 as lh
from tests import dense_util as du

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", [(1, 4, 2, 33, 128, 128), (2, 3, 1, 7, 64, 32), (1, 1, 1, 1, 64, 64),
                                              (2, 2, 2, 5, 80, 26), (1, 2, 1, 300, 128, 0), (3, 1, 0, 9, 64, 2)])
def test_rotary(layout, dtype, B, Hq, Hk, N, d, rot):
    q = randn((B, Hq, N, d), DT[dtype], 1)
    k = randn((B, Hk, N, d), DT[dtype], 2) if Hk else None
    f, amp = lh.rotary_frequencies(rot, 1e5, "yarn", 4.0, original=64) if rot else (torch.zeros(0, dtype=torch.float64,
                                                                                               device="cuda"), 1.0)
    pos = torch.randint(0, 1 << 30, (B, N), dtype=torch.int32, device="cuda")
    pos[0, 0] = 0
    for inverse in (False, True):
        got = lh.rotary(q, k, f, pos, layout=layout, amplitude=amp, inverse=inverse)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            want = du.rotate64(x, pos, f, layout, amp, inverse)
            # a product and a sum in fp32 (2^-22 of both terms), the sine and cosine (2^-22, and the angle reduced in
            # fp64 from up to 2^30 radians: 2^30 * 2^-52 * 4), then one rounding
            size = 2 * amp * x.double().abs().amax(-1, keepdim=True)
            du.check("rotary", y, (want, du.half_step(x.dtype) * want.abs() + (2.0 ** -20 + 2.0 ** -19) * size))
            assert torch.equal(y[..., rot:], x[..., rot:])


def test_rotary_strides_in_place_and_default_positions():
    B, N, d = 2, 37, 128
    qkv = randn((B, N, 3, 4, d), torch.bfloat16, 3)
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1, :2].transpose(1, 2)
    f, _ = lh.rotary_frequencies(d)
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    want = lh.rotary(q.contiguous(), k.contiguous(), f, pos)
    got = lh.rotary(q, k, f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rest = qkv.clone()
    lh.rotary(q, k, f, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, 2], rest[:, :, 2]) and torch.equal(qkv[:, :, 1, 2:], rest[:, :, 1, 2:])
    # an offset that keeps rows from 16-byte accesses takes the narrow form, with the same results
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(B, 4, N, d)
    x = randn((B, 4, N, d), torch.bfloat16, 4)
    odd.copy_(x)
    assert torch.equal(lh.rotary(odd, None, f)[0], lh.rotary(x, None, f)[0])


def test_rotary_gradient_is_the_inverse_turn():
    rope = lh.Rotary.make(32, layout="interleaved", scaling="ntk", factor=8.0)
    q, k = (randn((1, 2, 11, 64), torch.float32, s).requires_grad_() for s in (5, 6))
    gq, gk = (randn((1, 2, 11, 64), torch.float32, s) for s in (7, 8))
    pos = torch.randint(0, 100000, (1, 11), dtype=torch.int32, device="cuda")
    a, b = lh.apply_rotary(q, k, rope, pos)
    ((a * gq).sum() + (b * gk).sum()).backward()
    for x, g in ((q, gq), (k, gk)):
        want = du.rotate64(g, pos, rope.frequencies, "interleaved", rope.amplitude, inverse=True)
        du.check("grad", x.grad, (want, 2.0 ** -18 * g.double().abs().amax(-1, keepdim=True).expand_as(want) + 1e-9))
    one = lh.apply_rotary(q.detach(), None, rope, pos)
    assert torch.equal(one, a.detach())


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 4.0), ("yarn", 4.0)])
def test_rotary_frequencies(scaling, factor):
    f, amp = lh.rotary_frequencies(64, 10000.0, scaling, factor, original=4096)
    base = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    f = f.cpu()
    if scaling == "linear":
        torch.testing.assert_close(f, base / factor)
    elif scaling == "ntk":  # the fastest pair stays, the slowest is stretched by the factor
        assert abs(f[0] - 1) < 1e-12 and abs(f[-1] * factor / base[-1] - 1) < 1e-9
    elif scaling == "yarn":
        assert abs(f[0] - base[0]) < 1e-12 and abs(f[-1] * factor / base[-1] - 1) < 1e-9
        assert (f <= base + 1e-15).all() and amp == 0.1 * math.log(factor) + 1
    else:
        torch.testing.assert_close(f, base)
        assert amp == 1.0


# ------------------------------------------------------------------ masks

def mask_inputs(B, N, seed, pad=0.2):
    g = torch.Generator().manual_seed(seed)
    docs, prefix = torch.zeros(B, N, dtype=torch.int32), torch.zeros(B, N, dtype=torch.bool)
    for b in range(B):
        i, d = 0, 0
        while i < N:
            n = int(torch.randint(1, max(2, N // 2), (1,), generator=g)) if torch.rand(1, generator=g) < 0.7 else 1
            docs[b, i:i + n] = -1 if torch.rand(1, generator=g) < pad else d
            prefix[b, i:i + int(torch.randint(0, n + 1, (1,), generator=g))] = True
            prefix[b, i + n - 1:i + n] = torch.rand(1, generator=g) < 0.5  # after the lead: does not count
            i, d = i + n, d + 1
    return docs, prefix


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("N", [1, 31, 33, 128, 300, 1025])
def test_mask_spans(N, causal):
    docs, prefix = mask_inputs(2, N, N)
    mask = lh.attention_mask(docs.cuda(), prefix.cuda(), causal=causal)
    tiles = -(-N // 128)
    buf = mask.spans.cpu()
    off = 2 * 2 * tiles * 16
    rows = buf[off:off + 2 * N * 8].view(torch.int32).view(2, N, 2)
    cols = buf[off + 2 * N * 8:off + 4 * N * 8].view(torch.int32).view(2, N, 2)
    seen = du.seen_matrix(2, N, docs, prefix, causal)
    j = torch.arange(N)
    assert torch.equal((j >= rows[..., :1]) & (j < rows[..., 1:]), seen)
    assert torch.equal((j >= cols[..., :1]) & (j < cols[..., 1:]), seen.transpose(1, 2))


def test_mask_spans_of_a_long_row():
    # several chunks of 32K tokens, documents across their borders
    N = 70001
    lens = [1, 40000, 3, 20000, N - 60004]
    docs = torch.repeat_interleave(torch.arange(5, dtype=torch.int32), torch.tensor(lens))[None].contiguous()
    prefix = torch.zeros(1, N, dtype=torch.bool)
    prefix[0, 1:39001] = True
    prefix[0, 60004:60010] = True
    mask = lh.attention_mask(docs.cuda(), prefix.cuda())
    off = 2 * -(-N // 128) * 16
    rows = mask.spans.cpu()[off:off + N * 8].view(torch.int32).view(N, 2)
    start = torch.tensor([0, 1, 40001, 40004, 60004])[docs[0].long()]
    end = torch.tensor([0, 39001, 40001, 40004, 60010])[docs[0].long()]
    assert torch.equal(rows[:, 0].long(), start)
    assert torch.equal(rows[:, 1].long(), torch.maximum(torch.arange(1, N + 1), end))


# ------------------------------------------------------------------ attention

CASES = [
    # B, Hq, Hkv, N, d, dtype, docs, prefix, causal, softcap, alibi, token-major
    (1, 1, 1, 1, 64, "bf16", 0, 0, True, 0.0, 0, 0),
    (1, 2, 1, 2, 128, "fp16", 0, 0, True, 0.0, 0, 1),
    (2, 4, 2, 33, 64, "fp16", 1, 0, True, 5.0, 0, 1),
    (1, 2, 2, 127, 128, "bf16", 0, 0, True, 0.0, 1, 0),
    (1, 2, 2, 128, 64, "bf16", 0, 0, False, 0.0, 0, 0),
    (2, 3, 1, 129, 128, "bf16", 1, 1, True, 0.0, 0, 0),
    (1, 8, 1, 257, 64, "fp16", 1, 1, True, 30.0, 1, 1),
    (1, 4, 4, 300, 128, "fp16", 1, 1, False, 2.0, 1, 1),
    (2, 4, 1, 513, 128, "bf16", 1, 0, True, 20.0, 0, 1),
    (1, 16, 2, 700, 64, "bf16", 0, 0, True, 0.0, 0, 0),
    (1, 2, 1, 1100, 128, "bf16", 1, 1, True, 50.0, 1, 0),
]


def dense_inputs(case, seed=0):
    B, Hq, Hkv, N, d, dtype, docs, prefix, causal, cap, alibi, major = case

    def make(h, s, scale):
        x = randn((B, N, h, d), DT[dtype], seed * 10 + s, scale).transpose(1, 2)
        return x if major else x.contiguous()

    q, k, v, do = make(Hq, 1, 2.0), make(Hkv, 2, 1.0), make(Hkv, 3, 1.0), make(Hq, 4, 1.0)
    ids, pre = mask_inputs(B, N, 7 + N)
    ids, pre = (ids.cuda() if docs else None), (pre.cuda() if prefix else None)
    slopes = torch.tensor([2.0 ** -(i + 1) for i in range(Hq)], device="cuda") if alibi else None
    return q, k, v, do, ids, pre, slopes


def run_dense(case, tensors):
    q, k, v, do, ids, pre, slopes = tensors
    causal, cap = case[8], case[9]
    mask = lh.attention_mask(ids, pre, causal=causal) if ids is not None or pre is not None else None
    opt = dict(mask=mask, causal=causal, softcap=cap, slopes=slopes)
    o, saved = lh.dense_forward(q, k, v, **opt)
    grads = lh.dense_backward(do, q, k, v, o, saved, **opt)
    lh.check_dense_error()
    return dict(zip(("o", "lse", "dq", "dk", "dv"), (o, saved.lse, *grads)))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_attention_against_fp64(case):
    t = dense_inputs(case)
    got = run_dense(case, t)
    q, k, v, do, ids, pre, slopes = t
    seen = du.seen_matrix(case[0], case[3], ids, pre, case[8], "cuda")
    ref = du.attention64(q, k, v, do, seen, 1 / math.sqrt(case[4]), case[9], slopes)
    for n in got:
        du.check(n, got[n], ref[n])
    # the same bits again: no order of sums depends on scheduling
    again = run_dense(case, t)
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_padding_holds_anything():
    """NaN and infinities in padding tokens reach no output; empty rows give zeros and LSE = -inf."""
    case = (2, 4, 2, 300, 128, "bf16", 1, 0, True, 10.0, 1, 0)
    for cap, alibi in ((0.0, 0), (10.0, 1)):
        c = case[:9] + (cap, alibi, 0)
        q, k, v, do, _, _, slopes = dense_inputs(c)
        ids = torch.zeros(2, 300, dtype=torch.int32)
        ids[0, :50] = -1   # before the first document
        ids[0, 140:180] = -2  # between documents
        ids[0, 180:] = 3
        ids[1, 1:] = -1    # one token, the rest padding
        clean = [t.clone() for t in (q, k, v, do)]
        pads = (ids < 0).cuda()[:, None, :, None]
        dirty = [torch.where(pads, torch.tensor(x, dtype=t.dtype, device="cuda"), t)
                 for t, x in zip(clean, (float("nan"), float("inf"), float("nan"), float("-inf")))]
        want = run_dense(c, (*clean, ids.cuda(), None, slopes))
        got = run_dense(c, (*dirty, ids.cuda(), None, slopes))
        for n in want:
            assert torch.equal(got[n], want[n]), n
        empty = pads[:, 0, :, 0]
        assert (got["lse"].transpose(1, 2)[empty] == -math.inf).all()
        for n in ("o", "dq", "dk", "dv"):
            assert (got[n].transpose(1, 2)[empty] == 0).all(), n


# More than 148 query tiles (two of them a CTA in the forward) and more than 296 key tiles (no clusters in dK/dV): what
# the cases above stay below.
LARGE = [
    (2, 16, 16, 1300, 64, "fp16", 0, 0, True, 0.0, 0, 1),
    (2, 16, 16, 1299, 128, "bf16", 1, 1, True, 20.0, 1, 0),
    (2, 32, 16, 1281, 64, "bf16", 1, 1, True, 0.0, 0, 1),
    (2, 32, 16, 1340, 128, "fp16", 1, 0, False, 0.0, 1, 0),
    (3, 16, 16, 1290, 64, "bf16", 0, 0, False, 3.0, 0, 0),
    (1, 64, 32, 1270, 128, "bf16", 1, 1, False, 0.0, 0, 1),
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "-".join(map(str, c)))
def test_large_calls_against_fp64(case):
    test_attention_against_fp64(case)


@pytest.mark.parametrize("cap,alibi", [(0.0, 0), (10.0, 1)])
@pytest.mark.parametrize("heads,d", [((16, 16), 64), ((32, 16), 128)])
def test_padding_of_large_calls_holds_anything(heads, d, cap, alibi):
    case = (2, *heads, 1299, d, "bf16", 1, 0, True, cap, alibi, 1)
    q, k, v, do, _, _, slopes = dense_inputs(case)
    ids = torch.zeros(2, 1299, dtype=torch.int32)
    ids[0, :200] = -1   # more than a tile
    ids[0, 350:390] = -2
    ids[0, 390:] = 3
    ids[0, 1250:] = -1
    ids[1, ::7] = -1    # documents of six tokens
    pads = (ids < 0).cuda()[:, None, :, None]
    clean = [torch.where(pads, torch.zeros((), dtype=t.dtype, device="cuda"), t) for t in (q, k, v, do)]
    dirty = [torch.where(pads, torch.tensor(x, dtype=t.dtype, device="cuda"), t)
             for t, x in zip(clean, (float("nan"), float("inf"), float("nan"), float("-inf")))]
    want = run_dense(case, (*clean, ids.cuda(), None, slopes))
    got = run_dense(case, (*dirty, ids.cuda(), None, slopes))
    for n in want:
        assert torch.equal(got[n], want[n]), n
    ref = du.attention64(*clean, du.seen_matrix(2, 1299, ids, None, True, "cuda"), 1 / math.sqrt(d), cap, slopes)
    for n in want:
        du.check(n, got[n], ref[n])


@pytest.mark.parametrize("N", [90, 700])
def test_backward_without_what_rounding_took_off(N):
    """for_backward False: row sums from the rounded output, within the same bounds (they count its rounding)."""
    case = (2, 4, 2, N, 64, "bf16", 1, 1, True, 20.0, 0, 1)
    q, k, v, do, ids, pre, _ = dense_inputs(case)
    opt = dict(mask=lh.attention_mask(ids, pre), softcap=20.0)
    o, saved = lh.dense_forward(q, k, v, for_backward=False, **opt)
    assert saved.o_low is None
    ref = du.attention64(q, k, v, do, du.seen_matrix(2, N, ids, pre, True, "cuda"), 1 / 8.0, 20.0)
    for n, got in zip(("o", "dq", "dk", "dv"), (o, *lh.dense_backward(do, q, k, v, o, saved, **opt))):
        du.check(n, got, ref[n])


def test_gradients_of_a_long_row():
    """Outputs and gradients of 65537 tokens, sampled rows, against 64 bits (the bounds of dense_util, row by row)."""
    N, d = 65537, 64
    q, k, v, do = (randn((1, 1, N, d), torch.bfloat16, s) for s in (1, 2, 3, 4))
    o, saved = lh.dense_forward(q, k, v)
    dq, dk, dv = lh.dense_backward(do, q, k, v, o, saved)
    u, F, scale = du.half_step(torch.bfloat16), du.F, 1 / 8.0
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 40000, 65407, 65408, N - 1], device="cuda")
    q64, k64, v64, do64 = (t[0, 0].double() for t in (q, k, v, do))
    j = torch.arange(N, device="cuda")
    dk64, dv64, bk, bv = (torch.zeros(len(rows), d, dtype=torch.float64, device="cuda") for _ in range(4))
    o64, dq64, bo, bq, lse = {}, {}, {}, {}, {}
    for i0 in range(0, N, 2048):
        i = j[i0:i0 + 2048]
        e = int(i[-1]) + 1
        x = (q64[i] @ k64[:e].T * scale).masked_fill(j[:e] > i[:, None], -math.inf)
        l64 = torch.logsumexp(x, -1)
        p = torch.exp(x - l64[:, None])
        del x
        out, mag = p @ v64[:e], p @ v64[:e].abs()
        b = u * out.abs() + (u + F) * mag
        delta = (do64[i] * out).sum(-1, keepdim=True)
        slack = (do64[i].abs() * b).sum(-1, keepdim=True)
        for n, r in enumerate(rows.tolist()):
            at = r - i0
            if 0 <= at < len(i):
                dp = do64[r] @ v64[:e].T
                ds = p[at] * (dp - delta[at]) * scale
                off = (u + F) * ds.abs() + p[at] * scale * (slack[at] + F * (do64[r].abs() @ v64[:e].abs().T))
                o64[r], lse[r], bo[r] = out[at], l64[at], b[at]
                dq64[r] = ds @ k64[:e]
                bq[r] = u * dq64[r].abs() + off @ k64[:e].abs()
        live = rows < e  # the keys that these queries reach
        cols = rows[live]
        pc = p[:, cols]
        dp = do64[i] @ v64[cols].T
        ds = pc * (dp - delta) * scale
        off = (u + F) * ds.abs() + pc * scale * (slack + F * (do64[i].abs() @ v64[cols].abs().T))
        dk64[live] += ds.T @ q64[i]
        bk[live] += off.T @ q64[i].abs()
        dv64[live] += pc.T @ do64[i]
        bv[live] += (u + F) * (pc.T @ do64[i].abs())
    few = 1 + 2.0 ** -5
    pick = lambda t: torch.stack([t[r] for r in rows.tolist()])  # noqa: E731
    du.check("o", o[0, 0, rows], (pick(o64), pick(bo) * few))
    du.check("lse", saved.lse[0, 0, rows], (pick(lse), 2.0 ** -18 * (1 + pick(lse).abs())))
    du.check("dq", dq[0, 0, rows], (pick(dq64), pick(bq) * few + 1e-30))
    du.check("dk", dk[0, 0, rows], (dk64, (u * dk64.abs() + bk) * few + 1e-30))
    du.check("dv", dv[0, 0, rows], (dv64, (u * dv64.abs() + bv) * few + 1e-30))


def test_scores_of_the_lowest_values():
    """Keys that give scores of -1e30 beside others, and rows whose only keys do."""
    q, k, v = (torch.ones(1, 1, 130, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    k[0, 0, :64] = -3e28
    v[0, 0] = torch.arange(130, device="cuda")[:, None].bfloat16()
    o, (lse, _) = lh.dense_forward(q, k, v)
    i = torch.arange(130, device="cuda").double()
    # rows below 64 see equal scores of -2.4e29 each (exact in fp32: a sum of 64 equal terms), later rows the others
    want = torch.where(i < 64, i / 2, (64 + i) / 2)
    assert ((o[0, 0, :, 0].double() - want).abs() <= 2 * du.half_step(torch.bfloat16) * want + 1e-6).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("heads", [128, 16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_scores_that_are_not_finite(value, heads, cap):
    """A NaN or infinite score at every column of the unmasked and masked key tiles (head h: key 128 / heads * h), in
    calls of one and of two query tiles a CTA: every query that sees a NaN or +inf is NaN, one that sees -inf gives the
    key no weight whatever its value is, the others know nothing of it."""
    N, d = 384, 64
    q, k, v = (randn((1, heads, N, d), torch.bfloat16, s) for s in (1, 2, 3))
    q[..., 0] = 1.0
    for step in range(128 // heads):
        for causal in (True, False):
            j = torch.arange(heads, device="cuda") * (128 // heads) + step
            bad, big = k.clone(), v.clone()
            bad[0, torch.arange(heads), j, 0] = value
            if value < 0 and not cap:
                big[0, torch.arange(heads), j] = 3e38
            o, (lse, _) = lh.dense_forward(q, bad, big, causal=causal, softcap=cap)
            i = torch.arange(N, device="cuda")
            sees = (i >= j[:, None]) if causal else torch.ones(heads, N, dtype=torch.bool, device="cuda")
            x = (q.double() @ k.double().transpose(-1, -2)) / math.sqrt(d)
            if cap:
                x = cap * torch.tanh(x / cap)
            hide = torch.zeros(heads, N, N, dtype=torch.bool, device="cuda")
            if causal:
                hide |= i > i[:, None]
            at = torch.zeros_like(hide)
            at[torch.arange(heads), :, j] = True
            if cap and not math.isnan(value):  # a score of +-cap
                x = torch.where(at, math.copysign(cap, value), x)
                lost = torch.zeros_like(sees)
            elif value < 0:
                hide = hide | at
                lost = torch.zeros_like(sees)
            else:
                lost = sees
            assert o[0][lost].isnan().all() and lse[0][lost].isnan().all()
            x = x[0].masked_fill(hide, -math.inf)
            p = torch.softmax(x, -1)
            none = hide.all(-1)
            p = p.masked_fill(none[..., None], 0.0)
            u = du.half_step(torch.bfloat16)
            want, size = p @ v[0].double(), p @ v[0].double().abs()
            keep = ~lost
            du.check("o", o[0][keep], (want[keep], (u * want.abs() + (u + du.F) * size + 1e-30)[keep]))
            lse64 = torch.logsumexp(x, -1)
            du.check("lse", lse[0][keep], (lse64[keep], (2.0 ** -18 * (1 + lse64.abs().clamp_max(1e6)))[keep]))
            assert (o[0][none] == 0).all()
    # nothing but -inf: no weight anywhere, as for a query without keys
    if value < 0 and not cap:
        bad = k.clone()
        bad[..., 0] = value
        for causal in (True, False):
            o, (lse, _) = lh.dense_forward(q, bad, v, causal=causal)
            assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("N", [100, 300])
def test_scores_far_below_a_large_cap(N):
    """A cap of 2^16 over scores of ordinary size, beside rows whose scores reach it: the small ones keep their own
    digits, not those of the cap."""
    q, k, v, do = (randn((1, 2, N, 64), torch.float16, s, x) for s, x in ((1, 0.4), (2, 4.0), (3, 1.0), (4, 1.0)))
    far = torch.zeros(N, dtype=torch.bool, device="cuda")
    far[5::32] = True  # some in every warp
    q[:, :, far] *= 32768.0
    do[:, :, far] = 0  # no gradient passes through them
    cap = 65536.0
    o, saved = lh.dense_forward(q, k, v, softcap=cap)
    grads = lh.dense_backward(do, q, k, v, o, saved, softcap=cap)
    ref = du.attention64(q, k, v, do, du.seen_matrix(1, N, device="cuda"), 1 / 8.0, cap)
    for n, got in zip(("o", "lse", "dq", "dk", "dv"), (o, saved.lse, *grads)):
        keep = torch.ones_like(far) if n in ("dk", "dv") else ~far
        du.check(n, got[:, :, keep], tuple(t[:, :, keep] for t in ref[n]))


def test_gradient_against_differences():
    """The gradient of a weighted sum of outputs, against central differences of the fp64 form."""
    case = (1, 2, 1, 20, 64, "fp16", 1, 1, True, 8.0, 1, 0)
    q, k, v, do, ids, pre, slopes = dense_inputs(case)
    got = run_dense(case, (q, k, v, do, ids, pre, slopes))
    seen = du.seen_matrix(1, 20, ids, pre, True, "cuda")

    def loss(q, k, v):
        x = q @ k.repeat_interleave(2, 1).transpose(-1, -2) / 8.0
        x = 8.0 * torch.tanh(x / 8.0)
        i = torch.arange(20, device="cuda")
        x = x - slopes.double()[:, None, None] * (i[:, None] - i).abs()
        p = torch.softmax(x.masked_fill(~seen[:, None], -1e300), -1) * seen[:, None]
        return float((p @ v.repeat_interleave(2, 1) * do.double()).sum())

    args = [t.double() for t in (q, k, v)]
    g = torch.Generator().manual_seed(0)
    for which, name in enumerate(("dq", "dk", "dv")):
        for _ in range(8):
            way = torch.randn(args[which].shape, generator=g, dtype=torch.float64).cuda()
            h = 1e-5
            plus, minus = (loss(*[a + (s * h * way if i == which else 0) for i, a in enumerate(args)]) for s in (1, -1))
            slope = (got[name].double() * way).sum().item()
            # every element of the gradient within a few half steps of its own bound
            ref = du.attention64(q, k, v, do, seen, 1 / 8.0, 8.0, slopes)[name]
            assert abs(slope - (plus - minus) / (2 * h)) <= (ref[1] * way.abs()).sum().item() + 1e-6


def test_autograd_broadcast_and_shared_inputs():
    """Expanded keys and values (gradients summed by autograd), the same tensor as key and value, sum().backward()."""
    q = randn((2, 4, 40, 64), torch.bfloat16, 1).requires_grad_()
    kv = randn((1, 1, 40, 64), torch.bfloat16, 2).requires_grad_()
    y = lh.dense_attention(q, kv.expand(2, 4, 40, 64), kv.expand(2, 4, 40, 64))
    y.sum().backward()
    seen = du.seen_matrix(2, 40, device="cuda")
    ke = kv.detach().expand(2, 4, 40, 64)
    ref = du.attention64(q.detach(), ke, ke, torch.ones_like(y), seen, 1 / 8.0)
    du.check("dq", q.grad, ref["dq"])
    u = du.half_step(torch.bfloat16)
    terms = ref["dk"][0].abs().sum((0, 1)) + ref["dv"][0].abs().sum((0, 1))
    want = (ref["dk"][0] + ref["dv"][0]).sum((0, 1))
    # eight gradients summed in bf16 by autograd, each sum rounded (at most 9 roundings of at most the sum of sizes)
    bound = (ref["dk"][1] + ref["dv"][1]).sum((0, 1)) + 9 * u * terms
    du.check("dkv", kv.grad[0, 0], (want, bound))


def test_rotary_in_the_layer_and_the_dense_attention():
    """lighthouse_attention with one level is causal attention: with rotary positions it is the dense attention with the
    same positions, and equals turning q and k first."""
    q, k, v = (randn((1, 2, 256, 64), torch.bfloat16, s) for s in (1, 2, 3))
    rope = lh.Rotary.make(64)
    y = lh.lighthouse_attention(q, k, v, 1, 2, 64, rotary=rope)
    qr, kr = lh.apply_rotary(q, k, rope)
    assert torch.equal(y, lh.lighthouse_attention(qr, kr, v, 1, 2, 64))
    z = lh.dense_attention(q, k, v, rotary=rope)
    assert torch.equal(z, lh.dense_attention(qr, kr, v))
    seen = du.seen_matrix(1, 256, device="cuda")
    ref = du.attention64(qr, kr, v, torch.zeros_like(v), seen, 1 / 8.0)["o"]
    du.check("dense", z, ref)
    du.check("layer", y, ref)


def test_gradient_through_the_layer_with_rotary():
    """lighthouse_attention(rotary=): the gradients are the layer's on the turned inputs, turned back."""
    q, k, v, g = (randn((1, 2, 512, 64), torch.bfloat16, s) for s in (1, 2, 3, 4))
    rope = lh.Rotary.make(32, layout="interleaved", scaling="linear", factor=2.0)
    pos = torch.randint(0, 100000, (1, 512), dtype=torch.int32, device="cuda")
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    y = lh.lighthouse_attention(*x, 3, 2, 64, rotary=rope, positions=pos)
    y.backward(g)
    turned = [t.detach().requires_grad_() for t in (*lh.rotary(q, k, rope.frequencies, pos, "interleaved"), v)]
    z = lh.lighthouse_attention(*turned, 3, 2, 64)
    z.backward(g)
    assert torch.equal(y, z)
    back = lh.rotary(turned[0].grad, turned[1].grad, rope.frequencies, pos, "interleaved", inverse=True)
    for a, b in zip(x, (*back, turned[2].grad)):
        assert torch.equal(a.grad, b)
    # and those of the formula: with one level the layer is causal attention
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    lh.lighthouse_attention(*x, 1, 2, 64, rotary=rope, positions=pos).backward(g)
    qr, kr = lh.rotary(q, k, rope.frequencies, pos, "interleaved")
    ref = du.attention64(qr, kr, v, g, du.seen_matrix(1, 512, device="cuda"), 1 / 8.0)
    du.check("dv", x[2].grad, ref["dv"])


def test_streams_and_graphs():
    """Calls on another stream than the default one, and captured and replayed with new inputs in place."""
    case = (1, 4, 2, 200, 64, "bf16", 1, 1, True, 10.0, 0, 0)
    t = dense_inputs(case)
    want = run_dense(case, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_dense(case, t)
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(got[n], want[n])
    other = dense_inputs(case, seed=5)
    want2 = run_dense(case, other[:4] + t[4:])
    static = [x.clone() for x in t[:4]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mask = lh.attention_mask(t[4], t[5])
        o, saved = lh.dense_forward(*static[:3], mask=mask, softcap=10.0)
        grads = lh.dense_backward(static[3], *static[:3], o, saved, mask=mask, softcap=10.0)
    for src, want_ in ((t, want), (other, want2)):
        for a, b in zip(static, src[:4]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, saved.lse, *grads)):
            assert torch.equal(x, want_[n]), n

"""Plain fp64 forms of the dense attention's operators and the error bounds of
their kernels.  The bounds count roundings: a value held in a 16-bit type is off
by at most half a step, u = finfo.eps / 2 relative; sums and exponentials are
fp32, whose errors (the exponent of a score of size 2^6 carries 2^-17) are
covered by F = 2^-14 of the sums of magnitudes."""

import math

import torch

F = 2.0 ** -14


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def seen_matrix(B, N, docs=None, prefix=None, causal=True, device="cpu"):
    """[B, N, N] truth: query i sees key j, from the definition (runs of equal ids, leading prefix tokens)."""
    ids = torch.zeros(B, N, dtype=torch.int64) if docs is None else docs.cpu().long()
    pre = torch.zeros(B, N, dtype=torch.bool) if prefix is None else prefix.cpu().bool()
    out = torch.zeros(B, N, N, dtype=torch.bool)
    for b in range(B):
        i = 0
        while i < N:
            e = i
            while e < N and ids[b, e] == ids[b, i]:
                e += 1
            if ids[b, i] >= 0:
                p = i
                while p < e and pre[b, p]:
                    p += 1
                block = torch.ones(e - i, e - i, dtype=torch.bool)
                out[b, i:e, i:e] = block.tril() if causal else block
                out[b, i:e, i:p] = True
            i = e
    return out.to(device)


def attention64(q, k, v, do, seen, scale, softcap=0.0, slopes=None):
    """Outputs, gradients and their bounds (a dict name -> (value, bound)) of the masked attention, in fp64.  Rows of
    padding (seen by nothing) may hold anything: they enter as zeros."""
    dt = q.dtype
    u = half_step(dt)
    live_q, live_k = seen.any(-1), seen.any(-2)
    q, do = (torch.where(live_q[:, None, :, None], t.double(), 0.0) for t in (q, do))
    k, v = (torch.where(live_k[:, None, :, None], t.double(), 0.0) for t in (k, v))
    B, Hq, N, d = q.shape
    G = Hq // k.shape[1]
    ke, ve = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = q @ ke.transpose(-1, -2) * scale
    slope = torch.ones_like(x)
    if softcap:
        t = torch.tanh(x / softcap)
        x, slope = softcap * t, 1 - t * t
    if slopes is not None:
        i = torch.arange(N, device=q.device)
        x = x - slopes.double()[:, None, None] * (i[:, None] - i).abs()
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e300)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total))[..., 0].masked_fill(~live_q[:, None], -math.inf)
    p = p / total.clamp_min(1e-300)
    o = p @ ve
    dp = do @ ve.transpose(-1, -2)
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * slope * scale
    fold = lambda t: t.view(B, Hq // G, G, N, -1).sum(2)  # noqa: E731
    val = dict(o=o, dq=ds @ ke, dk=fold(ds.transpose(-1, -2) @ q), dv=fold(p.transpose(-1, -2) @ do))
    # O: P's roundings and O's own; dV: P's and its own
    bo = u * o.abs() + (u + F) * (p @ ve.abs())
    bv = u * val["dv"].abs() + (u + F) * fold(p.transpose(-1, -2) @ do.abs())
    # dS: its own rounding, and Delta = rowsum(dO * O), off by what O is off by
    off = (u + F) * ds.abs() + p * slope * scale * ((do.abs() * bo).sum(-1, keepdim=True)
                                                    + F * (do.abs() @ ve.abs().transpose(-1, -2)))
    bq = u * val["dq"].abs() + off @ ke.abs()
    bk = u * val["dk"].abs() + fold(off.transpose(-1, -2) @ q.abs())
    bound = dict(o=bo, dq=bq, dk=bk, dv=bv)
    tiny = float(torch.finfo(dt).smallest_normal) * u * 2  # half a step of the smallest numbers
    out = {n: (val[n], bound[n] * (1 + 2.0 ** -5) + tiny * max(1, N)) for n in val}
    out["lse"] = (lse, 2.0 ** -18 * (1 + lse.abs().clamp_max(1e6)))
    return out


def check(name, got, ref):
    value, bound = ref
    got = got.double()
    same = torch.isinf(value) & (got == value)
    err = torch.where(same, 0.0, (got - value).abs())
    bad = ~(err <= torch.where(same, 1.0, bound))
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: got {got[at].item()}, "
                             f"expected {value[at].item()} +- {bound[at].item()}")


def rotate64(x, positions, frequencies, layout, amplitude=1.0, inverse=False):
    """[B, H, N, d] turned by positions [B, N] * frequencies, in fp64."""
    n = 2 * frequencies.numel()
    angle = positions.double()[:, None, :, None] * frequencies.double()
    turn = torch.polar(torch.full_like(angle, amplitude), -angle if inverse else angle)
    y = x.double().clone()
    a, b = (slice(0, n // 2), slice(n // 2, n)) if layout == "half" else (slice(0, n, 2), slice(1, n, 2))
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def quantise64(x, kind):
    """What a row of an 8-bit cache stands for (rows last), by arithmetic in fp64, and how far a held value may be off:
    the fp32 multiplier may move a value across the border of two steps, by one step of the held type."""
    x = x.double()
    top = 448.0 if kind == "e4m3" else 127.0
    scale = x.abs().amax(-1, keepdim=True) / top
    y = x / torch.where(scale > 0, scale, 1.0)
    if kind == "e4m3":
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    else:
        step = torch.ones_like(y)
    return torch.round(y / step) * step * scale, step * scale


def cache_attention64(q, keys, values, T_start, lens, tree=None, scale=None, softcap=0.0, slopes=None):
    """q [n, Hq, d]; keys, values: list of [len, Hkv, d] (fp64) per sequence; T_start: first token of each sequence and
    the end.  -> value, bound (probabilities rounded to the operand type, the output to its own)."""
    u = half_step(q.dtype)
    n, Hq, d = q.shape
    out, mag = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device), torch.zeros(n, Hq, d, dtype=torch.float64,
                                                                                        device=q.device)
    scale = 1 / math.sqrt(d) if scale is None else scale
    for s, (k, v) in enumerate(zip(keys, values)):
        L, T = lens[s], T_start[s + 1] - T_start[s]
        G = Hq // k.shape[1]
        j = torch.arange(L, device=q.device)
        for t in range(T):
            row, at = T_start[s] + t, L - T + t
            x = torch.einsum("hd,jhd->hj", q[row].double(), k.repeat_interleave(G, 1)) * scale
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - slopes.double()[:, None] * (at - j).abs()
            seen = j <= at
            if tree is not None:
                bits = int(tree[row])
                seen = torch.tensor([i < L - T or bool(bits >> (i - (L - T)) & 1) for i in range(L)], device=q.device)
            if L == 0 or not bool(seen.any()):
                continue
            p = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
            out[row] = torch.einsum("hj,jhd->hd", p, v.repeat_interleave(G, 1))
            mag[row] = torch.einsum("hj,jhd->hd", p, v.repeat_interleave(G, 1).abs())
    return out, (u * out.abs() + (u + F) * mag) * (1 + 2.0 ** -5) + float(torch.finfo(q.dtype).smallest_normal) * u * 2

"""The operators around the dense attention that a model trained with the Lighthouse layer resumes on and is served
with: rotary positions, masked attention with its gradient, a quantised paged cache, and the attention over that cache.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` the inputs a program has in hand, `run(state)` one pass:
the package's calls where `own` is true, and the same operators in elementary torch operations where it is false.
`exact(case, seed)` computes the outputs in 64 bits from the definitions, and `work(case)` counts what a pass cannot
do without."""

import math

import torch

own = False

FP8_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    rot = dict(op="rotary", base=1e6, factor=1.0, original=8192, layout="half")
    attn = dict(op="attention", B=1, docs=0, prefix=False, pad=0, softcap=0.0, alibi=False, token_major=True)
    rw = dict(op="cache", page=64, dtype="bf16")
    dec = dict(op="decode", page=64, tokens=1, tree=False, softcap=0.0, alibi=False, dtype="bf16")
    return [
        # one decoding step of 48 sequences: the queries and keys of one token each, at far apart positions, half of
        # the channels rotated in interleaved pairs
        dict(rot, name="rotary_step", B=1, N=48, Hq=16, Hk=4, d=128, rot=64, layout="interleaved", dtype="bf16",
             ragged=True, backward=False),
        # a training step's forward and backward rotation over 128K tokens, positions stretched 16 times (YaRN)
        dict(rot, name="rotary_128k_train", B=1, N=131072, Hq=16, Hk=4, d=128, rot=128, dtype="bf16", factor=16.0,
             ragged=False, backward=True),
        # a short batch: odd length, prefix masks, capped scores, grouped heads
        dict(attn, name="attn_small_prefix", B=2, N=257, Hq=8, Hkv=2, d=64, dtype="fp16", docs=3, prefix=True,
             softcap=30.0),
        # packed documents of a training batch, causal within each, grouped heads
        dict(attn, name="attn_8k_docs", N=8192, Hq=16, Hkv=4, d=128, dtype="bf16", docs=7),
        # distance bias over a padded batch of odd length
        dict(attn, name="attn_4k_alibi", B=2, N=4001, Hq=8, Hkv=8, d=128, dtype="bf16", pad=313, alibi=True,
             token_major=False),
        # the dense resume of a long context: plain causal attention, 8 heads of 16K tokens
        dict(attn, name="attn_16k_causal", N=16384, Hq=8, Hkv=8, d=128, dtype="bf16"),
        # 48 sequences write their newest token; the short contexts are read back
        dict(rw, name="cache_step", kind="int8", seqs=48, longest=200, heads=4, d=128),
        # the prompts of a batch are quantised into pages and read back for the prefill's attention
        dict(rw, name="cache_prompts", kind="e4m3", seqs=12, longest=16384, heads=4, d=128),
        # smallest step: 4 short sequences, unquantised cache
        dict(dec, name="decode_small", kind="bf16", seqs=4, longest=600, Hq=16, Hkv=4, d=128),
        # a serving batch: 64 sequences of up to 8K tokens in 8 bits, capped scores
        dict(dec, name="decode_batch", kind="e4m3", seqs=64, longest=8192, Hq=16, Hkv=4, d=128, softcap=50.0),
        # one sequence of 512K tokens in 8 bits
        dict(dec, name="decode_512k", kind="int8", seqs=1, longest=524288, Hq=16, Hkv=4, d=128),
        # verification of a tree of 24 drafted tokens for each of 16 sequences
        dict(dec, name="decode_tree", kind="e4m3", seqs=16, longest=5000, Hq=16, Hkv=4, d=128, page=16, tokens=24,
             tree=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "cache", "decode", "decode"])
    group = rng.choice([1, 2, 4, 8])
    hk = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    if op == "rotary":
        c = dict(op=op, base=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([1.0, 4.0, 16.0]), original=8192,
                 layout=rng.choice(["half", "interleaved"]), B=rng.choice([1, 2, 3]), N=_log_uniform(rng, 1, 131072),
                 Hq=hk * group, Hk=hk, d=d, rot=rng.choice([d, d // 2, d // 4, d - 16, 2 * rng.randint(1, d // 2)]),
                 dtype=rng.choice(["bf16", "fp16", "fp32"]), ragged=rng.random() < 0.5, backward=rng.random() < 0.5)
    elif op == "attention":
        c = dict(op=op, B=rng.choice([1, 1, 2]), N=_log_uniform(rng, 4, 16384), Hq=hk * group, Hkv=hk, d=d,
                 dtype=rng.choice(["bf16", "fp16"]), docs=rng.choice([0, 1, 2, 5, 9]), prefix=rng.random() < 0.4,
                 pad=rng.choice([0, 0, 1, 70]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=rng.random() < 0.3,
                 token_major=rng.random() < 0.5)
        c["pad"] = min(c["pad"], c["N"] - 4)
        if not c["docs"] and (c["prefix"] or c["pad"]):
            c["docs"] = 1
    elif op == "cache":
        c = dict(op=op, kind=rng.choice(["e4m3", "int8", "bf16", "fp16"]), seqs=rng.randint(1, 48),
                 longest=_log_uniform(rng, 1, 16384), heads=hk, d=d, page=rng.choice([16, 32, 64, 128]),
                 dtype=rng.choice(["bf16", "fp16", "fp32"]))
        if c["kind"] in ("bf16", "fp16"):
            c["dtype"] = c["kind"]
    else:
        tree = rng.random() < 0.4
        c = dict(op=op, kind=rng.choice(["e4m3", "int8", "bf16", "fp16"]), seqs=_log_uniform(rng, 1, 96),
                 longest=_log_uniform(rng, 1, 262144), Hq=hk * group, Hkv=hk, d=d, page=rng.choice([16, 32, 64, 128]),
                 tokens=rng.randint(2, 40) if tree else rng.choice([1, 1, 1, 4]), tree=tree,
                 softcap=rng.choice([0.0, 0.0, 50.0]), alibi=(not tree) and rng.random() < 0.3,
                 dtype=rng.choice(["bf16", "fp16"]))
        if c["kind"] in ("bf16", "fp16"):
            c["dtype"] = c["kind"]
        c["longest"] = max(c["longest"], c["tokens"])
    # a drawn case costs no more than the largest listed one of its operator
    most = max((work(x) for x in listed() if x["op"] == op), key=_cost)
    if _cost(work(c)) > _cost(most) or _plain_elements(c) > 3 << 30:
        return draw(rng)
    return c


def _cost(w):
    return w["bytes"] / 6.5e12 + w["flops"] / 1.5e15


def _plain_elements(c):
    """Scores the plain form holds at once (it makes whole score matrices)."""
    if c["op"] == "attention":
        return c["B"] * c["Hq"] * c["N"] ** 2
    if c["op"] == "decode":
        return c["seqs"] * c["longest"] * (c["Hkv"] * c["d"] + c["Hq"] * c["tokens"])
    return 0


# ----------------------------------------------------------------------------------------------- what a case holds

def _lengths(c):
    """Lengths of the cached sequences, from one token to the longest, the same for every seed."""
    n, hi, lo = c["seqs"], c["longest"], c.get("tokens", 1)
    if n == 1:
        return [hi]
    return [max(lo, int(hi * (((i * 7919) % n + 1) / n) ** 1.5)) for i in range(n)]


def _doc_lengths(c):
    """Lengths of one row's documents (they fill N - pad tokens); none: the whole row is one document."""
    n = c["N"] - c["pad"]
    # two tokens a document at least: where every query has one key alone, the gradients are zero but for rounding
    k = min(max(1, c["docs"]), n // 4 + 1)
    w = [1 + (i * 5 + 3) % (2 * k + 1) for i in range(k)]
    cut = [2 * i + (n - 2 * k) * sum(w[:i]) // sum(w) for i in range(k + 1)]
    return [b - a for a, b in zip(cut, cut[1:])]


def _pairs(c):
    """(query, key) pairs that the masks of one row leave."""
    total = 0
    for n in _doc_lengths(c):
        p = (n // 3 + 1) if c["prefix"] else 0
        total += n * (n + 1) // 2 + max(0, p * (p - 1) // 2)
    return total


def work(c):
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rotary":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hk"]) * c["d"]
        passes = 2 if c["backward"] else 1
        return {"bytes": 2.0 * n * e * passes + 4.0 * c["B"] * c["N"], "flops": 3.0 * n * passes}
    if c["op"] == "attention":
        q, kv = c["B"] * c["Hq"] * c["N"] * c["d"], c["B"] * c["Hkv"] * c["N"] * c["d"]
        # in: q, k, v, the output's gradient; out: the output and three gradients
        return {"bytes": e * (4.0 * q + 4.0 * kv), "flops": 14.0 * c["d"] * c["B"] * c["Hq"] * _pairs(c)}
    held = {"e4m3": 1, "int8": 1, "bf16": 2, "fp16": 2}[c["kind"]]
    row = held * c["d"] + (4 if held == 1 else 0)
    if c["op"] == "cache":
        # read the tokens, write them as they are held, read that, write them back out
        n = 2.0 * sum(_lengths(c)) * c["heads"]
        return {"bytes": n * (2 * row + 2 * e * c["d"]), "flops": 4.0 * n * c["d"]}
    n = float(sum(_lengths(c)))
    q = c["seqs"] * c["tokens"] * c["Hq"] * c["d"]
    return {"bytes": 2 * n * c["Hkv"] * row + 2.0 * e * q, "flops": 4.0 * n * c["tokens"] * c["Hq"] * c["d"]}


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dt)

    if c["op"] == "rotary":
        s = dict(c)
        shapes = [(c["B"], c["N"], h, c["d"]) for h in (c["Hq"], c["Hk"])]
        # the projections' outputs, tokens before heads; the calls see [B, H, N, d]
        s["q"], s["k"] = (normal(*x).transpose(1, 2) for x in shapes)
        if c["backward"]:
            s["dq"], s["dk"] = (normal(*x).transpose(1, 2) for x in shapes)
        hi = 1 << 20
        if c["ragged"]:
            s["positions"] = torch.randint(0, hi, (c["B"], c["N"]), generator=g, device=dev, dtype=torch.int32)
        else:
            s["positions"] = torch.arange(c["N"], device=dev, dtype=torch.int32).expand(c["B"], -1).contiguous()
        s["frequencies"], s["amplitude"] = _frequencies(c)
        s["frequencies"] = s["frequencies"].to(dev)
        return s
    if c["op"] == "attention":
        s = dict(c)

        def heads(h, scale=1.0):
            if c["token_major"]:
                return normal(c["B"], c["N"], h, c["d"], scale=scale).transpose(1, 2)
            return normal(c["B"], h, c["N"], c["d"], scale=scale)

        s["q"], s["k"], s["v"], s["do"] = heads(c["Hq"], 1.5), heads(c["Hkv"]), heads(c["Hkv"]), heads(c["Hq"])
        s["docs_ids"] = s["prefix_mask"] = None
        if c["docs"]:
            lens = _doc_lengths(c)
            ids = sum(([i] * n for i, n in enumerate(lens)), []) + [-1] * c["pad"]
            s["docs_ids"] = torch.tensor([ids] * c["B"], dtype=torch.int32, device=dev)
            if c["prefix"]:
                pre = sum(([t < n // 3 + 1 for t in range(n)] for n in lens), []) + [False] * c["pad"]
                s["prefix_mask"] = torch.tensor([pre] * c["B"], device=dev)
        s["slopes"] = _slopes(c["Hq"]).to(dev) if c["alibi"] else None
        return s
    s = dict(c)
    lens = _lengths(c)
    page, heads, d = c["page"], c["heads" if c["op"] == "cache" else "Hkv"], c["d"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64)
    width = max(need)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    owner = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(need))
    first = torch.tensor([0] + need).cumsum(0)
    col = torch.arange(sum(need)) - first[owner]
    table[owner, col] = order[: sum(need)].cpu().to(torch.int32)
    s["page_table"] = table.to(dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["starts"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    s["total"] = sum(lens)
    s["width"] = max(lens)
    held = KINDS[c["kind"]]
    shape = (pages, heads, page, d)
    if c["op"] == "cache":
        s["k"], s["v"] = normal(s["total"], heads, d), normal(s["total"], heads, d, scale=0.3)
        s["cache"] = [torch.zeros(shape, dtype=torch.uint8, device=dev).to(held) for _ in range(2)]
        s["scales"] = [torch.zeros(shape[:3], device=dev) for _ in range(2)] if held.itemsize == 1 else [None, None]
        tok = torch.arange(s["total"], device=dev)
        seq = torch.searchsorted(s["starts"].long(), tok, right=True) - 1
        pos = tok - s["starts"].long()[seq]
        s["slots"] = s["page_table"].long()[seq, pos // page] * page + pos % page
        return s
    s["q"] = normal(len(lens) * c["tokens"], c["Hq"], d, scale=1.5)
    s["cache"], s["scales"] = [], []
    for scale in (1.0, 0.5):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if held.itemsize == 1:
            lim = 110.0 if held == torch.float8_e4m3fn else 32.0
            s["cache"].append((x * lim).clamp(-FP8_MAX if lim > 100 else -127, FP8_MAX if lim > 100 else 127).to(held))
            s["scales"].append((torch.rand(shape[:3], generator=g, device=dev) + 0.5) * (scale / lim))
        else:
            s["cache"].append((x * scale).to(held))
            s["scales"].append(None)
    s["q_start"] = (torch.arange(len(lens) + 1, dtype=torch.int32) * c["tokens"]).to(dev)
    s["slopes"] = _slopes(c["Hq"]).to(dev) if c["alibi"] else None
    s["tree_mask"] = None
    if c["tree"]:
        # a random tree for every sequence: each drafted token continues an earlier one (or the last cached token)
        r = torch.rand(len(lens), c["tokens"], generator=g, device=dev).cpu().tolist()
        masks = []
        for row in r:
            seen = []
            for t, u in enumerate(row):
                parent = int(u * (t + 1)) - 1
                seen.append((seen[parent] if parent >= 0 else 0) | (1 << t))
            masks += seen
        s["tree_mask"] = torch.tensor(masks, dtype=torch.int64, device=dev)
    return s


def _slopes(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32)


def _frequencies(c):
    """Angle per position of each rotated pair, in 64 bits, and the amplitude: YaRN's blend of stretched and plain
    frequencies where the factor is above 1."""
    n = c["rot"]
    i = torch.arange(0, n, 2, dtype=torch.float64)
    f = float(c["base"]) ** (-i / n)
    if c["factor"] == 1.0:
        return f, 1.0
    at = [n * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"])) for turns in (32.0, 1.0)]
    lo, hi = max(0, math.floor(at[0])), min(n - 1, math.ceil(at[1]))
    ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / c["factor"] * ramp, 0.1 * math.log(c["factor"]) + 1.0


# --------------------------------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "rotary":
        out = [_rotate(s[n], s, 1.0) for n in ("q", "k")]
        if s["backward"]:
            out += [_rotate(s[n], s, -1.0) for n in ("dq", "dk")]
        return out
    if s["op"] == "attention":
        return _attention(s)
    if s["op"] == "cache":
        return _write_and_read(s)
    return _decode(s)


def _run_own(s):
    import hierarchical_sparse_attention_pyramid_b200 as lh
    if s["op"] == "rotary":
        opt = dict(layout=s["layout"], amplitude=s["amplitude"])
        out = list(lh.rotary(s["q"], s["k"], s["frequencies"], s["positions"], **opt))
        if s["backward"]:
            out += lh.rotary(s["dq"], s["dk"], s["frequencies"], s["positions"], inverse=True, **opt)
        return out
    if s["op"] == "attention":
        mask = None
        if s["docs_ids"] is not None:
            mask = lh.attention_mask(s["docs_ids"], s["prefix_mask"])
        opt = dict(mask=mask, softcap=s["softcap"], slopes=s["slopes"])
        o, lse = lh.dense_forward(s["q"], s["k"], s["v"], **opt)
        return [o, *lh.dense_backward(s["do"], s["q"], s["k"], s["v"], o, lse, **opt)]
    cache = lh.KVCache(*s["cache"], *s["scales"])
    if s["op"] == "cache":
        lh.cache_write(cache, s["k"], s["v"], s["slots"])
        return list(lh.cache_read(cache, s["page_table"], s["starts"], s["total"], dtype=DTYPES[s["dtype"]]))
    return lh.cache_attention(cache, s["q"], s["page_table"], s["lens"], q_start=s["q_start"],
                              max_tokens=s["tokens"], tree_mask=s["tree_mask"], softcap=s["softcap"],
                              slopes=s["slopes"])


def _rotate(x, s, sign):
    """Pairs of the first `rot` channels turned by position * frequency; the angle is taken in 64 bits, since far
    positions leave no fraction of a turn in 32."""
    angle = (s["positions"].double()[:, None, :, None] * s["frequencies"])
    sin, cos = (torch.sin(angle) * sign * s["amplitude"]).float(), (torch.cos(angle) * s["amplitude"]).float()
    n = s["rot"]
    x32 = x.float()
    if s["layout"] == "half":
        a, b = x32[..., : n // 2], x32[..., n // 2: n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x32[..., 0:n:2], x32[..., 1:n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x32[..., n:]], -1).to(x.dtype)


def _spans(s):
    """[lo, hi) of the keys each query sees: its document up to itself, and the document's leading prefix tokens."""
    i = torch.arange(s["N"], device=s["q"].device)
    if s["docs_ids"] is None:
        return torch.zeros_like(i)[None], (i + 1)[None]
    ids = s["docs_ids"]
    edge = torch.ones_like(ids, dtype=torch.bool)
    edge[:, 1:] = ids[:, 1:] != ids[:, :-1]
    lo = torch.where(edge, i, 0).cummax(1).values
    hi = (i + 1).expand_as(lo)
    if s["prefix_mask"] is not None:
        # the number of leading prefix tokens: those with no plain token of the document before them
        broken = (~s["prefix_mask"]).long().cumsum(1)
        before = broken.gather(1, lo) - (~s["prefix_mask"]).long().gather(1, lo)
        leading = s["prefix_mask"] & (broken == before)
        run = edge.long().cumsum(1) - 1
        count = torch.zeros_like(run).scatter_add_(1, run, leading.long()).gather(1, run)
        hi = torch.maximum(hi, lo + count)
    hi = torch.where(ids >= 0, hi, lo)
    return lo, hi


def _attention(s):
    """Masked attention and its gradient as whole matrices in 32 bits."""
    q, k, v, do = (s[n].float() for n in ("q", "k", "v", "do"))
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q, do = q.reshape(B, Hkv, G * N, d), do.reshape(B, Hkv, G * N, d)
    scale = 1.0 / math.sqrt(d)
    lo, hi = _spans(s)
    j = torch.arange(N, device=q.device)
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, None]  # [B or 1, 1, 1, N, N]
    x = (q @ k.transpose(-1, -2)).mul_(scale).view(B, Hkv, G, N, N)
    slope = None
    if s["softcap"]:
        x = torch.tanh(x.div_(s["softcap"]))
        slope = 1 - x * x
        x = x.mul_(s["softcap"])
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, Hkv, G, 1, 1) * (j[:, None] - j).abs().float()
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(x.sub_(m))
    del x
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1))
    p = p.view(B, Hkv, G * N, N)
    o = p @ v
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    if slope is not None:
        ds.mul_(slope.view_as(ds))
    ds.mul_(scale)
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    dt = s["q"].dtype
    return [o.view(B, Hq, N, d).to(dt), dq.view(B, Hq, N, d).to(dt), dk.to(dt), dv.to(dt)]


def _quantise(x, held):
    """One scale for a token's head: its largest magnitude over the type's; what is held is x over the scale, rounded
    to nearest even."""
    if held.itemsize != 1:
        return x.to(held), None
    top = FP8_MAX if held == torch.float8_e4m3fn else 127.0
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    y = x * torch.where(amax > 0, top / amax, 0)
    return (y if held == torch.float8_e4m3fn else y.round()).clamp(-top, top).to(held), (amax / top)[..., 0]


def _dequantise(x, scale):
    return x.float() if scale is None else x.float() * scale[..., None]


def _write_and_read(s):
    pages, heads, page, d = s["cache"][0].shape
    at, row = s["slots"] // page, s["slots"] % page
    tok = torch.arange(s["total"], device=at.device)
    seq = torch.searchsorted(s["starts"].long(), tok, right=True) - 1
    pos = tok - s["starts"].long()[seq]
    src = s["page_table"].long()[seq, pos // page]

    def through(x, cache, scales):
        held, scale = _quantise(x, cache.dtype)
        cache.view(torch.int8 if cache.element_size() == 1 else torch.int16)[at, :, row] = held.view(
            torch.int8 if cache.element_size() == 1 else torch.int16)
        if scale is not None:
            scales[at, :, row] = scale
        got = cache.view(torch.int8 if cache.element_size() == 1 else torch.int16)[src, :, pos % page].view(cache.dtype)
        return _dequantise(got, None if scale is None else scales[src, :, pos % page]).to(DTYPES[s["dtype"]])

    return [through(s["k"], s["cache"][0], s["scales"][0]), through(s["v"], s["cache"][1], s["scales"][1])]


def _decode(s):
    """Every sequence's cache gathered, padded to the longest, and attended as one batch in 32 bits."""
    pages, Hkv, page, d = s["cache"][0].shape
    T, n, Hq = s["tokens"], s["lens"].numel(), s["q"].shape[1]
    G, L = Hq // Hkv, s["width"]
    j = torch.arange(L, device=s["q"].device)
    lens = s["lens"].long()[:, None]
    at = torch.where(j < lens, s["page_table"].long().gather(1, (j // page).expand(n, -1)), 0)

    def fetch(cache, scales):
        raw = torch.int8 if cache.element_size() == 1 else torch.int16
        x = cache.view(raw).transpose(1, 2)[at, (j % page).expand_as(at)].view(cache.dtype)  # [n, L, Hkv, d]
        x = _dequantise(x, None if scales is None else scales.transpose(1, 2)[at, (j % page).expand_as(at)])
        return x.transpose(1, 2)

    k = fetch(s["cache"][0], s["scales"][0])
    q = s["q"].float().view(n, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * T, d)
    x = (q @ k.transpose(-1, -2)).view(n, Hkv, G, T, L) * (1.0 / math.sqrt(d))
    del k
    t = torch.arange(T, device=j.device)
    last = lens + t - T  # position of each query token [n, T]
    if s["softcap"]:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, G, 1, 1) * (last[..., None] - j).abs().float()[:, None, None]
    seen = j <= last[..., None]
    if s["tree_mask"] is not None:
        drafted = j - (lens - T)  # index among the drafted tokens, negative for the context
        bits = s["tree_mask"].view(n, T, 1) >> drafted.clamp(0, T - 1)[:, None]
        seen = ((drafted < 0)[:, None] | ((bits & 1) > 0)) & (j < lens)[:, None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p = p / p.sum(-1, keepdim=True)
    o = p.view(n, Hkv, G * T, L) @ fetch(s["cache"][1], s["scales"][1])
    return o.view(n, Hkv, G, T, d).permute(0, 3, 1, 2, 4).reshape(n * T, Hq, d).to(s["q"].dtype)


# ----------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"rotary": _exact_rotary, "attention": _exact_attention, "cache": _exact_cache,
            "decode": _exact_decode}[c["op"]](s)


def _exact_rotary(s):
    # a pair of channels as a complex number, turned by exp(i angle)
    n = s["rot"]
    angle = s["positions"].double()[:, None, :, None] * s["frequencies"]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)
    out = []
    for name in ("q", "k", "dq", "dk") if s["backward"] else ("q", "k"):
        x = s[name].double().contiguous()
        y = x.clone()
        a, b = (slice(0, n // 2), slice(n // 2, n)) if s["layout"] == "half" else (slice(0, n, 2), slice(1, n, 2))
        z = torch.complex(x[..., a], x[..., b]) * (turn.conj() if name[0] == "d" else turn)
        y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return out


def _exact_attention(s):
    # row blocks of one head at a time, the gradient by automatic differentiation
    B, Hq, N, d = s["q"].shape
    if B * Hq * N * N > 2 << 30:
        return None
    G = Hq // s["k"].shape[1]
    q, k, v = (s[n].double().contiguous().requires_grad_() for n in ("q", "k", "v"))
    o = torch.zeros_like(q, requires_grad=False)
    dev = q.device
    j = torch.arange(N, device=dev)
    for b in range(B):
        ids = torch.zeros(N, dtype=torch.int32, device=dev) if s["docs_ids"] is None else s["docs_ids"][b]
        pre = torch.zeros(N, dtype=torch.bool, device=dev) if s["prefix_mask"] is None else s["prefix_mask"][b]
        for h in range(Hq):
            for i0 in range(0, N, 2048):
                i = j[i0:i0 + 2048]
                x = q[b, h, i0:i0 + 2048] @ k[b, h // G].T / math.sqrt(d)
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (i[:, None] - j).abs()
                seen = (ids[i][:, None] == ids) & (ids >= 0) & ((j <= i[:, None]) | pre)
                p = torch.softmax(x.masked_fill(~seen, -1e300), -1) * seen
                y = p @ v[b, h // G]
                o[b, h, i0:i0 + 2048] = y.detach()
                torch.autograd.backward(y, s["do"][b, h, i0:i0 + 2048].double())
    return [o, q.grad, k.grad, v.grad]


def _exact_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        x = x.double()
        held = s["cache"][0].dtype
        if held.itemsize == 1:
            top = FP8_MAX if held == torch.float8_e4m3fn else 127.0
            scale = x.abs().amax(-1, keepdim=True) / top
            y = x / torch.where(scale > 0, scale, 1)
            if held == torch.float8_e4m3fn:
                # steps of an eighth of the power of two below the value, none finer than 2^-9
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
                x = torch.round(y / step) * step * scale
            else:
                x = torch.round(y) * scale
        out.append(x)
    return out


def _exact_decode(s):
    pages, Hkv, page, d = s["cache"][0].shape
    T, Hq = s["tokens"], s["q"].shape[1]
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["lens"].tolist()):
        used = s["page_table"][i, : -(-n // page)].long()
        j = torch.arange(n, device=out.device)
        for h in range(Hkv):
            k, v = (torch.stack([x[a, h] for a in used.tolist()]).reshape(-1, d)[:n].double()
                    if len(used) < 64 else x.view(torch.int8 if x.element_size() == 1 else torch.int16)[:, h][used]
                    .view(x.dtype).reshape(-1, d)[:n].double() for x in s["cache"])
            if s["scales"][0] is not None:
                k, v = (y * z[used, h].reshape(-1)[:n, None].double() for y, z in zip((k, v), s["scales"]))
            for t in range(T):
                row, at = i * T + t, n - T + t
                x = s["q"][row, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h * G:(h + 1) * G, None].double() * (at - j).abs()
                seen = j <= at
                if s["tree_mask"] is not None:
                    mask = int(s["tree_mask"][row])
                    seen = torch.tensor([True] * (n - T) + [bool(mask >> u & 1) for u in range(T)], device=out.device)
                out[row, h * G:(h + 1) * G] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ v
    return out

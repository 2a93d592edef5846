"""Cases for timing the operators of a serving step over the paged cache.

A layer that decodes or prefills in chunks over the paged cache runs four
operators around the indexer: it norms and rotates its queries and keys
(``rope``), writes the new keys and values into the cache's pages (``append``),
attends densely from the new tokens (``attend``), or attends over the index
rows (``sparse``).  Each case below is one call of one of them; with ``own``
set it is the library's call, otherwise the plain form in elementary torch
operations.

Shapes follow the repository's workloads (16 heads of 128 at L = 8192, 32 heads
at 32768, 64-channel heads of the small one, steps of two tokens) next to
generic grouped-head ones.  Keys carry the generators' heavy rows: 1 % of the
positions are four times as long.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ the cases
def rope_case(T, Hq, Hk, d, rot, layout, scaling, norm, dtype, far):
    """T tokens ending at position `far`; Hq + Hk heads; the first `rot` channels turn."""
    return {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "layout": layout, "scaling": scaling,
            "norm": norm, "dtype": dtype, "far": far}


def append_case(B, new, ragged, Hq, Hk, d, page, ctx, rot, layout, norm, values, dtype):
    """B sequences of up to `ctx` cached rows take up to `new` rows each; Hq = 0 leaves the queries out."""
    return {"op": "append", "B": B, "new": new, "ragged": ragged, "Hq": Hq, "Hk": Hk, "d": d, "page": page,
            "ctx": ctx, "rot": rot, "layout": layout, "norm": norm, "values": values, "dtype": dtype}


def attend_case(B, new, ragged, Hq, Hk, d, page, ctx, itself):
    """Dense causal attention of up to `new` new tokens per sequence over up to `ctx` rows before them."""
    return {"op": "attend", "B": B, "new": new, "ragged": ragged, "Hq": Hq, "Hk": Hk, "d": d, "page": page,
            "ctx": ctx, "itself": itself}


def sparse_case(B, g, H, d, page, ctx, top_k):
    """Attention over index rows of top_k entries, g rows (one step) per sequence."""
    return {"op": "sparse", "B": B, "g": g, "H": H, "d": d, "page": page, "ctx": ctx, "top_k": top_k}


def listed():
    return [
        # one sequence's step of two tokens: the smallest call, all latency
        {"name": "rope step", **rope_case(2, 16, 16, 128, 128, "half", "none", True, "bf16", 131072)},
        # a whole prefill layer before the indexer, norms of each head included
        {"name": "rope prefill", **rope_case(8192, 16, 16, 128, 128, "half", "none", True, "bf16", 8192)},
        # part of the head, interleaved, scaled for long contexts, far positions, fp32 projections, an odd length
        {"name": "rope long partial", **rope_case(30011, 32, 4, 64, 32, "interleaved", "yarn", False, "fp32", 1000003)},
        # a batch's decode step: two tokens of each of 64 sequences, queries turned in the same call
        {"name": "append step", **append_case(64, 2, False, 16, 16, 128, 16, 1024, 128, "half", True, True, "bf16")},
        # chunked prefill of a ragged batch, fewer key heads than query heads
        {"name": "append chunk", **append_case(5, 4001, True, 32, 8, 128, 64, 4096, 128, "half", True, True, "bf16")},
        # a few short ragged chunks in small pages, queries that do not see their own key, three query heads to a key head
        {"name": "attend small", **attend_case(3, 70, True, 12, 4, 64, 16, 700, False)},
        # decode of a few long sequences, as many key heads as query heads
        {"name": "attend long step", **attend_case(4, 2, False, 16, 16, 128, 64, 65536, True)},
        # decode of a full batch, four query heads to a key head
        {"name": "attend batch step", **attend_case(64, 1, False, 32, 8, 128, 16, 8192, True)},
        # a layer's prefill from nothing
        {"name": "attend prefill", **attend_case(1, 8192, False, 16, 16, 128, 128, 0, True)},
        # a chunk of new tokens over a long cached context
        {"name": "attend chunk", **attend_case(1, 2048, False, 32, 8, 128, 64, 16384, True)},
        # index rows of the small workload: one sequence's step
        {"name": "sparse small", **sparse_case(1, 2, 8, 64, 16, 1024, 64)},
        # index rows of a decode batch's step
        {"name": "sparse step", **sparse_case(32, 2, 16, 128, 16, 16384, 2048)},
    ]


def between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0.0, "flops": 0.0})
        m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    op = rng.choice(["rope", "append", "attend", "attend", "sparse"])
    while True:
        d = rng.choice([64, 128])
        page = rng.choice([1, 8, 16, 32, 64, 128, 256])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 3, 4, 5, 8])
        rot = rng.choice([d, d, d // 2, d // 4, 48])
        layout = rng.choice(["half", "interleaved"])
        norm = rng.random() < 0.5
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op == "rope":
            T = between(rng, 1, 30011)
            c = rope_case(T, Hq, Hk, d, rot, layout, rng.choice(["none", "linear", "yarn"]), norm, dtype,
                          T + between(rng, 1, 1 << 20))
        elif op == "append":
            B = between(rng, 1, 200)
            c = append_case(B, between(rng, 1, 4001), rng.random() < 0.5, rng.choice([0, Hq]), Hk, d, page,
                            between(rng, 1, 8192), rot, layout, norm, rng.random() < 0.8, dtype)
        elif op == "attend":
            B = between(rng, 1, 64)
            c = attend_case(B, between(rng, 1, 4001), rng.random() < 0.5, Hq, Hk, d, page, between(rng, 1, 65536),
                            rng.random() < 0.7)
        else:
            c = sparse_case(between(rng, 1, 64), rng.choice([1, 2, 3, 4]), Hk, d, page, between(rng, 16, 32768),
                            between(rng, 1, 2048))
        w = work(c)
        if w["bytes"] > most[op]["bytes"] or w["flops"] > most[op]["flops"]:
            continue
        if c["op"] != "rope" and cache_bytes(c) > 6e9:      # what is held, not only what a call touches
            continue
        if c["op"] == "attend" and 4.0 * c["B"] * c["Hq"] * c["new"] * (c["ctx"] + c["new"]) > 5e9:
            continue                                         # the plain form's score matrix
        return c


# ------------------------------------------------------------------ lengths, which the case alone decides
def lengths(c):
    """(rows held before the call, new rows) of each sequence."""
    r = random.Random("%s" % sorted(c.items()).__repr__() if "name" not in c else
                      "%s" % sorted((k, v) for k, v in c.items() if k != "name").__repr__())
    B, ctx = c["B"], c["ctx"]
    most = c.get("new", c.get("g", 1))
    new = [most] + [r.randint(max(1, most // 4), most) for _ in range(B - 1)] if c.get("ragged") else [most] * B
    held = [ctx] + [r.randint(ctx // 4, ctx) for _ in range(B - 1)]
    return held, new


def pages_of(c):
    held, new = lengths(c)
    return [-(-(h + n) // c["page"]) for h, n in zip(held, new)]


def cache_bytes(c):
    H = c.get("Hk", c.get("H"))
    return 2.0 * (sum(pages_of(c)) + 3) * c["page"] * H * c["d"] * 2


def pool(c):
    """Rows that a step's g index rows are drawn from, per sequence and head: neighbouring queries share most."""
    held, _ = lengths(c)
    return [min(h, c["top_k"] + (c["g"] - 1) * c["top_k"] // 4) for h in held]


def work(c):
    op, d = c["op"], c["d"]
    if op == "rope":
        H = c["Hq"] + c["Hk"]
        return {"bytes": float(c["T"]) * (H * d * (BYTES[c["dtype"]] + 2) + 4),
                "flops": float(c["T"]) * H * (3.0 * c["rot"] + (4.0 * d if c["norm"] else 0.0))}
    held, new = lengths(c)
    T = float(sum(new))
    if op == "append":
        turned, kept = c["Hq"] + c["Hk"], c["Hk"] if c["values"] else 0
        return {"bytes": T * (turned + kept) * d * (BYTES[c["dtype"]] + 2),
                "flops": T * turned * (3.0 * c["rot"] + (4.0 * d if c["norm"] else 0.0))}
    if op == "attend":
        off = 0 if c["itself"] else 1
        seen = sum(n * h + n * (n + 1) / 2.0 - off * n for h, n in zip(held, new))
        rows = float(sum(h + n - off for h, n in zip(held, new)))
        return {"bytes": rows * c["Hk"] * d * 4 + T * c["Hq"] * (d * 4 + 4), "flops": 4.0 * d * c["Hq"] * seen}
    rows = float(sum(pool(c)))
    per = float(sum(min(h, c["top_k"]) for h in held)) * c["g"]
    return {"bytes": rows * c["H"] * d * 4 + c["B"] * c["g"] * c["H"] * (c["top_k"] * 4.0 + d * 6),
            "flops": 4.0 * d * c["H"] * per}


# ------------------------------------------------------------------ inputs
def frequencies(rot, scaling):
    """(radians a position of each pair, amplitude), fp64: plain, all positions drawn in by 4, or by 8 for the slow
    pairs only (fast ones keep their rate, those between are mixed) with the amplitude that goes with it."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        where = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(BASE)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(where[0]), 0), min(math.ceil(where[1]), rot - 1)
        mix = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / 8.0 * mix + f * (1 - mix), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def heavy(gen, rows, H, d, dtype):
    """Keys: unit normal rows, 1 % of them four times as long."""
    x = torch.randn((rows, H, d), generator=gen, device=DEV, dtype=torch.float32)
    x *= torch.where(torch.rand((rows, 1, 1), generator=gen, device=DEV) < 0.01, 4.0, 1.0)
    return x.to(dtype)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    s = {"c": c}
    d = c["d"]
    if c["op"] in ("rope", "append"):
        freqs, s["amplitude"] = frequencies(c["rot"], c.get("scaling", "none"))
        s["freqs"] = freqs.to(DEV)
        t = TYPES[c["dtype"]]
        one = lambda: (1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(t)  # noqa: E731
        s["qw"], s["kw"] = (one(), one()) if c["norm"] else (None, None)
    if c["op"] == "rope":
        s["q"] = normal(gen, (c["T"], c["Hq"], d), t)
        s["k"] = heavy(gen, c["T"], c["Hk"], d, t)
        s["positions"] = torch.arange(c["far"] - c["T"], c["far"], device=DEV, dtype=torch.int32)
        return s
    held, new = lengths(c)
    B, page, H = c["B"], c["page"], c.get("Hk", c.get("H"))
    np_ = pages_of(c)
    total = sum(np_) + 3
    order = torch.randperm(total, generator=gen, device=DEV)[:sum(np_)].to(torch.int32)
    first = torch.tensor([0] + np_, device=DEV).cumsum(0)
    col = torch.arange(max(np_), device=DEV)
    s["table"] = torch.where(col[None] < torch.tensor(np_, device=DEV)[:, None],
                             order[(first[:-1, None] + col[None]).clamp(max=sum(np_) - 1)], 0).to(torch.int32)
    s["seqlens"] = torch.tensor([h + n for h, n in zip(held, new)], device=DEV, dtype=torch.int32)
    s["longest"] = max(h + n for h, n in zip(held, new))
    s["most_new"] = max(new)
    s["kpages"] = heavy(gen, total * page, H, d, torch.bfloat16).view(total, page, H, d)
    s["vpages"] = normal(gen, (total, page, H, d), torch.bfloat16)
    T = sum(new)
    cu = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["cu"] = cu if c.get("ragged") else None
    lead = (T,) if c.get("ragged") else (B, new[0])
    if c["op"] == "append":
        s["k"] = heavy(gen, T, H, d, t).view(*lead, H, d)
        s["v"] = normal(gen, (*lead, H, d), t) if c["values"] else None
        if not c["values"]:
            s["vpages"] = None
        s["q"] = normal(gen, (*lead, c["Hq"], d), t) if c["Hq"] else None
    elif c["op"] == "attend":
        s["q"] = normal(gen, (*lead, c["Hq"], d), torch.bfloat16)
    else:
        s["q"] = normal(gen, (*lead, H, d), torch.bfloat16)
        s["idx"] = index_rows(gen, c, held)
    return s


def index_rows(gen, c, held):
    """int32 [B, g, H, top_k]: each row a random part of its sequence's pool of rows, ascending, -1 behind."""
    B, g, H, k = c["B"], c["g"], c["H"], c["top_k"]
    u = pool(c)
    hb = torch.tensor(held, device=DEV)
    at = torch.rand((B, H, c["ctx"]), generator=gen, device=DEV)
    at = at.masked_fill(torch.arange(c["ctx"], device=DEV) >= hb[:, None, None], 2.0)
    some = at.topk(max(u), dim=-1, largest=False).indices                     # [B, H, max pool]
    ub = torch.tensor(u, device=DEV)
    mark = torch.rand((B, g, H, max(u)), generator=gen, device=DEV)
    mark = mark.masked_fill(torch.arange(max(u), device=DEV) >= ub[:, None, None, None], 2.0)
    n = min(k, max(u))
    low = mark.topk(n, dim=-1, largest=False)
    rows = some[:, None].expand(B, g, H, max(u)).gather(-1, low.indices)
    rows = rows.masked_fill(low.values >= 2.0, 1 << 30).sort(dim=-1).values
    rows = rows.masked_fill(rows >= 1 << 30, -1)
    return torch.nn.functional.pad(rows, (0, k - n), value=-1).to(torch.int32).contiguous()


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        return run_own(s)
    return {"rope": plain_rope, "append": plain_append, "attend": plain_attend, "sparse": plain_sparse}[c["op"]](s)


def run_own(s):
    import query_group_top_b200 as qg

    c = s["c"]
    if c["op"] == "rope":
        return qg.qk_rope(s["q"], s["k"], s["positions"], s["freqs"], layout=c["layout"], amplitude=s["amplitude"],
                          q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
    if c["op"] == "append":
        out = qg.paged_append(s["k"], s["v"], s["kpages"], s["vpages"], s["table"], s["seqlens"], cu_new=s["cu"],
                              freqs=s["freqs"], layout=c["layout"], amplitude=s["amplitude"], k_weight=s["kw"],
                              q=s["q"], q_weight=s["qw"] if c["Hq"] else None, eps=EPS)
        return s["kpages"], s["vpages"], out
    if c["op"] == "attend":
        T, Hq = s["q"].numel() // (c["Hq"] * c["d"]), c["Hq"]
        lse = torch.empty((*s["q"].shape[:-2], Hq), dtype=torch.float32, device=DEV) if T else None
        out = qg.paged_attention(s["q"], s["kpages"], s["vpages"], s["table"], s["seqlens"], s["longest"],
                                 cu_q=s["cu"], include_self=c["itself"], out_lse=lse)
        return out, lse
    return qg.sparse_attention_paged(s["q"], s["kpages"], s["vpages"], s["table"], s["seqlens"], s["idx"])


# ------------------------------------------------------------------ the plain forms
def turn(x, weight, positions, freqs, amplitude, layout):
    """x [T, H, d] in 32 bits: each head over its root mean square times `weight`, then its pairs turned."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot = 2 * freqs.numel()
    angle = positions.double()[:, None] * freqs[None]
    cos, sin = (torch.cos(angle) * amplitude).float()[:, None], (torch.sin(angle) * amplitude).float()[:, None]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def plain_rope(s):
    c = s["c"]
    how = (s["positions"], s["freqs"], s["amplitude"], c["layout"])
    return turn(s["q"], s["qw"], *how), turn(s["k"], s["kw"], *how)


def places(s, T):
    """(sequence, cache row, place in the sequence's chunk) of each of the T new tokens."""
    t = torch.arange(T, device=DEV)
    if s["cu"] is None:
        seq, i = t // s["most_new"], t % s["most_new"]
        return seq, s["seqlens"].long()[seq] - s["most_new"] + i, i
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[seq]
    return seq, s["seqlens"].long()[seq] - (cu[seq + 1] - cu[seq]) + i, i


def plain_append(s):
    c = s["c"]
    flat = lambda x: x.reshape(-1, x.shape[-2], x.shape[-1])  # noqa: E731
    k = flat(s["k"])
    seq, row, _ = places(s, k.shape[0])
    page, slot = s["table"].long()[seq, row // c["page"]], row % c["page"]
    how = (row, s["freqs"], s["amplitude"], c["layout"])
    s["kpages"][page, slot] = turn(k, s["kw"], *how)
    if s["v"] is not None:
        s["vpages"][page, slot] = flat(s["v"]).to(torch.bfloat16)
    out = None if s["q"] is None else turn(flat(s["q"]), s["qw"], *how).view(s["q"].shape)
    return s["kpages"], s["vpages"], out


def plain_attend(s):
    c = s["c"]
    Hq, Hk, d, page, S = c["Hq"], c["Hk"], c["d"], c["page"], s["longest"]
    q = s["q"].reshape(-1, Hq, d)
    T, B, N, grp = q.shape[0], c["B"], s["most_new"], Hq // Hk
    seq, row, i = places(s, T)
    npg = -(-S // page)
    at = s["table"][:, :npg].long()
    k = s["kpages"][at].view(B, npg * page, Hk, d)[:, :S].float().transpose(1, 2)        # [B, Hk, S, d]
    v = s["vpages"][at].view(B, npg * page, Hk, d)[:, :S].float().transpose(1, 2)
    qp = torch.zeros((B, N, Hq, d), device=DEV)
    qp[seq, i] = q.float() / math.sqrt(d)
    qp = qp.view(B, N, Hk, grp, d).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * grp, d)
    lim = torch.zeros((B, N), dtype=torch.long, device=DEV)                               # keys that a query sees
    lim[seq, i] = row + (1 if c["itself"] else 0)
    dark = torch.arange(S, device=DEV) >= lim.repeat_interleave(grp, 1)[:, None, :, None]
    x = (qp @ k.transpose(2, 3)).masked_fill_(dark, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x @ v) / torch.where(l > 0, l, 1.0)
    back = lambda y: y.view(B, Hk, N, grp, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, -1)[seq, i]  # noqa: E731
    return back(o).to(torch.bfloat16).view(s["q"].shape), back(m + torch.log(l)).view(s["q"].shape[:-1])


def plain_sparse(s):
    c = s["c"]
    B, H, page = c["B"], c["H"], c["page"]
    idx = s["idx"].long()                                                                 # [B, g, H, top_k]
    j = idx.clamp(min=0)
    b = torch.arange(B, device=DEV)[:, None, None, None]
    h = torch.arange(H, device=DEV)[None, None, :, None]
    at = s["table"].long()[b, j // page]
    x = (s["kpages"][at, j % page, h].float() @ (s["q"].float() / math.sqrt(c["d"]))[..., None])[..., 0]
    x = x.masked_fill(idx < 0, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = (p[..., None, :] @ s["vpages"][at, j % page, h].float())[..., 0, :]
    return o / torch.where(l > 0, l, 1.0)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        pos = [int(p) for p in (s["positions"][0], s["positions"][-1])]
        pos = torch.linspace(pos[0], pos[1], c["T"], dtype=torch.float64, device=DEV).round()
        return spun(s["q"], s["qw"], pos, s, c), spun(s["k"], s["kw"], pos, s, c)
    held, new = lengths(c)
    return {"append": exact_append, "attend": exact_attend, "sparse": exact_sparse}[c["op"]](s, c, held, new)


def spun(x, weight, pos, s, c):
    """x [T, H, d]: the pairs as complex numbers, turned by a product with amplitude * e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
    n = c["rot"]
    pair = x[..., :n].unflatten(-1, (2, n // 2)).transpose(-1, -2) if c["layout"] == "half" else \
        x[..., :n].unflatten(-1, (n // 2, 2))
    z = torch.view_as_complex(pair.contiguous())
    z = z * torch.polar(torch.full_like(pos, s["amplitude"])[:, None].expand(-1, n // 2).contiguous(),
                        torch.outer(pos, s["freqs"]))[:, None, :]
    pair = torch.view_as_real(z)
    y = pair.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else pair.flatten(-2)
    return torch.cat((y, x[..., n:]), -1)


def exact_append(s, c, held, new):
    kp = s["kpages"].double()
    vp = None if s["vpages"] is None else s["vpages"].double()
    pos = torch.cat([torch.arange(h, h + n, dtype=torch.float64, device=DEV) for h, n in zip(held, new)])
    k = spun(s["k"].reshape(-1, c["Hk"], c["d"]), s["kw"], pos, s, c)
    v = None if s["v"] is None else s["v"].reshape(k.shape).double()
    table, done = s["table"].tolist(), 0
    for b, (h, n) in enumerate(zip(held, new)):
        rows = torch.arange(h, h + n, device=DEV)
        where = torch.tensor(table[b], device=DEV)[rows // c["page"]] * c["page"] + rows % c["page"]
        kp.view(-1, c["Hk"], c["d"])[where] = k[done:done + n]
        if v is not None:
            vp.view(-1, c["Hk"], c["d"])[where] = v[done:done + n]
        done += n
    q = None if s["q"] is None else spun(s["q"].reshape(-1, c["Hq"], c["d"]), s["qw"], pos, s, c).view(s["q"].shape)
    return kp, vp, q


def exact_attend(s, c, held, new):
    Hq, Hk, d = c["Hq"], c["Hk"], c["d"]
    q = s["q"].reshape(-1, Hq, d).double()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    done = 0
    for b, (h, n) in enumerate(zip(held, new)):
        at = s["table"][b, :-(-(h + n) // c["page"])].long()
        pos = torch.arange(h, h + n, device=DEV)
        seen = torch.arange(h + n, device=DEV)[None] < (pos + (1 if c["itself"] else 0))[:, None]
        for hk in range(Hk):
            k = s["kpages"][at, :, hk].reshape(-1, d)[:h + n].double()
            v = s["vpages"][at, :, hk].reshape(-1, d)[:h + n].double()
            for hq in range(hk * (Hq // Hk), (hk + 1) * (Hq // Hk)):
                x = (q[done:done + n, hq] @ k.T * d ** -0.5).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                out[done:done + n, hq] = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[:, None]) @ v
                lse[done:done + n, hq] = z
        done += n
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def exact_sparse(s, c, held, new):
    B, g, H, d = s["q"].shape
    out = torch.empty((B, g, H, d), dtype=torch.float64, device=DEV)
    for b in range(B):
        at = s["table"][b, :-(-(held[b] + new[b]) // c["page"])].long()
        k = s["kpages"][at].reshape(-1, H, d)
        v = s["vpages"][at].reshape(-1, H, d)
        for h in range(H):
            idx = s["idx"][b, :, h].long()                                               # [g, top_k]
            x = (k[idx.clamp(min=0), h].double() * s["q"][b, :, h, None].double()).sum(-1) * d ** -0.5
            p = torch.softmax(x.masked_fill(idx < 0, -math.inf), -1)
            out[b, :, h] = (torch.nan_to_num(p)[..., None] * v[idx.clamp(min=0), h].double()).sum(-2)
    return out

"""Measured cases of the operators around a paged cache's attention: norm and rotation of queries and
keys, attention of chunks of new tokens over the pages, and verification of drafted trees.

A case is a dict of plain values. ``prepare`` makes its inputs on the GPU, ``run`` takes one pass
(``own`` false: the plain form in elementary torch operations; true: the library's calls), ``work``
counts what a pass cannot do without and ``exact`` gives the outputs in 64 bits.
"""
import math
import random

import torch

own = False
bw = None  # the package, imported by the first pass that calls it


def _chunk(name, B, Hq, Hkv, d, page, ctx, new, mixed, fused, mix):
    """B requests with up to `ctx` keys before up to `new` new tokens; mixed: ragged, most of them of one token."""
    return {"name": name, "op": "chunk", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "ctx": ctx, "new": new,
            "mixed": mixed, "fused": fused, "mix": mix}


def _rope(name, rows, Hq, Hkv, d, pairs, axes, inter, norm, fused, far):
    return {"name": name, "op": "rope", "rows": rows, "Hq": Hq, "Hkv": Hkv, "d": d, "pairs": pairs, "axes": axes,
            "inter": inter, "norm": norm, "fused": fused, "far": far}


def _verify(name, B, nodes, vocab, drawn, chain, ragged, mix):
    """Trees (or chains) of `nodes` nodes, the root among them; drawn: drafts drawn from given probabilities."""
    return {"name": name, "op": "verify", "B": B, "nodes": nodes, "vocab": vocab, "drawn": drawn, "chain": chain,
            "ragged": ragged, "mix": mix}


def listed():
    return [
        # a chat's short turn behind a short context: latency is all
        _chunk("chunk_b1_h32x8_ctx1000_n16_d128_p16", 1, 32, 8, 128, 16, 1000, 16, False, True, 1),
        # one chunk of a long document's prefill, far into the document
        _chunk("chunk_b1_h32x8_ctx65024_n512_d128_p16", 1, 32, 8, 128, 16, 65024, 512, False, False, 2),
        # two prompts of 8192 tokens with nothing before them
        _chunk("chunk_b2_h32x8_n8192_d128_p64", 2, 32, 8, 128, 64, 0, 8192, False, False, 3),
        # a server's mixed batch: requests that decode one token, others that bring prompt chunks; odd groups and pages
        _chunk("chunk_b40_h24x8_mixed9000_n700_d64_p48", 40, 24, 8, 64, 48, 9000, 700, True, True, 4),
        # head dim 256, chunks behind contexts of mixed length
        _chunk("chunk_b6_h16x4_mixed12000_n1000_d256_p32", 6, 16, 4, 256, 32, 12000, 1000, True, False, 5),
        # a decode batch: one row a request, out of the fused projection's rows
        _rope("rope_b32_h32x8_d128", 32, 32, 8, 128, 64, 1, False, True, True, 30000),
        # a prompt's rows
        _rope("rope_n16384_h32x8_d128", 16384, 32, 8, 128, 64, 1, False, True, True, 131072),
        # frames of a video: time, height and width, the three axes' frequencies in turns
        _rope("rope_n9001_h28x4_d128_axes3", 9001, 28, 4, 128, 64, 3, False, True, False, 4000),
        # one chat with a small draft tree of most probable tokens
        _verify("verify_b1_n8_v32000", 1, 8, 32000, False, False, False, 6),
        # a full batch of trees over a large vocabulary
        _verify("verify_b64_n16_v131072", 64, 16, 131072, False, False, True, 7),
        # a draft model's chains, odd vocabulary
        _verify("verify_b32_chain6_v50001_drawn", 32, 6, 50001, True, True, False, 8),
        # trees with several drafts drawn behind each node
        _verify("verify_b40_n20_v151007_drawn", 40, 20, 151007, True, False, True, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rope", "rope", "verify", "verify"])
    mix = rng.randrange(1000, 1 << 20)
    if op == "chunk":
        while True:
            Hkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.choice([64, 128, 128, 256])
            c = _chunk("", _log(rng, 1, 64), g * Hkv, Hkv, d, rng.choice([16, 16, 32, 48, 64, 128]),
                       rng.choice([0, _log(rng, 1, 100000)]), _log(rng, 1, 8192), rng.random() < 0.6, rng.random() < 0.4, mix)
            # no more cache than 8 x 65536 x 8 x 128, nor more products than the largest listed case
            pairs = c["B"] * c["new"] * (c["ctx"] + 0.5 * c["new"])
            if c["B"] * (c["ctx"] + c["new"]) * Hkv * d <= 1 << 28 and pairs * g * Hkv * d <= 2 * 8192 * 4096 * 32 * 128:
                break
    elif op == "rope":
        Hkv, g, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.choice([64, 128, 128, 256])
        most = 16384 * 40 * 128 // ((g + 1) * Hkv * d)
        pairs = rng.choice([d // 2, d // 2, d // 4, d // 8 + 1])
        c = _rope("", _log(rng, 1, min(most, 32768)), g * Hkv, Hkv, d, pairs, rng.choice([1, 1, 2, 3]), rng.random() < 0.4,
                  rng.random() < 0.7, rng.random() < 0.5, _log(rng, 100, 1000000))
    else:
        vocab, drawn = _log(rng, 1000, 200000), rng.random() < 0.5
        B = _log(rng, 1, 64)
        most = 64 * 16 * 131072 // ((2 if drawn else 1) * B * vocab)
        c = _verify("", B, _log(rng, 1, max(1, min(64, most))), vocab, drawn, rng.random() < 0.3, rng.random() < 0.5, mix)
    c.pop("name")
    return c


# ---------------------------------------------------------------- lengths (of the case alone)


def _chunk_lengths(c):
    """(keys before, new tokens) of each request; the first has the most of both."""
    r = random.Random(c["mix"])
    out = [(c["ctx"], c["new"])]
    for _ in range(c["B"] - 1):
        if not c["mixed"]:
            out.append((c["ctx"], c["new"]))
        else:
            out.append((r.randint(0, c["ctx"]), 1 if r.random() < 0.6 else r.randint(0, c["new"])))
    return out


def _verify_lengths(c):
    r = random.Random(c["mix"])
    return [c["nodes"]] + [r.randint(0, c["nodes"]) if c["ragged"] else c["nodes"] for _ in range(c["B"] - 1)]


def _parents(c):
    """Parent links: node 0 is the root, the token decided last; the others hang under one of the last few."""
    r = random.Random(c["mix"] + 1)
    return [[-1 if i == 0 else (i - 1 if c["chain"] else max(0, i - r.randint(1, 5))) for i in range(n)]
            for n in _verify_lengths(c)]


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _normal(shape, g, factor=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat, step = out.view(-1), 1 << 26
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device="cuda") * factor
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sums(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return _i32(out)


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "rope": _prepare_rope, "verify": _prepare_verify}[case["op"]](case, _gen(seed))


def _prepare_chunk(c, g):
    lengths = _chunk_lengths(c)
    Hq, Hkv, d, page = (c[k] for k in ("Hq", "Hkv", "d", "page"))
    nk, nq = [a + b for a, b in lengths], [b for _, b in lengths]
    total, columns = sum(nq), (max(nk) + page - 1) // page
    if c["fused"]:  # rows of a fused query, key and value projection
        q = _normal((total, Hq + 2 * Hkv, d), g, 1.5)[:, :Hq]
    else:
        q = _normal((total, Hq, d), g, 1.5)
    pages = sum((n + page - 1) // page for n in nk)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((c["B"], columns), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(nk):
        m = (n + page - 1) // page
        table[b, :m] = order[at:at + m]
        at += m
    return {"op": "chunk", "q": q, "k": _normal((pages, page, Hkv, d), g), "v": _normal((pages, page, Hkv, d), g), "table": table,
            "nk": _i32(nk), "cu": _sums(nq), "lengths": lengths, "most": max(nq), "page": page,
            "o": torch.zeros((total, Hq, d), dtype=torch.bfloat16, device="cuda"),
            "lse": torch.zeros((total, Hq), dtype=torch.float32, device="cuda")}


def _prepare_rope(c, g):
    n, Hq, Hkv, d, pairs = (c[k] for k in ("rows", "Hq", "Hkv", "d", "pairs"))
    if c["fused"]:
        rows = _normal((n, Hq + 2 * Hkv, d), g, 1.3)
        q, k = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
    else:
        q, k = _normal((n, Hq, d), g, 1.3), _normal((n, Hkv, d), g, 1.3)
    s = {"op": "rope", "q": q, "k": k, "inter": c["inter"], "axes": None, "qw": None, "kw": None, "eps": 1e-6,
         "freq": (10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)).float(),
         "q_out": torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda"),
         "k_out": torch.zeros((n, Hkv, d), dtype=torch.bfloat16, device="cuda")}
    if c["axes"] > 1:
        s["positions"] = torch.randint(0, c["far"], (c["axes"], n), generator=g, device="cuda").to(torch.int32)
        s["axes"] = (torch.arange(pairs, device="cuda") % c["axes"]).to(torch.int32)
    else:
        s["positions"] = torch.randint(0, c["far"], (n,), generator=g, device="cuda").to(torch.int32)
    if c["norm"]:
        s["qw"], s["kw"] = ((1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    return s


def _prepare_verify(c, g):
    B, V = c["B"], c["vocab"]
    links = _parents(c)
    lengths = [len(x) for x in links]
    total = sum(lengths)
    cu = _sums(lengths)
    p = torch.empty((total, V), dtype=torch.float32, device="cuda")
    q = torch.empty((total, V), dtype=torch.float32, device="cuda") if c["drawn"] else None
    parent = _i32([x for link in links for x in link])
    order, row_of, at = [], [], 0  # a node's place among its parent's children, and its parent's row
    for link in links:
        seen = {}
        for x in link:
            order.append(seen.get(x, 0))
            seen[x] = order[-1] + 1
            row_of.append(at + max(x, 0))
        at += len(link)
    most = max(order, default=0) + 1
    few = min(most, V)
    drafts = torch.empty((total, most), dtype=torch.int64, device="cuda")  # the first tokens drafted behind each row
    step = max(1, (1 << 25) // V)
    for lo in range(0, total, step):
        hi = min(total, lo + step)
        x = torch.randn((hi - lo, V), generator=g, device="cuda") * 2.0
        x -= torch.logsumexp(x, 1, keepdim=True)
        likely = (torch.randint(0, V, (hi - lo, 1), generator=g, device="cuda") + torch.arange(6, device="cuda") * (V // 7)) % V
        x.scatter_(1, likely, torch.tensor([1.5, 0.8, 0.0, -0.7, -1.4, -2.0], device="cuda").expand(hi - lo, 6).contiguous())
        p[lo:hi] = torch.softmax(x, 1)
        x += 0.6 * torch.randn((hi - lo, V), generator=g, device="cuda")
        if c["drawn"]:
            q[lo:hi] = torch.softmax(x, 1)
            sums = q[lo:hi].double().cumsum(1)
            u = torch.rand((hi - lo, most), generator=g, device="cuda", dtype=torch.float64) * sums[:, -1:]
            drafts[lo:hi] = torch.searchsorted(sums, u, right=True).clamp(max=V - 1)
        else:
            best = x.topk(few, 1).indices
            drafts[lo:hi, :few] = best
            drafts[lo:hi, few:] = best[:, :1]
    if total:
        tokens = drafts[torch.tensor(row_of, device="cuda"), torch.tensor(order, device="cuda")].to(torch.int32)
    else:
        tokens = _i32([])
    return {"op": "verify", "tokens": tokens, "parents": parent, "cu": cu, "nodes": c["nodes"], "p": p, "draft": q,
            "u": torch.rand(total, generator=g, device="cuda"), "w": torch.rand(B, generator=g, device="cuda")}


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"chunk": _plain_chunk, "rope": _plain_rope, "verify": _plain_verify}[s["op"]](s)


def _run_own(s):
    global bw
    if bw is None:
        import exact_attention_flashattn_gb300 as bw
    if s["op"] == "chunk":
        if "ws" not in s:
            need = bw.chunk_workspace_size(s["nk"].numel(), s["most"], s["q"].shape[1], s["k"].shape[2], s["q"].shape[2])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return bw.attn_chunk_paged(s["q"], s["k"], s["v"], s["table"], s["nk"], s["cu"], s["most"], workspace=s["ws"],
                                   out=s["o"], lse=s["lse"])
    if s["op"] == "rope":
        return bw.attn_qk_norm_rope(s["q"], s["k"], s["positions"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                                    axes=s["axes"], interleaved=s["inter"], q_out=s["q_out"], k_out=s["k_out"])
    return bw.attn_tree_verify(s["tokens"], s["parents"], s["cu"], s["p"], s["u"], s["w"], s["nodes"], draft_probs=s["draft"])


def _plain_chunk(s):
    q, page = s["q"], s["page"]
    total, Hq, d = q.shape
    Hkv = s["k"].shape[2]
    g, at = Hq // Hkv, 0
    for b, (ctx, n) in enumerate(s["lengths"]):
        if n == 0:
            continue
        nk = ctx + n
        pages = s["table"][b, :(nk + page - 1) // page].long()
        k, v = (s[x][pages].view(-1, Hkv, d)[:nk].float() for x in "kv")
        hidden = torch.arange(nk, device=q.device)[None] > torch.arange(ctx, nk, device=q.device)[:, None]
        for h in range(Hkv):
            x = q[at:at + n, h * g:h * g + g].float().transpose(0, 1) * (1.0 / math.sqrt(d))  # [g, n, d]
            x = (x @ k[:, h].T).masked_fill_(hidden, -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            l = x.sum(-1, keepdim=True)
            s["o"][at:at + n, h * g:h * g + g] = ((x @ v[:, h]) / l).transpose(0, 1).to(torch.bfloat16)
            s["lse"][at:at + n, h * g:h * g + g] = (top + l.log())[..., 0].T
        at += n
    return s["o"], s["lse"]


def _plain_rope(s):
    pos, f = s["positions"], s["freq"]
    pos = pos[:, None] if s["axes"] is None else pos[s["axes"].long()].T  # [rows, pairs] or [rows, 1]
    angle = pos.double() * f.double()  # far positions need more than 32 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    pairs = f.numel()
    for name, weight, out in (("q", "qw", "q_out"), ("k", "kw", "k_out")):
        x = s[name].float()
        if s[weight] is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s[weight].float()
        if s["inter"]:
            a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :pairs], x[..., pairs:2 * pairs]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        s[out].copy_(torch.cat([turned, x[..., 2 * pairs:]], -1))
    return s["q_out"], s["k_out"]


def _plain_verify(s):
    """All requests side by side, one draft after the other: what is left of p after the drafts refused so far is
    max(p - A q, 0) (drawn drafts), or p without their tokens. 64 bits: sums next to a border decide."""
    p, draft, cu = s["p"], s["draft"], s["cu"].long()
    B, V = cu.numel() - 1, p.shape[1]
    dev, n = p.device, cu[1:] - cu[:-1]
    total = p.shape[0]
    rows = torch.full((total,), -1, dtype=torch.int32, device=dev)
    counts = (n > 0).to(torch.int32)
    none = torch.full((B,), -1, dtype=torch.int32, device=dev)
    if total == 0:
        return rows, counts, none
    has = n > 0
    first = cu[:-1].clamp(max=total - 1)
    rows[first[has]] = first[has].to(torch.int32)
    at = torch.zeros(B, dtype=torch.long, device=dev)  # the path's last node
    A = torch.zeros(B, dtype=torch.float64, device=dev)
    S = torch.ones(B, dtype=torch.float64, device=dev)
    gone = torch.zeros((B, V), dtype=torch.bool, device=dev)  # tokens refused behind the path's last node

    def left(A):
        row = first + at
        if draft is None:
            return torch.where(gone, 0.0, p[row].double())
        return (p[row].double() - A[:, None] * draft[row].double()).clamp(min=0)

    for i in range(1, s["nodes"]):
        node = (first + i).clamp(max=total - 1)
        mine = (i < n) & (s["parents"][node].long() == at)
        t, row, u = s["tokens"][node].long(), first + at, s["u"][node].double()
        if draft is None:
            pt = torch.where(gone.gather(1, t[:, None])[:, 0], 0.0, p[row, t].double())
            take = mine & (u * S < pt)
        else:
            qt = draft[row, t].double()
            pt = (p[row, t].double() - A * qt).clamp(min=0)
            take = mine & (u * S * qt < pt)
        refuse = mine & ~take
        # refused
        if draft is None:
            S = torch.where(refuse, (S - pt).clamp(min=0), S)
            gone.scatter_(1, t[:, None], refuse[:, None] | gone.gather(1, t[:, None]))
        else:
            A = torch.where(refuse, A + S, A)
            S = torch.where(refuse, left(A).sum(1), S)
        # taken: the next node of the path, with nothing refused behind it
        at = torch.where(take, i, at)
        A, S = torch.where(take, 0.0, A), torch.where(take, 1.0, S)
        gone &= ~take[:, None]
        where = (first + counts).clamp(max=total - 1)
        rows[where] = torch.where(take, node.to(torch.int32), rows[where])
        counts = counts + take.to(torch.int32)
    r = left(A)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p[first + at].double())  # nothing left: the target's own
    sums = r.cumsum(1)
    token = (sums <= s["w"].double()[:, None] * sums[:, -1:]).sum(1).clamp(max=V - 1).to(torch.int32)
    return rows, counts, torch.where(has, token, none)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "chunk":
        Hq, Hkv, d, page = (case[k] for k in ("Hq", "Hkv", "d", "page"))
        live = [(a, n) for a, n in _chunk_lengths(case) if n > 0]  # a request without new tokens reads no cache
        total = sum(n for _, n in live)
        table = sum(4 * ((a + n + page - 1) // page) for a, n in live)
        return {"bytes": sum(a + n for a, n in live) * Hkv * d * 4 + total * Hq * (4 * d + 4) + table + 8 * case["B"],
                "flops": sum(4 * Hq * d * (n * a + n * (n + 1) // 2) for a, n in live)}
    if case["op"] == "rope":
        values = case["rows"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 4 * values + 4 * case["rows"] * case["axes"], "flops": (7 if case["norm"] else 3) * values}
    lengths = _verify_lengths(case)
    live = sum(n > 0 for n in lengths)  # one row of each distribution a request, and every node's token, link and number
    return {"bytes": live * case["vocab"] * (8 if case["drawn"] else 4) + 16 * sum(lengths) + 16 * case["B"],
            "flops": live * case["vocab"] * (4 if case["drawn"] else 2)}


# ---------------------------------------------------------------- 64 bits, from the definition


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_chunk(s) if case["op"] == "chunk" else _exact_rope(s)


def _exact_chunk(s):
    total, Hq, d = s["q"].shape
    Hkv, page = s["k"].shape[2], s["page"]
    g = Hq // Hkv
    out = torch.zeros((total, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((total, Hq), dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for b, nk in enumerate(s["nk"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        j = torch.arange(nk, device="cuda")
        where = s["table"][b].long()[j // page] * page + j % page
        for h in range(Hkv):
            k, v = (s[x].view(-1, Hkv, d)[where, h].double() for x in "kv")
            for i in range(h * g, h * g + g):
                for a in range(lo, hi, 2048):  # some rows at a time; the last row of the request sees every key
                    e = min(a + 2048, hi)
                    seen = nk - (hi - e)
                    x = s["q"][a:e, i].double() @ k[:seen].T / math.sqrt(d)
                    limit = nk - hi + torch.arange(a, e, device="cuda")
                    x = torch.where(j[None, :seen] <= limit[:, None], x, -math.inf)
                    z = torch.logsumexp(x, 1)
                    lse[a:e, i] = z
                    out[a:e, i] = torch.exp(x - z[:, None]) @ v[:seen]
    return out, lse


def _exact_rope(s):
    found = []
    pairs, n = s["freq"].numel(), s["q"].shape[0]
    for name, weight in (("q", "qw"), ("k", "kw")):
        x = s[name].double()
        if s[weight] is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * s[weight].double()
        for i in range(pairs):  # each pair as a complex number, turned by its angle
            c0, c1 = (2 * i, 2 * i + 1) if s["inter"] else (i, i + pairs)
            pos = s["positions"] if s["axes"] is None else s["positions"][int(s["axes"][i])]
            turn = torch.polar(torch.ones(n, dtype=torch.float64, device="cuda"), pos.double() * s["freq"][i].double())
            z = torch.complex(x[:, :, c0].clone(), x[:, :, c1].clone()) * turn[:, None]
            x[:, :, c0], x[:, :, c1] = z.real, z.imag
        found.append(x)
    return tuple(found)

"""Measured cases of the speculative-decoding operators: tree attention over a KV cache, tree masks
built from parent links, paged block tables and slot maps, and K/V rows appended to the pages.

A case is a dict of plain values. ``prepare`` makes its inputs on the GPU, ``run`` takes one pass
(``own`` false: the plain form in elementary torch operations; true: the library's calls), ``work``
counts what a pass cannot do without and ``exact`` gives the outputs in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False
bw = None  # the package, imported by the first pass that calls it

KEYS = ("op", "B", "Hq", "Hkv", "d", "page", "nk", "nodes", "ragged", "mix")


def _tree(name, *values):
    return dict(zip(KEYS, ("tree",) + values), name=name)


def listed():
    return [
        # one request of a chat, a short context and a small draft tree: latency is all
        _tree("tree_b1_h32x8_n1024_d128", 1, 32, 8, 128, 16, 1024, 8, False, 1),
        # a full serving batch, every request verifying a 64-node tree over 16-token pages (256 rows a KV head)
        _tree("tree_b8_h32x8_n32768_d128_p16", 8, 32, 8, 128, 16, 32768, 64, False, 2),
        # one long document in a contiguous cache, a narrow tree
        _tree("tree_b1_h64x8_n262144_d128", 1, 64, 8, 128, 0, 262144, 13, False, 3),
        # many requests of mixed age and draft length, odd group and page sizes, head dim 64
        _tree("tree_b48_h24x8_ragged9000_d64_p48", 48, 24, 8, 64, 48, 9000, 21, True, 4),
        # head dim 256, contiguous caches of mixed fill
        _tree("tree_b4_h16x4_ragged12000_d256", 4, 16, 4, 256, 0, 12000, 32, True, 5),
        # the masks and positions of one verification step, and of a large batch of wide trees
        {"name": "mask_b8_n64", "op": "mask", "B": 8, "nodes": 64, "ragged": False, "mix": 6},
        {"name": "mask_b256_ragged250", "op": "mask", "B": 256, "nodes": 250, "ragged": True, "mix": 7},
        # block tables and slots of a decode batch of drafts, and of a large batch with prompt chunks among it
        {"name": "plan_b16_drafts", "op": "plan", "B": 16, "page": 16, "nk": 4096, "new": 64, "chunks": 0, "mix": 8},
        {"name": "plan_b1500_chunks", "op": "plan", "B": 1500, "page": 16, "nk": 9000, "new": 5, "chunks": 12, "mix": 9},
        # the accepted nodes of a verification step, gathered from the drafts
        {"name": "append_b8_accepted_d128", "op": "append", "tokens": 512, "Hkv": 8, "d": 128, "page": 16,
         "fp8": False, "gather": True, "fused": 0, "mix": 10},
        # a prompt's keys and values out of a fused projection's rows, into bf16 pages
        {"name": "append_prompt32768_d128", "op": "append", "tokens": 32768, "Hkv": 8, "d": 128, "page": 16,
         "fp8": False, "gather": False, "fused": 32, "mix": 11},
        # prompt chunks quantised into E4M3 pages
        {"name": "append_prompt20001_fp8_d128", "op": "append", "tokens": 20001, "Hkv": 8, "d": 128, "page": 64,
         "fp8": True, "gather": False, "fused": 0, "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tree", "mask", "plan", "append", "append"])
    mix = rng.randrange(1000, 1 << 20)
    if op == "tree":
        B, Hkv, g = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        d, nodes = rng.choice([64, 128, 128, 256]), _log(rng, 1, 128)
        # no more cache than the largest listed case, nor more products
        most = min((8 * 32768 * 8 * 128) // (B * Hkv * d), (8 * 32768 * 32 * 64 * 128) // (B * Hkv * g * nodes * d))
        nk = _log(rng, 1, max(2, min(262144, most)))
        c = _tree("", B, g * Hkv, Hkv, d, rng.choice([0, 0, 16, 16, 32, 48, 64, 128]), nk, nodes, rng.random() < 0.6, mix)
    elif op == "mask":
        c = {"op": "mask", "B": _log(rng, 1, 256), "nodes": _log(rng, 1, 250), "ragged": rng.random() < 0.5, "mix": mix}
    elif op == "plan":
        c = {"op": "plan", "B": _log(rng, 1, 1500), "page": rng.choice([16, 32, 48, 64, 128]), "nk": _log(rng, 1, 9000),
             "new": _log(rng, 1, 64), "chunks": rng.randrange(0, 8), "mix": mix}
    else:
        fp8 = rng.random() < 0.4
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        most = 32768 * 8 * 128 // (Hkv * d)
        c = {"op": "append", "tokens": _log(rng, 1, min(32768, most)), "Hkv": Hkv, "d": d, "page": rng.choice([16, 32, 48, 64, 128]),
             "fp8": fp8, "gather": rng.random() < 0.3, "fused": rng.choice([0, 4 * Hkv]), "mix": mix}
    c.pop("name", None)
    return c


# ---------------------------------------------------------------- lengths (of the case alone)


def _lengths(most, count, ragged, mix):
    """`count` lengths up to `most`; ragged ones go down to none, the first stays at `most`."""
    r = random.Random(mix)
    return [most] + [r.randint(0, most) if ragged else most for _ in range(count - 1)]


def _tree_lengths(c):
    return _lengths(c["nk"], c["B"], c["ragged"], c["mix"]), _lengths(c["nodes"], c["B"], c["ragged"], c["mix"] + 77)


def _plan_lengths(c):
    r = random.Random(c["mix"])
    nk = [r.randint(0, c["nk"]) for _ in range(c["B"])]
    new = [r.randint(0, c["new"]) for _ in range(c["B"])]
    for _ in range(min(c["chunks"], c["B"])):  # a prompt chunk in place of a draft
        new[r.randrange(c["B"])] = r.randint(512, 4096)
    new[0] = max(new[0], 1)
    spare = [r.randint(0, 2) for _ in range(c["B"])]  # pages that a request holds beyond its keys
    return nk, new, spare


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
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
    return _i32(np.concatenate([[0], np.cumsum(lengths)]).tolist())


def _parents(lengths, seed):
    """Trees in the order of their drafting: a node hangs under one of the last few before it, or under the context."""
    r, flat = np.random.default_rng(seed), []
    for n in lengths:
        back = np.minimum(r.integers(1, 9, n), np.arange(n) + 1)
        flat.append(np.arange(n) - back)  # -1: a root
    return np.concatenate(flat).astype(np.int32) if flat else np.zeros(0, np.int32)


def _ancestor_bits(lengths, parents, words):
    """int64 [nodes, words]: bit j of a node's row is set where node j is the node itself or an ancestor."""
    out, at = np.zeros((int(sum(lengths)), words), np.uint64), 0
    for n in lengths:
        for i in range(n):
            p = int(parents[at + i])
            if p >= 0:
                out[at + i] = out[at + p]
            out[at + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        at += n
    return torch.from_numpy(out.view(np.int64)).cuda()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "tree":
        nk, nodes = _tree_lengths(case)
        B, Hq, Hkv, d, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "page"))
        total, words = sum(nodes), (case["nodes"] + 63) // 64
        parents = _parents(nodes, seed)
        s = {"op": op, "q": _normal((total, Hq, d), g, 2.0), "k_new": _normal((total, Hkv, d), g), "v_new": _normal((total, Hkv, d), g),
             "nk": _i32(nk), "cu": _sums(nodes), "mask": _ancestor_bits(nodes, parents, words), "parents": parents,
             "nodes": case["nodes"], "page": page, "o": torch.zeros((total, Hq, d), dtype=torch.bfloat16, device="cuda"),
             "lse": torch.zeros((total, Hq), dtype=torch.float32, device="cuda")}
        if page:
            columns = (case["nk"] + page - 1) // page
            s["k"], s["v"] = (_normal((B * columns, page, Hkv, d), g) for _ in range(2))
            s["table"] = torch.randperm(B * columns, generator=g, device="cuda").to(torch.int32).view(B, columns)
        else:
            s["k"], s["v"] = (_normal((B, Hkv, case["nk"], d), g) for _ in range(2))
        return s
    if op == "mask":
        nodes = _lengths(case["nodes"], case["B"], case["ragged"], case["mix"])
        base = torch.randint(0, 30000, (case["B"],), generator=g, device="cuda").to(torch.int32)
        return {"op": op, "parents": torch.from_numpy(_parents(nodes, seed)).cuda(), "cu": _sums(nodes), "nodes": case["nodes"], "nk": base}
    if op == "plan":
        nk, new, spare = _plan_lengths(case)
        page, held = case["page"], [(n + case["page"] - 1) // case["page"] + x for n, x in zip(nk, spare)]
        columns = max(max(held), max((n + m + page - 1) // page for n, m in zip(nk, new)))
        need = sum(max(0, (n + m + page - 1) // page - h) for n, m, h in zip(nk, new, held))
        pool = torch.randperm(sum(held) + need + 100, generator=g, device="cuda").to(torch.int32)
        inside = torch.arange(columns, device="cuda")[None] < _i32(held)[:, None]
        table = torch.full((case["B"], columns), -1, dtype=torch.int32, device="cuda")
        table[inside] = pool[:sum(held)]
        free = pool[sum(held):].clone()
        return {"op": op, "nk": _i32(nk), "new": _i32(new), "table": table, "held": _i32(held), "free": free,
                "count": _i32([free.numel()]), "page": page, "tokens": sum(new) + 3}
    tokens, Hkv, d, page = (case[k] for k in ("tokens", "Hkv", "d", "page"))
    n = tokens // 4 + 1 if case["gather"] else tokens  # a quarter of the drafts is accepted
    pages = (n + page - 1) // page + 8
    if case["fused"]:  # rows of a fused query, key and value projection
        rows = _normal((tokens, case["fused"] + 2 * Hkv, d), g)
        k_new, v_new = rows[:, case["fused"]:case["fused"] + Hkv], rows[:, case["fused"] + Hkv:]
    else:
        k_new, v_new = _normal((tokens, Hkv, d), g), _normal((tokens, Hkv, d), g)
    order = torch.randperm(pages, generator=g, device="cuda")
    first = int(seed) % page  # the request's last page is partly full
    at = torch.arange(first, first + n, device="cuda")
    slots = (order[at // page] * page + at % page).to(torch.int32)
    slots[torch.rand(n, generator=g, device="cuda") < 0.02] = -1  # padding
    s = {"op": op, "k_new": k_new, "v_new": v_new, "slots": slots, "rows": None, "fp8": case["fp8"]}
    if case["gather"]:
        s["rows"] = torch.randperm(tokens, generator=g, device="cuda")[:n].sort().values.to(torch.int32)
    if case["fp8"]:
        s["k"], s["v"] = (torch.randint(0, 120, (pages, page, Hkv, d), generator=g, device="cuda").to(torch.uint8) for _ in range(2))
        s["ks"], s["vs"] = ((0.5 + 1.5 * torch.rand((Hkv, d), generator=g, device="cuda")) * (4.5 / 448) for _ in range(2))
    else:
        s["k"], s["v"] = _normal((pages, page, Hkv, d), g), _normal((pages, page, Hkv, d), g)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"tree": _plain_tree, "mask": _plain_mask, "plan": _plain_plan, "append": _plain_append}[s["op"]](s)


def _run_own(s):
    global bw
    if bw is None:
        import exact_attention_flashattn_gb300 as bw
    if s["op"] == "tree":
        if "ws" not in s:
            need = bw.tree_workspace_size(s["nk"].numel(), s["nodes"], s["q"].shape[1], s["k_new"].shape[1], s["q"].shape[2])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        if s["page"]:
            return bw.attn_tree_paged(s["q"], s["k"], s["v"], s["table"], s["k_new"], s["v_new"], s["nk"], s["cu"], s["mask"], s["nodes"],
                                      workspace=s["ws"], out=s["o"], lse=s["lse"])
        return bw.attn_tree(s["q"], s["k"], s["v"], s["k_new"], s["v_new"], s["nk"], s["cu"], s["mask"], s["nodes"],
                            workspace=s["ws"], out=s["o"], lse=s["lse"])
    if s["op"] == "mask":
        return bw.attn_tree_mask(s["parents"], s["cu"], s["nodes"], nk=s["nk"])
    if s["op"] == "plan":
        got = bw.kv_plan_paged(s["nk"], s["new"], s["table"], s["held"], s["free"], s["count"], s["page"], s["tokens"])
        return (s["table"],) + tuple(got)
    if s["fp8"]:
        k, v = bw.kv_append_paged_fp8(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"], s["ks"], s["vs"], rows=s["rows"])
        return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return bw.kv_append_paged(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"], rows=s["rows"])


def _plain_tree(s):
    q, cu, nk, N = s["q"], s["cu"].long(), s["nk"].long(), s["nodes"]
    total, Hq, d = q.shape
    B, Hkv = nk.numel(), s["k_new"].shape[1]
    g = Hq // Hkv
    if s["page"]:
        k, v = (s[x][s["table"].long()].reshape(B, -1, Hkv, d).transpose(1, 2).float() for x in "kv")
    else:
        k, v = s["k"].float(), s["v"].float()
    node = torch.arange(N, device=q.device)
    real = node[None] < (cu[1:] - cu[:-1])[:, None]  # [B, N]
    at = (cu[:-1, None] + node[None]).clamp(max=total - 1)
    qs = q[at].float().view(B, N, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * N, d) * (1.0 / math.sqrt(d))
    kn, vn = (s[x][at].float().transpose(1, 2) for x in ("k_new", "v_new"))  # [B, Hkv, N, d]
    # scores against the context, then against the drafts that the node's bits show
    old = torch.arange(k.shape[2], device=q.device)[None] < nk[:, None]
    bits = (s["mask"][at][:, :, node // 64] >> (node % 64)) & 1  # [B, N, N]
    seen = (bits == 1) & real[:, None, :] & real[:, :, None]
    sc = (qs @ k.transpose(2, 3)).masked_fill(~old[:, None, None, :], -math.inf)
    sn = (qs @ kn.transpose(2, 3)).view(B, Hkv, g, N, N).masked_fill(~seen[:, None, None], -math.inf).view(B, Hkv, g * N, N)
    top = torch.maximum(sc.amax(-1, keepdim=True), sn.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    pc, pn = (sc - top).exp_(), (sn - top).exp_()
    l = pc.sum(-1, keepdim=True) + pn.sum(-1, keepdim=True)
    o = (pc @ v + pn @ vn) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.view(B, Hkv, g, N, d).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, d)
    lse = (top + l.log()).view(B, Hkv, g, N).permute(0, 3, 1, 2).reshape(B, N, Hq)
    s["o"][at[real]] = o[real].to(torch.bfloat16)
    s["lse"][at[real]] = lse[real]
    return s["o"], s["lse"]


def _plain_mask(s):
    parents, cu, N = s["parents"], s["cu"].long(), s["nodes"]
    node = torch.arange(N, device=parents.device)
    real = node[None] < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + node[None]).clamp(max=parents.numel() - 1)
    up = torch.where(real, parents[at].long(), -1)
    A = ((node[None, None, :] == up[:, :, None]) | (node[None, None, :] == node[None, :, None])).float()
    for _ in range(max(1, (N - 1).bit_length())):  # links of up to 1, 2, 4, ... steps
        A = ((A @ A) > 0).float()
    words = (N + 63) // 64
    bits = torch.nn.functional.pad(A.long(), (0, 64 * words - N)).view(A.shape[0], N, words, 64)
    mask = (bits << torch.arange(64, device=parents.device)).sum(-1)
    positions = s["nk"].long()[:, None] + A.sum(-1).long() - 1
    return mask[real], positions[real].to(torch.int32)


def _plain_plan(s):
    nk, new, held, P = s["nk"].long(), s["new"].long(), s["held"].long(), s["page"]
    after = nk + new
    need = ((after + P - 1) // P - held).clamp(min=0)
    first = need.cumsum(0) - need
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    column = torch.arange(s["table"].shape[1], device=nk.device)[None]
    taken = (column >= held[:, None]) & (column < (held + need)[:, None])
    place = s["count"].long() - 1 - (first[:, None] + column - held[:, None])
    table = torch.where(taken, s["free"].long()[place.clamp(0, s["free"].numel() - 1)], s["table"].long())
    token = torch.arange(s["tokens"], device=nk.device)
    b = torch.searchsorted(cu[1:].contiguous(), token, right=True).clamp(max=nk.numel() - 1)
    at = (nk[b] + token - cu[b]).clamp(max=table.shape[1] * P - 1)
    slots = torch.where(token < cu[-1], table[b, at // P] * P + at % P, -1)
    return tuple(x.to(torch.int32) for x in (table, after, held + need, cu, slots, s["count"].long() - need.sum()))


def _plain_e4m3(x):
    """The E4M3 value nearest to x (ties to the even code), at most 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _plain_append(s):
    kept = s["slots"] >= 0
    to = s["slots"][kept].long()
    src = s["rows"][kept].long() if s["rows"] is not None else kept.nonzero()[:, 0]
    for name, new, scale in (("k", "k_new", "ks"), ("v", "v_new", "vs")):
        pages, rows = s[name], s[new][src]
        if s["fp8"]:  # a quotient next to a border between two codes needs more than 32 bits
            rows = _plain_e4m3(rows.double() / s[scale].double()).to(torch.float8_e4m3fn).view(torch.uint8)
        pages.view((-1,) + tuple(pages.shape[2:]))[to] = rows
    if s["fp8"]:
        return s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    return s["k"], s["v"]


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "tree":
        nk, nodes = _tree_lengths(case)
        Hq, Hkv, d, page = (case[k] for k in ("Hq", "Hkv", "d", "page"))
        total = sum(nodes)
        live = [(n, m) for n, m in zip(nk, nodes) if m > 0]  # a request without drafts reads no cache
        keys = sum(n + m for n, m in live)
        table = sum(4 * ((n + page - 1) // page) for n, _ in live) if page else 0
        return {"bytes": keys * Hkv * d * 4 + total * Hq * (4 * d + 4) + total * ((case["nodes"] + 63) // 64) * 8 + table + 8 * case["B"],
                "flops": sum(4 * Hq * d * m * (n + 1) for n, m in live)}
    if op == "mask":
        total = sum(_lengths(case["nodes"], case["B"], case["ragged"], case["mix"]))
        return {"bytes": total * (8 + 8 * ((case["nodes"] + 63) // 64)) + 8 * case["B"], "flops": 0}
    if op == "plan":
        nk, new, spare = _plan_lengths(case)
        P = case["page"]
        held = [(n + P - 1) // P + x for n, x in zip(nk, spare)]
        need = sum(max(0, (n + m + P - 1) // P - h) for n, m, h in zip(nk, new, held))
        return {"bytes": 24 * case["B"] + 8 * need + 4 * sum(new) + 4 * sum((m + P - 1) // P for m in new), "flops": 0}
    n = case["tokens"] // 4 + 1 if case["gather"] else case["tokens"]
    return {"bytes": 2 * n * case["Hkv"] * case["d"] * (3 if case["fp8"] else 4) + 4 * n, "flops": 2 * n * case["Hkv"] * case["d"] if case["fp8"] else 0}


# ---------------------------------------------------------------- 64 bits, from the definition


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "append":
        return _exact_append(s)
    return None  # whole numbers


def _exact_tree(s):
    nk, cu = s["nk"].tolist(), s["cu"].tolist()
    total, Hq, d = s["q"].shape
    Hkv = s["k_new"].shape[1]
    g = Hq // Hkv
    out = torch.zeros((total, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((total, Hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(nk):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        # a node sees the whole context, itself and the nodes on its way to the root
        sees = torch.zeros((hi - lo, hi - lo), dtype=torch.bool)
        for i in range(hi - lo):
            j = i
            while j >= 0:
                sees[i, j] = True
                j = int(s["parents"][lo + j])
        sees = sees.cuda()
        for h in range(Hkv):
            if s["page"]:
                j = torch.arange(n, device="cuda")
                page, row = s["table"][b].long()[j // s["page"]], j % s["page"]
                k, v = s["k"][page, row, h], s["v"][page, row, h]
            else:
                k, v = s["k"][b, h, :n], s["v"][b, h, :n]
            k, v = (torch.cat([x, y[lo:hi, h]]).double() for x, y in ((k, s["k_new"]), (v, s["v_new"])))
            for i in range(h * g, h * g + g):
                x = s["q"][lo:hi, i].double() @ k.T / math.sqrt(d)
                x[:, n:][~sees] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[lo:hi, i] = z
                out[lo:hi, i] = torch.exp(x - z[:, None]) @ v
    return out, lse


def _exact_append(s):
    if s["fp8"]:  # every non-negative value of the format, by its code: exponent bias 7, three fraction bits
        codes = np.arange(127)
        e, f = codes >> 3, codes & 7
        values = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
        values = torch.from_numpy(values).cuda()
        between = (values[1:] + values[:-1]) / 2
    found = []
    for name, new, scale in (("k", "k_new", "ks"), ("v", "v_new", "vs")):
        flat = s[name].view((-1,) + tuple(s[name].shape[2:]))
        to = s["slots"].long()
        rows = s[new] if s["rows"] is None else s[new].index_select(0, s["rows"].long())
        if s["fp8"]:
            flat = flat.view(torch.float8_e4m3fn).double()
            x = rows.double() / s[scale].double()
            low = torch.bucketize(x.abs(), between, right=False)  # a tie goes to the lower code ...
            tie = (low < 126) & (x.abs() == between[low.clamp(max=125)]) & (low % 2 == 1)
            rows = values[low + tie.long()] * torch.sign(x)  # ... or up, to the even one
        else:
            flat = flat.double()
        spare = torch.cat([flat, flat[:1]])  # padding goes to a row of its own
        spare[torch.where(to < 0, flat.shape[0], to)] = rows.double()
        found.append(spare[:-1].view(s[name].shape))
    return tuple(found)

"""Chunks over a paged cache, norm and rotation of q and k, and verification of drafted trees on the GPU against
plain 64-bit implementations.

Tolerances, from the roundings (each at most half a step: bf16 2^-8, fp32 2^-24, relative).
Chunks: as for tree attention. With A = sum_j p_j |v_j| / l of the element and E the largest error of a row's scores,
* the products of bf16 values are exact in fp32 and d of them are summed: E <= (d + 8) 2^-24 sum_c |q_c k_c| scale
  (8 for the scale, the running maximum and the exponential);
* weights may be rounded to bf16 and shift by E in numerator and l: |dO| <= (2^-8 + 4 E) A;
* the output is rounded to bf16 once: 2^-8 (|O| + |dO|);
* LSE: E, the sum of n weights in fp32 (n 2^-24), and 2^-21 (1 + |LSE|) for its logarithm and products.
Norm and rotation, relative to |a| + |b| of a pair's normalised values:
* the norm: a sum of d squares (d 2^-24, half of it behind the root), rsqrt (2 units in the last place: 2^-22) and
  two products: (d / 2 + 6) 2^-24;
* the angle: rounded to 32 bits once (at most pi 2^-24) and its 2^-32 of a turn, and 2^-51 of itself for the
  frequency's and the reference's own rounding in 64 bits; sin and cos are off by 2 units in the last place: with
  the two products and their sum 2^-21 + 2^-51 |position frequency|;
* the output is rounded to bf16 once.
Verification: whole numbers, equal to a walk in 64 bits.
"""
import math
import threading

import numpy as np
import pytest
import torch

import exact_attention_flashattn_gb300 as bw
from exact_attention_flashattn_gb300 import build as bw_build

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    bw_build.build()
    bw.lib()
    torch.cuda.init()
    yield
    assert bw.get_status() == bw.OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sums(lengths):
    return i32([0] + [int(x) for x in np.cumsum(lengths)])


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, factor=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * factor).to(torch.bfloat16)


# ---------------------------------------------------------------- verification


def walk(tokens, parents, p, q, u, w):
    """One request in 64 bits: (path, next token)."""
    n = len(tokens)
    if n == 0:
        return [], -1
    clean = lambda x: np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)
    path, V = [0], p.shape[1]
    row = clean(p[0])
    qrow = None if q is None else clean(q[0])
    r, S, A = row.copy(), 1.0, 0.0
    for i in range(1, n):
        if not 0 <= parents[i] < i or parents[i] != path[-1] or not 0 <= tokens[i] < V:
            continue
        t = tokens[i]
        if u[i] * S * (1.0 if q is None else qrow[t]) < r[t]:
            path.append(i)
            row = clean(p[i])
            qrow = None if q is None else clean(q[i])
            r, S, A = row.copy(), 1.0, 0.0
        elif q is None:
            S = max(S - r[t], 0.0)
            r[t] = 0.0
        else:
            A += S
            r = np.maximum(row - A * qrow, 0.0)
            S = math.fsum(r)
    if not r.any():
        r = row
    if not r.any():
        return path, -1
    total = math.fsum(r)
    return path, int(np.searchsorted(np.cumsum(r), w * total, side="right"))


def check_verify(tokens, parents, lengths, p, q, u, w, max_nodes=None, pad=0, what=""):
    """The call against the walks; tensors on the GPU, `pad` rows behind the last request."""
    max_nodes = max(max(lengths, default=1), 1) if max_nodes is None else max_nodes
    acc, counts, nxt = bw.attn_tree_verify(tokens, parents, sums(lengths), p, u, w, max_nodes, draft_probs=q)
    acc, counts, nxt = acc.tolist(), counts.tolist(), nxt.tolist()
    host = [None if x is None else x.cpu().numpy() for x in (tokens, parents, p, q, u, w)]
    at = 0
    for b, n in enumerate(lengths):
        m = min(n, max_nodes)
        s = slice(at, at + m)
        path, token = walk(host[0][s], host[1][s], host[2][s], None if q is None else host[3][s], host[4][s].astype(np.float64),
                           float(host[5][b]))
        assert counts[b] == len(path), (what, b, counts[b], path)
        assert acc[at:at + n] == [at + x for x in path] + [-1] * (n - len(path)), (what, b)
        assert nxt[b] == token, (what, b, nxt[b], token)
        at += n
    assert acc[at:] == [-1] * pad, what


def trees(lengths, kind, r):
    out = []
    for n in lengths:
        for i in range(n):
            if kind == "chain":
                out.append(i - 1)
            elif kind == "star":
                out.append(0 if i else -1)
            elif kind == "any":  # roots in between, links forward and to itself
                out.append(int(r.integers(-2, n + 1)))
            else:
                out.append(int(r.integers(max(0, i - 5), i)) if i else -1)
    return out


def probs(n, V, g, sharp=3.0):
    x = torch.randn((n, V), generator=g, device="cuda") * sharp
    return torch.softmax(x, 1)


def drafted(parents, lengths, q, g):
    """Tokens drawn from (mostly likely under) the rows of the nodes' parents."""
    out, at = torch.zeros(sum(lengths), dtype=torch.long, device="cuda"), 0
    for n in lengths:
        for i in range(1, n):
            up = parents[at + i]
            out[at + i] = torch.multinomial(q[at + (up if 0 <= up < i else 0)], 1, generator=g)[0]
        at += n
    return out.to(torch.int32)


LENGTHS = [[1], [0, 8, 1, 0, 3], [16, 16], [64, 5, 33], [200]]


@pytest.mark.parametrize("V", [1, 2, 3, 31, 1000, 4097, 50001, 131072])
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_sizes(V, drawn):
    for i, lengths in enumerate(LENGTHS):
        for kind in ("tree", "chain", "star"):
            if V > 5000 and (kind != "tree" or i == 3):
                continue
            g, r = gen(17 * i + V), np.random.default_rng(V + i)
            parents = trees(lengths, kind, r)
            n = sum(lengths)
            p = probs(n, V, g)
            q = torch.softmax(torch.log(p) + 0.7 * torch.randn((n, V), generator=g, device="cuda"), 1)
            tokens = drafted(parents, lengths, q, g)
            u, w = torch.rand(n, generator=g, device="cuda"), torch.rand(len(lengths), generator=g, device="cuda")
            check_verify(tokens, i32(parents), lengths, p, q if drawn else None, u, w, what=(i, kind))


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_verify_strides_and_alignment(drawn, shift):
    # rows that lie apart by odd distances and begin anywhere; q's rows aligned otherwise than p's; NaN around them
    V, lengths = 9001, [12, 7, 1]
    n, g = sum(lengths), gen(shift)
    parents = trees(lengths, "tree", np.random.default_rng(shift))
    wide_p, wide_q = (torch.full((n, V + 5 + x), NAN, device="cuda") for x in (0, 2))
    p, q = wide_p[:, shift:shift + V], wide_q[:, 1:1 + V]
    p.copy_(probs(n, V, g))
    q.copy_(torch.softmax(torch.log(p) + torch.randn((n, V), generator=g, device="cuda"), 1))
    tokens = drafted(parents, lengths, q.contiguous(), g)
    u, w = torch.rand(n, generator=g, device="cuda"), torch.rand(3, generator=g, device="cuda")
    check_verify(tokens, i32(parents), lengths, p, q if drawn else None, u, w)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_borders(drawn):
    # dyadic probabilities: every sum is exact, and the numbers stand on the borders themselves
    V = 64
    p = torch.zeros((3, V), device="cuda")
    p[:, 5], p[:, 9], p[:, 60] = 0.5, 0.25, 0.25
    q = torch.zeros((3, V), device="cuda")
    q[:, 5], q[:, 7] = 0.75, 0.25
    tokens, parents = i32([0, 5, 7]), i32([-1, 0, 0])
    for u1 in (0.0, 0.5, 2 / 3, np.nextafter(np.float32(0.5), np.float32(0)), 0.75):
        for u2 in (0.0, 0.3):
            for w in (0.0, 0.25, 0.5, np.nextafter(np.float32(0.5), np.float32(0)), 0.75, 1.0 - 2.0 ** -24):
                check_verify(tokens, parents, [3], p, q if drawn else None, torch.tensor([0.9, u1, u2], device="cuda", dtype=torch.float32),
                             torch.tensor([w], device="cuda", dtype=torch.float32), what=(u1, u2, w))


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_odd_inputs(drawn):
    # links of any kind, tokens out of range, the same token twice, numbers that are none, rows behind the requests
    lengths, V, pad = [20, 0, 33, 7], 333, 5
    n, r = sum(lengths) + pad, np.random.default_rng(5)
    for seed in range(6):
        g = gen(seed)
        parents = trees(lengths, "any" if seed % 2 else "tree", r) + [0] * pad
        p, q = probs(n, V, g), probs(n, V, g)
        bad = torch.tensor([NAN, -1.0, -INF], device="cuda")
        for x in (p, q):
            x[torch.rand((n, V), generator=g, device="cuda") < 0.05] = bad[seed % 3]
        p[:, 3] = 1.5 if seed == 4 else p[:, 3]
        tokens = torch.randint(-2, 12, (n,), generator=g, device="cuda").to(torch.int32)
        tokens[torch.rand(n, generator=g, device="cuda") < 0.1] = V
        u, w = torch.rand(n, generator=g, device="cuda"), torch.rand(len(lengths), generator=g, device="cuda")
        u[torch.rand(n, generator=g, device="cuda") < 0.1] = NAN
        check_verify(tokens, i32(parents), lengths, p, q if drawn else None, u, w, pad=pad, what=seed)


def test_verify_numbers_of_minus_zero():
    # -0 is 0: every draft that is possible is kept, and the first possible token comes behind the path
    p = torch.zeros((2, 40), device="cuda")
    p[0, 3] = p[0, 7] = p[1, 9] = p[1, 11] = 0.5
    zeros, w = torch.tensor([-0.0, -0.0], device="cuda"), torch.tensor([-0.0], device="cuda")
    for drawn in (None, p.clone()):
        for token, path, following in ((7, [0, 1], 9), (8, [0, -1], 3)):
            acc, counts, nxt = bw.attn_tree_verify(i32([0, token]), i32([-1, 0]), i32([0, 2]), p, zeros, w, 2, draft_probs=drawn)
            # (a token that the draft's distribution does not have is refused, and p less that distribution is nothing: p itself)
            assert acc.tolist() == path and nxt.tolist() == [following]


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_values_below_the_sums_step(drawn):
    # values are summed as multiples of 2^-44: up to half of one they have no weight, and where a refusal leaves only such
    # ones the token comes from p itself; from 2^-45 on they are a whole one, and what is left is theirs
    q = torch.zeros((2, 40), device="cuda")
    q[0, 3] = 1.0
    for small, following in ((2.0 ** -60, 3), (2.0 ** -46, 3), (2.0 ** -45, 3), (1.5 * 2.0 ** -45, 7), (2.0 ** -44, 7), (2.0 ** -30, 7)):
        p = torch.zeros((2, 40), device="cuda")
        p[0, 3], p[0, 7] = 0.5, small
        acc, counts, nxt = bw.attn_tree_verify(i32([0, 3]), i32([-1, 0]), i32([0, 2]), p, torch.tensor([0.0, 0.75], device="cuda"),
                                               torch.tensor([0.3], device="cuda"), 2, draft_probs=q if drawn else None)
        assert counts.tolist() == [1] and acc.tolist() == [0, -1] and nxt.tolist() == [following], small


def test_verify_nothing_left():
    V = 40
    p = torch.zeros((4, V), device="cuda")
    p[0, 3], p[2, 7] = 0.5, 0.25  # request 0: all of p refused; request 1: no probabilities; request 2: drafts like the target
    p[2, 9] = 0.25
    tokens, parents, lengths = i32([0, 3, 1, 7]), i32([-1, 0, -1, 0]), [2, 0, 2]
    u = torch.tensor([0.0, 0.5, 0.0, NAN], device="cuda")
    w = torch.tensor([0.3, 0.3, 0.3], device="cuda")
    check_verify(tokens, parents, lengths, p, None, u, w)
    acc, counts, nxt = bw.attn_tree_verify(tokens, parents, sums(lengths), p, u, w, 2)
    assert nxt.tolist() == [3, -1, 9] and counts.tolist() == [1, 0, 1]
    check_verify(tokens, parents, lengths, p, p.clone(), u, w)  # r = max(p - p, 0)
    check_verify(i32([0]), i32([-1]), [1], torch.zeros((1, V), device="cuda"), None, u[:1], w[:1])
    # all ones: the largest sums that there are
    V = 500000
    check_verify(i32([4]), i32([9]), [1], torch.ones((1, V), device="cuda"), None, u[:1], torch.tensor([0.999999], device="cuda"))


def test_verify_limits():
    # 1024 nodes in a line and as one node's children; more nodes than max_nodes; requests without any
    for kind in ("chain", "star"):
        lengths, V = [1024, 1024], 128
        g = gen(3)
        parents = trees(lengths, kind, None)
        p = probs(2048, V, g, 0.3)
        u = torch.rand(2048, generator=g, device="cuda") * (0.01 if kind == "chain" else 1.0)
        tokens = torch.randint(0, V, (2048,), generator=g, device="cuda").to(torch.int32)
        w = torch.rand(2, generator=g, device="cuda")
        check_verify(tokens, i32(parents), lengths, p, None, u, w)
        check_verify(tokens, i32(parents), lengths, p, probs(2048, V, g, 0.3), u, w)
        check_verify(tokens, i32(parents), lengths, p, None, u, w, max_nodes=100)
    p = torch.rand((4, 10), device="cuda")
    acc, counts, nxt = bw.attn_tree_verify(i32([1, 2, 3, 4]), i32([-1, 0, 0, 0]), i32([0]), p, p[:, 0].contiguous(), p[0, :0], 3)
    assert acc.tolist() == [-1] * 4 and counts.numel() == nxt.numel() == 0
    acc, counts, nxt = bw.attn_tree_verify(i32([]), i32([]), i32([0, 0, 0]), p[:0], p[:0, 0].contiguous(), p[0, :2].contiguous(), 3)
    assert counts.tolist() == [0, 0] and nxt.tolist() == [-1, -1]


def test_verify_rows_to_31_bits():
    # 2^31 - 1 rows: behind the last request, behind the last node that is tried, of a request that may try none
    n = (1 << 31) - 1
    links = torch.zeros(n, dtype=torch.int32, device="cuda")  # every node has token 0 and hangs under the first
    p = torch.ones((n, 1), device="cuda")
    u, w = links.view(torch.float32), torch.tensor([0.5], device="cuda")  # numbers of 0
    acc = torch.empty_like(links)
    for last, most, kept in ((3, 3, 2), (n, 5, 2), (n - 200, 0, 0)):
        acc.fill_(7)
        _, counts, nxt = bw.attn_tree_verify(links, links, i32([0, last]), p, u, w, most, accepted=acc)
        assert counts.tolist() == [kept] and nxt.tolist() == [0 if kept else -1]
        assert acc[:kept].tolist() == list(range(kept)) and int(acc[kept:].max()) == -1 and int(acc[kept:].min()) == -1


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("requests, V", [(130, 9001), (250, 9001), (450, 9001), (900, 9001), (150, 140001), (260, 300001)])
def test_verify_many_requests(requests, V, drawn):
    # fewer CTAs a request; rows whose groups need more of them than the requests leave
    g, r = gen(requests), np.random.default_rng(requests)
    lengths = [3, 0, 1] + r.integers(0, 4 if V < 10000 else 2, requests - 3).tolist()
    n = sum(lengths)
    parents = trees(lengths, "star", r)
    p = probs(n, V, g)
    q = torch.softmax(torch.log(p) + 0.7 * torch.randn((n, V), generator=g, device="cuda"), 1)
    tokens = drafted(parents, lengths, q, g)
    u, w = torch.rand(n, generator=g, device="cuda"), torch.rand(requests, generator=g, device="cuda")
    check_verify(tokens, i32(parents), lengths, p, q if drawn else None, u, w)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_distribution(drawn):
    """The first token behind the root is distributed as p, whatever the drafts: each count of B trials lies within 5
    standard deviations of B p (of 13 tokens and two cases, less than one run in 10^5 would not)."""
    B, V, kids = 60000, 13, 3
    g = gen(11)
    p1, q1 = probs(1, V, g, 1.0), probs(1, V, g, 1.0)
    p, q = (x.repeat(B * (kids + 1), 1) for x in (p1, q1))
    parents = i32([-1] + [0] * kids).repeat(B)
    if drawn:
        tokens = torch.multinomial(q1[0], B * (kids + 1), replacement=True, generator=g).to(torch.int32)
    else:
        tokens = i32([0] + q1[0].topk(kids).indices.tolist()).repeat(B)
    lengths = [kids + 1] * B
    u, w = torch.rand(B * (kids + 1), generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    acc, counts, nxt = bw.attn_tree_verify(tokens, parents, sums(lengths), p, u, w, kids + 1, draft_probs=q if drawn else None)
    second = acc.view(B, -1)[:, 1]
    first = torch.where(counts > 1, tokens[second.clamp(min=0).long()], nxt)
    got = torch.bincount(first.long(), minlength=V).double().cpu()
    want = B * p1[0].double().cpu()
    assert bool(((got - want).abs() <= 5 * (want * (1 - want / B)).sqrt() + 1e-6).all()), (got, want)
    assert 0.2 < float((counts > 1).double().mean()) < 0.999


# ---------------------------------------------------------------- norm and rotation


def check_rope(Hq, Hkv, d, n, pairs, axes=1, inter=False, norm=(True, True), fused=False, inplace=False, seed=0, far=100000, eps=1e-6,
               base=10000.0):
    g = gen(seed)
    if fused:
        rows = randn((n, Hq + 2 * Hkv, d), g, 1.7)
        keep = rows.clone()
        q, k = rows[:, :Hq], rows[:, Hq:Hq + Hkv]
    else:
        q, k = randn((n, Hq, d), g, 1.7), randn((n, Hkv, d), g, 0.6)
    f = (base ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / max(pairs, 1))).float()
    pos = torch.randint(-far, far + 1, (axes, n) if axes > 1 else (n,), generator=g, device="cuda").to(torch.int32)
    ax = torch.randint(0, axes, (pairs,), generator=g, device="cuda").to(torch.int32) if axes > 1 else None
    qw, kw = (randn((d,), g) if x else None for x in norm)
    src = (q.double(), k.double())
    out = dict(q_out=q, k_out=k) if inplace else {}
    got = bw.attn_qk_norm_rope(q, k, pos, f, qw, kw, eps, ax, inter, **out)
    if inplace:
        assert got[0] is q and got[1] is k
    if fused:  # what lies beside q and k in the rows is as it was
        assert torch.equal(rows[:, Hq + Hkv:], keep[:, Hq + Hkv:]) and (inplace or torch.equal(rows, keep))
    where = pos[None] if axes == 1 else pos
    angle = torch.stack([where[0 if ax is None else int(ax[i])].double() * f[i].double() for i in range(pairs)], -1) if pairs else None
    for x, w, y in ((src[0], qw, got[0]), (src[1], kw, got[1])):
        assert y.shape == x.shape and y.dtype is torch.bfloat16
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
        ref, size = x.clone(), x.abs()
        extra = torch.zeros_like(x)
        for i in range(pairs):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + pairs)
            c, s = torch.cos(angle[:, i])[:, None], torch.sin(angle[:, i])[:, None]
            ref[..., a], ref[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
            both = x[..., a].abs() + x[..., b].abs()
            size[..., a] = size[..., b] = both
            extra[..., a] = extra[..., b] = both * (2.0 ** -21 + 2.0 ** -51 * angle[:, i].abs()[:, None])
        dv = size * (d / 2 + 6) * 2.0 ** -24 * (w is not None) + extra
        tol = dv + 2.0 ** -8 * (ref.abs() + dv) + 1e-38
        err = (y.double() - ref).abs()
        assert bool((err <= tol).all()), (Hq, Hkv, d, n, pairs, axes, inter, float((err / tol).max()))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_sizes(d, inter):
    for i, (Hq, Hkv, n) in enumerate([(1, 1, 1), (8, 2, 3), (32, 8, 40), (7, 1, 129), (5, 3, 700), (71, 1, 2), (16, 16, 5000)]):
        for pairs in (d // 2, d // 4, 8, 0, d // 8 + 1, d // 2 - 1, 1):
            check_rope(Hq, Hkv, d, n, pairs, inter=inter, fused=i % 2 == 0, seed=i)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [(True, False), (False, True), (False, False)])
def test_rope_without_norms(inter, norm):
    check_rope(6, 2, 128, 50, 64, inter=inter, norm=norm)
    check_rope(6, 2, 64, 50, 20, inter=inter, norm=norm, fused=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("axes", [2, 3, 7])
def test_rope_axes(d, axes):
    for pairs in (d // 2, d // 2 - 4, d // 8 + 3):
        check_rope(8, 2, d, 33, pairs, axes=axes, seed=axes)
        check_rope(8, 2, d, 33, pairs, axes=axes, inter=True, fused=True, seed=axes)


def test_rope_far_positions_and_in_place():
    for far in (1 << 20, (1 << 31) - 1):
        check_rope(4, 2, 128, 200, 64, far=far, base=500000.0)
        check_rope(4, 2, 64, 200, 32, far=far, inter=True)
    check_rope(4, 2, 128, 64, 64, base=1e-3)  # more than a turn per position
    for fused in (False, True):
        for inter in (False, True):
            check_rope(32, 8, 128, 300, 64, inplace=True, fused=fused, inter=inter)
            check_rope(8, 2, 64, 9, 13, inplace=True, fused=fused, inter=inter)
    # the largest and smallest rows
    g = gen(1)
    q = randn((4, 2, 128), g) * torch.tensor([1e-30, 1.0, 1e15, 0.0], device="cuda").to(torch.bfloat16)[:, None, None]
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    y, _ = bw.attn_qk_norm_rope(q, q.clone(), i32([5, 6, 7, 8]), torch.ones(64, device="cuda"), w, w)
    assert bool(torch.isfinite(y).all()) and float(y[3].abs().max()) == 0
    q[1, 1, 3] = NAN
    y, _ = bw.attn_qk_norm_rope(q, q.clone(), i32([5, 6, 7, 8]), torch.ones(64, device="cuda"), w, w)
    assert bool(torch.isnan(y[1, 1]).all()) and not bool(torch.isnan(y[0]).any() | torch.isnan(y[1, 0]).any())


@pytest.mark.parametrize("d, Hq, Hkv, pairs, inter", [(128, 4, 2, 64, False), (128, 5, 1, 17, False), (64, 7, 2, 32, True), (256, 3, 3, 128, False), (256, 4, 1, 9, False)])
def test_rope_norm_of_any_magnitude(d, Hq, Hkv, pairs, inter):
    # squares that pass 2^128 and such that vanish; heads of ordinary size beside them in a turn
    sizes = [1e-40, 1e-38, 1e-30, 1e-25, 1e-19, 1e-15, 1.0, 1e15, 1e18, 1e20, 1e30, 2e37]
    n, g = len(sizes), gen(d)
    w = randn((d,), g)
    f = (100.0 ** (-torch.arange(pairs, device="cuda") / pairs)).float()
    pos = torch.randint(0, 50, (n,), generator=g, device="cuda").to(torch.int32)
    for eps in (0.0, 1e-35, 1e-6, 1.0, 1e30):
        q, k = (torch.randn((n, h, d), generator=g, device="cuda", dtype=torch.float64).clamp(-4, 4) for h in (Hq, Hkv))
        for x in (q, k):
            for h in range(x.shape[1]):
                x[:, h] *= torch.tensor(sizes[h:] + sizes[:h], device="cuda", dtype=torch.float64)[:, None]
        q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
        q[n - 1, 0] = torch.where(q[n - 1, 0] > 0, 3e38, -3e38).to(torch.bfloat16)
        for x, y in zip((q, k), bw.attn_qk_norm_rope(q, k, pos, f, w, w, eps, interleaved=inter)):
            x = x.double()
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
            ref, size, extra = x.clone(), x.abs(), torch.zeros_like(x)
            for i in range(pairs):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + pairs)
                t = pos.double() * f[i].double()
                c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
                ref[..., a], ref[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
                size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
                extra[..., a] = extra[..., b] = size[..., a] * (2.0 ** -21 + 2.0 ** -51 * t.abs()[:, None])
            dv = size * (d / 2 + 6) * 2.0 ** -24 + extra
            tol = dv + 2.0 ** -8 * (ref.abs() + dv) + 1e-38
            err = (y.double() - ref).abs()
            bad = ~(err <= tol)
            assert not bool(bad.any()), (eps, bad.any(-1).nonzero().tolist(), y[bad][:5], ref[bad][:5])


@pytest.mark.parametrize("inter, pairs", [(False, 32), (True, 20), (False, 13)])
def test_rope_frequencies_that_are_none(inter, pairs):
    # infinities and NaN turn their own pairs into NaN, at position 0 too, and no others
    g = gen(pairs)
    q, k, w = randn((6, 3, 64), g), randn((6, 1, 64), g), randn((64,), g)
    pos, f = i32([0, 1, 5, -7, 1 << 30, 3]), torch.rand(pairs, device="cuda")
    f[1], f[2] = 3.5e-19, -3.5e-19  # one 2^-64th of a turn a position, and a part
    bad = f.clone()
    bad[0], bad[4], bad[pairs - 1] = INF, NAN, -INF
    for weight in (None, w):
        for x, y in zip(bw.attn_qk_norm_rope(q, k, pos, f, weight, weight, interleaved=inter), bw.attn_qk_norm_rope(q, k, pos, bad, weight, weight, interleaved=inter)):
            channels = [c for i in (0, 4, pairs - 1) for c in ((2 * i, 2 * i + 1) if inter else (i, i + pairs))]
            others = [c for c in range(64) if c not in channels]
            assert bool(torch.isnan(y[..., channels]).all()) and torch.equal(y[..., others], x[..., others]) and bool(torch.isfinite(x).all())


def test_rope_axes_out_of_range_and_no_rows():
    q, f = randn((5, 2, 64), gen(1)), torch.rand(32, device="cuda")
    pos = torch.randint(0, 1000, (2, 5), device="cuda").to(torch.int32)
    a = bw.attn_qk_norm_rope(q, q.clone(), pos, f, axes=i32([-5] * 16 + [9] * 16))
    b = bw.attn_qk_norm_rope(q, q.clone(), pos, f, axes=i32([0] * 16 + [1] * 16))
    assert torch.equal(a[0], b[0])
    y, z = bw.attn_qk_norm_rope(q[:0], q[:0].clone(), pos[0, :0], f)
    assert y.shape == (0, 2, 64) and z.shape == (0, 2, 64)


# ---------------------------------------------------------------- chunks over pages


class Chunk:
    """Inputs of a chunk call; pool rows of no sequence's keys hold NaN and infinities."""

    def __init__(self, Hq, Hkv, d, page, nk, nq, causal=True, seed=0, pad=2, fused=False, bound=None, factor=2.0):
        g = gen(seed)
        self.Hq, self.Hkv, self.d, self.page, self.nk, self.nq, self.causal = Hq, Hkv, d, page, nk, nq, causal
        total = sum(nq) + pad
        self.q = randn((total, Hq + 2 * Hkv, d), g, factor)[:, :Hq] if fused else randn((total, Hq, d), g, factor)
        self.keys = [(randn((n, Hkv, d), g), randn((n, Hkv, d), g)) for n in nk]
        bad = torch.tensor([NAN, INF, -INF, 3e38], device="cuda").to(torch.bfloat16)
        cols = [(n + page - 1) // page for n in nk]
        pool = sum(cols) + 5
        order = torch.randperm(pool, generator=g, device="cuda")
        self.table = torch.full((len(nk), max(max(cols), 1) + 1), 1 << 30, dtype=torch.int32, device="cuda")
        self.k = bad[torch.randint(0, 4, (pool, page, Hkv, d), generator=g, device="cuda")]
        self.v = bad[torch.randint(0, 4, (pool, page, Hkv, d), generator=g, device="cuda")]
        at = 0
        self.where = []
        for b, (n, c) in enumerate(zip(nk, cols)):
            pages = order[at:at + c]
            self.table[b, :c] = pages.to(torch.int32)
            j = torch.arange(n, device="cuda")
            self.where.append((pages[j // page], j % page))
            for dst, src in ((self.k, self.keys[b][0]), (self.v, self.keys[b][1])):
                dst[self.where[b]] = src
            at += c
        self.nk_t, self.cu, self.most = i32(nk), sums(nq), bound or max(max(nq), 1)

    def run(self, **kw):
        return bw.attn_chunk_paged(self.q, self.k, self.v, self.table, self.nk_t, self.cu, self.most, causal=self.causal, **kw)

    def check(self, o, lse, what=""):
        g, at, scale = self.Hq // self.Hkv, 0, 1 / math.sqrt(self.d)
        for b, n in enumerate(self.nq):
            lo, at = at, at + n
            if n == 0:
                continue
            nk = self.nk[b]
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(nk, device="cuda")[None]
            see = (j <= i + nk - n) if self.causal else torch.ones((n, nk), dtype=torch.bool, device="cuda")
            for h in range(self.Hkv):
                k, v = (x[:, h].double() for x in self.keys[b])
                q = self.q[lo:at, h * g:(h + 1) * g].double()
                s = (torch.einsum("ngc,jc->ngj", q, k) * scale).masked_fill(~see[:, None], -INF)
                z = torch.logsumexp(s, -1) if nk else torch.full((n, g), -INF, dtype=torch.float64, device="cuda")
                p = torch.where(see[:, None], torch.exp(s - torch.where(z == -INF, 0.0, z)[..., None]), 0.0)
                ref, A = p @ v, p @ v.abs()
                E = (self.d + 8) * 2.0 ** -24 * (torch.einsum("ngc,jc->ngj", q.abs(), k.abs()) * scale)
                E = E.masked_fill(~see[:, None], 0.0).amax(-1) if nk else torch.zeros_like(z)
                dO = (2.0 ** -8 + 4 * E)[..., None] * A
                tol = dO + 2.0 ** -8 * (ref.abs() + dO) + 1e-30
                err = (o[lo:at, h * g:(h + 1) * g].double() - ref).abs()
                assert bool((err <= tol).all()), (what, b, h, float((err / tol).max()))
                if lse is not None:
                    gl = lse[lo:at, h * g:(h + 1) * g].double()
                    empty = z == -INF
                    assert torch.equal(torch.isneginf(gl), empty), (what, b, h)
                    lt = E + nk * 2.0 ** -24 + 2.0 ** -21 * (1 + z.abs())
                    assert bool(((gl - z).abs() <= lt)[~empty].all()), (what, b, h, float((gl - z).abs()[~empty].max()))


CHUNKS = [
    # Hq, Hkv, d, page, keys, new tokens
    (8, 2, 128, 16, [300, 1, 17, 128, 9], [5, 1, 0, 128, 9]),
    (8, 2, 128, 16, [70], [1]),
    (32, 8, 128, 16, [1000, 77, 640], [300, 1, 640]),
    (4, 4, 128, 48, [500, 130], [100, 129]),          # one head a group, two row tiles
    (8, 1, 128, 64, [700], [140]),
    (6, 2, 64, 16, [333, 20, 901], [21, 20, 900]),    # group of 3: 126 rows a tile
    (10, 2, 64, 112, [257, 1], [60, 1]),              # group of 5
    (14, 2, 256, 32, [200, 45], [18, 45]),            # group of 7
    (8, 8, 256, 16, [65, 64, 400], [1, 2, 400]),
    (16, 4, 256, 1024, [1500, 3], [320, 3]),
    (71, 1, 64, 16, [100], [33]),                     # one token a tile
    (128, 1, 128, 16, [40], [20]),
    (4, 2, 64, 128, [128, 256, 384], [2, 256, 130]),  # whole tiles
    (3, 3, 128, 112, [1000, 111, 112], [4, 111, 1]),
    (4, 1, 128, 16, [5000, 1, 4000], [1, 1, 1]),      # decode
    (8, 2, 128, 16, [5, 0, 3, 200], [9, 4, 200, 300]),  # fewer keys than new tokens: rows without any
    (2, 1, 64, 16, [0, 0], [3, 200]),
    (2, 1, 256, 16, [0, 1], [3, 130]),
    (128, 1, 256, 32, [300, 40], [30, 1]),
    (8, 2, 128, 16, [5000, 900, 3000, 700], [1, 200, 2, 1]),  # decode steps among chunks, units of many CTAs
    (12, 4, 64, 16, [7000, 350, 129, 40], [1, 350, 2, 40]),
]


@pytest.mark.parametrize("i", range(len(CHUNKS)))
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_shapes(i, causal):
    c = Chunk(*CHUNKS[i], causal=causal, seed=i, fused=i % 2 == 1, bound=[None, 2000][i % 3 == 2])
    o = torch.full((c.q.shape[0], c.Hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.q.shape[0], c.Hq), 7.0, device="cuda")
    c.run(out=o, lse=lse)
    c.check(o, lse)
    assert bool((o[sum(c.nq):] == 7).all() and (lse[sum(c.nq):] == 7).all())  # rows of no sequence
    o2, none = c.run(lse=None)
    assert none is None and torch.equal(o2[:sum(c.nq)], o[:sum(c.nq)])  # the same results each time


def test_chunk_many_sequences():
    r = np.random.default_rng(0)
    nq = [int(x) for x in np.where(r.random(300) < 0.6, 1, r.integers(0, 90, 300))]
    nk = [n + int(x) for n, x in zip(nq, r.integers(0, 500, 300))]
    for d, page in ((64, 16), (128, 32)):
        c = Chunk(6, 2, d, page, nk, nq, seed=d)
        c.check(*c.run())


def test_chunk_long():
    # units that many CTAs share, prompts of several thousand tokens
    for d, Hq, Hkv, nk, nq in ((128, 8, 2, [20000], [200]), (64, 8, 2, [3000, 9000], [3000, 1]), (128, 4, 1, [2500], [2500]),
                               (256, 4, 2, [1700, 6000], [1700, 70]), (128, 16, 2, [30000], [3])):
        c = Chunk(Hq, Hkv, d, 16, nk, nq, seed=d)
        c.check(*c.run(), what=(d, nk))


@pytest.mark.parametrize("d, B", [(64, 3), (128, 70), (64, 170), (256, 40)])
def test_chunk_many_units(d, B):
    # sequences of many units among such of one or none, one and several a lane of the list
    r = np.random.default_rng(B)
    nq = [int(x) for x in r.choice([0, 1, 5, 40, 300, 700], B, p=[0.1, 0.3, 0.2, 0.2, 0.1, 0.1])]
    nq[0], nq[-1] = 700, 450
    nk = [n + int(x) for n, x in zip(nq, r.integers(0, 200, B))]
    for causal in (True, False):
        c = Chunk(16, 2, d, 32, nk, nq, causal=causal, seed=B)
        c.check(*c.run())


def test_chunk_infinities_in_later_values():
    # V rows of a token that hold infinities and NaN reach its own and later tokens only
    for d in (64, 128, 256):
        c = Chunk(4, 2, d, 16, [300, 150], [100, 150], seed=d)
        ref, _ = c.run()
        ref = ref.clone()
        for b, j, value in ((0, 250, INF), (0, 270, NAN), (1, 149, -INF), (1, 40, NAN)):
            page, row = c.where[b][0][j], c.where[b][1][j]
            c.v[page, row, 1, 5] = value
        got, _ = c.run()
        for b, at, first in ((0, 0, 50), (1, 100, 40)):
            n = c.nq[b]
            for h, ch in ((0, None), (1, 5)):
                x, y = got[at:at + n, 2 * h:2 * h + 2], ref[at:at + n, 2 * h:2 * h + 2]
                if ch is None:
                    assert torch.equal(x, y)
                else:
                    others = [e for e in range(d) if e != ch]
                    assert torch.equal(x[:, :, others], y[:, :, others]) and torch.equal(x[:first], y[:first])
        assert bool(torch.isinf(got[50:70, 2:, 5]).all()) and bool(torch.isnan(got[70:100, 2:, 5]).all())
        assert bool(torch.isnan(got[140:250, 2:, 5]).all())


SHARED = [
    # d, Hq, Hkv, page, keys, new tokens, bound
    (128, 8, 2, 16, [20000, 300], [200, 150], None),
    (128, 16, 2, 16, [30000], [3], None),
    (128, 16, 2, 64, [30000, 40], [30, 40], None),
    (128, 16, 2, 16, [30000, 9000], [3, 1], 2000),
    (64, 12, 4, 48, [25000, 7000], [250, 9], None),
    (64, 2, 2, 16, [40000], [5], 900),
    (64, 8, 2, 32, [9000], [7], None),
    (256, 4, 2, 16, [6000, 2000], [70, 300], None),
    (256, 8, 1, 64, [20000], [4], None),
]


@pytest.mark.parametrize("i", range(len(SHARED)))
def test_chunk_infinities_in_shared_units(i):
    d, Hq, Hkv, page, nk, nq, bound = SHARED[i]
    c = Chunk(Hq, Hkv, d, page, nk, nq, seed=i, bound=bound)
    ref, z = (x.clone() for x in c.run())
    c.check(ref, z)
    g, at = Hq // Hkv, 0
    # the last KV head's values of some of the new tokens, in two channels
    seen = torch.zeros_like(ref, dtype=torch.int32)  # 1: an infinity, 2: a NaN
    for b, n in enumerate(nq):
        for t, ch, value, mark in ((n // 3, 5, INF, 1), (n - 1, 5, NAN, 2), (n // 2, d - 3, -INF, 1)):
            j = nk[b] - n + t
            c.v[c.where[b][0][j], c.where[b][1][j], Hkv - 1, ch] = value
            seen[at + t:at + n, Hq - g:, ch] |= mark
        at += n
    got, z2 = c.run()
    m = sum(nq)
    assert torch.equal(z2[:m], z[:m])
    assert torch.equal(got[:m][seen[:m] == 0], ref[:m][seen[:m] == 0])
    assert bool(torch.isinf(got[:m][seen[:m] == 1]).all()) and bool(torch.isnan(got[:m][seen[:m] >= 2]).all())


def test_chunk_scale_and_caller_buffers():
    c = Chunk(8, 2, 128, 16, [300, 77], [40, 77], seed=3, pad=0)
    ref, z = c.run(scale=0.5 / math.sqrt(128))
    half = Chunk(8, 2, 128, 16, [300, 77], [40, 77], seed=3, pad=0)
    half.q = (c.q.float() * 0.5).to(torch.bfloat16)  # exact
    ws = torch.empty(bw.chunk_workspace_size(2, 77, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = half.run(workspace=ws)
    assert torch.equal(o, ref) and torch.equal(lse, z)
    half.check(o, lse)


def test_chunk_pool_past_32_bits():
    # pages beyond 2^32 bytes and 2^31 elements of the pool
    Hkv, d, page = 8, 128, 64
    pool = (1 << 31) // (page * Hkv * d) + 40
    c = Chunk(16, Hkv, d, page, [500, 90], [120, 90], seed=5)
    k, v = (torch.empty((pool, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m = c.k.shape[0]
    k[pool - m:], v[pool - m:] = c.k, c.v
    table = torch.where(c.table < m, c.table + (pool - m), c.table)
    v[table[0, 499 // page].long(), 499 % page, 3, 7] = INF  # the last token's value, looked up through the table
    o, lse = bw.attn_chunk_paged(c.q, k, v, table, c.nk_t, c.cu, c.most)
    assert bool(torch.isinf(o[119, 6:8, 7]).all())
    o[119, 6:8, 7] = 0
    c.keys[0][1][499, 3, 7] = 0
    ref, lse_ref = c.run()
    assert torch.equal(lse[:210], lse_ref[:210])
    ref[119, 6:8, 7] = 0
    assert torch.equal(o[:210], ref[:210])


@pytest.mark.parametrize("d, Hq, n", [(64, 1, 2), (128, 16, 15), (256, 1, 2)])
def test_chunk_capacity_of_31_bits(d, Hq, n):
    # 2^31 - 48 keys, one page again and again; the last tile's end is past 31 bits. All scores are 0 and all values 1, so
    # that every sum is of whole numbers; the last token's own value holds an infinity, the third to last's a NaN
    page, cols = 400, 5368709
    nk = page * cols
    assert nk == (1 << 31) - 48
    q = randn((n, Hq, d), gen(1))
    k, v = torch.zeros((2, page, 1, d), dtype=torch.bfloat16, device="cuda"), torch.ones((2, page, 1, d), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, cols), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    v[1, page - 1, 0, 5] = INF
    v[1, page - 3, 0, 6] = NAN
    o, lse = bw.attn_chunk_paged(q, k, v, table, i32([nk]), i32([0, n]), n)
    see_inf, see_nan = torch.isinf(o[:, :, 5]), torch.isnan(o[:, :, 6])
    assert bool(see_inf[-1].all()) and not bool(see_inf[:-1].any())
    assert bool(see_nan[max(n - 3, 0):].all()) and not bool(see_nan[:max(n - 3, 0)].any())
    o[-1, :, 5] = 1
    o[max(n - 3, 0):, :, 6] = 1
    assert bool((o == 1).all())
    # the logarithm and its products, as above; 304 parts at most, of whole sums, added one by one
    assert float((lse.double() - math.log(nk)).abs().max()) <= 2.0 ** -21 * 23 + 400 * 2.0 ** -24


def test_chunk_thousands_of_sequences():
    r = np.random.default_rng(1)
    nq = [1] * 3000
    nk = [int(x) for x in r.integers(1, 40, 3000)]
    c = Chunk(4, 1, 64, 16, nk, nq, seed=1)
    o, lse = c.run()
    some = [int(x) for x in r.integers(0, 3000, 40)] + [0, 2999]
    for b in some:
        k, v = (x[:, 0].double() for x in c.keys[b])
        p = torch.softmax(c.q[b].double() @ k.T / 8, 1)
        A = p @ v.abs()
        E = (64 + 8) * 2.0 ** -24 * float((c.q[b].double().abs() @ k.abs().T / 8).max())
        dO = (2.0 ** -8 + 4 * E) * A
        assert bool(((o[b].double() - p @ v).abs() <= dO + 2.0 ** -8 * ((p @ v).abs() + dO) + 1e-30).all())


def test_rope_far_apart_rows_and_odd_frequencies():
    # rows whose offsets pass 2^31 elements
    big = torch.empty((1 << 32) + (1 << 13), dtype=torch.bfloat16, device="cuda")
    g = gen(8)
    q = big.as_strided((3, 4, 128), (1 << 31, 128, 1))
    q.copy_(randn((3, 4, 128), g))
    k, w = randn((3, 2, 128), g), randn((128,), g)
    pos, f = i32([3, 70000, -5]), torch.rand(64, device="cuda")
    a = bw.attn_qk_norm_rope(q, k, pos, f, w, w)
    b = bw.attn_qk_norm_rope(q.contiguous(), k, pos, f, w, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a negative frequency turns the other way; 0 and the smallest not at all
    f = torch.tensor([0.7, 1e-45, 0.0, 1e-30] * 16, device="cuda")
    plus, minus = bw.attn_qk_norm_rope(k, k.clone(), pos, f), bw.attn_qk_norm_rope(k, k.clone(), -pos, -f)
    assert torch.equal(plus[0], minus[0]) and torch.equal(plus[0][:, :, 1::4], k[:, :, 1::4]) and torch.equal(plus[0][:, :, 2::4], k[:, :, 2::4])


def test_verify_rows_far_apart_and_caller_buffers():
    V, n = 1000, 6
    big = torch.empty(5 * (1 << 29) + V, device="cuda")
    g = gen(6)
    p = big.as_strided((n, V), (1 << 29, 1))
    p.copy_(probs(n, V, g))
    q = torch.softmax(torch.log(p) + torch.randn((n, V), generator=g, device="cuda"), 1)
    parents = trees([2, 4], "tree", np.random.default_rng(0))
    tokens = drafted(parents, [2, 4], q, g)
    u, w = torch.rand(n, generator=g, device="cuda") * 0.1, torch.rand(2, generator=g, device="cuda")
    for drawn in (None, q):
        check_verify(tokens, i32(parents), [2, 4], p, drawn, u, w)
    outs = dict(accepted=i32([7] * n), counts=i32([7, 7]), next_tokens=i32([7, 7]))
    got = bw.attn_tree_verify(tokens, i32(parents), sums([2, 4]), p, u, w, 4, **outs)
    assert got[0] is outs["accepted"] and got[1] is outs["counts"] and got[2] is outs["next_tokens"]
    want = bw.attn_tree_verify(tokens, i32(parents), sums([2, 4]), p, u, w, 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # no node may be tried: not even the roots are
    acc, counts, nxt = bw.attn_tree_verify(tokens, i32(parents), sums([2, 4]), p, u, w, 0)
    assert acc.tolist() == [-1] * n and counts.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
    with pytest.raises(ValueError):
        bw.attn_tree_verify(tokens, i32(parents), sums([2, 4]), p, u, w, 4, counts=i32([1]))
    with pytest.raises(bw.BwattnError):
        bw.attn_tree_verify(tokens, i32(parents), sums([2, 4]), p, u, w, 4, accepted=tokens)


def test_chunk_equals_tree_and_decode():
    # a line of drafts over a cache, appended and run as a chunk; one token as a decode step
    g = gen(4)
    nk, nq = [70, 333], [9, 30]
    c = Chunk(8, 2, 128, 16, nk, nq, seed=9)
    c.check(*c.run())
    one = Chunk(8, 2, 128, 16, nk, [1, 1], seed=9, pad=0)
    o, lse = one.run()
    one.check(o, lse)
    o2, lse2 = bw.attn_decode_paged(one.q, one.k, one.v, one.table.clamp(max=one.k.shape[0] - 1), one.nk_t, 2)
    one.check(o2, lse2)


# ---------------------------------------------------------------- together, graphs and streams


def serve_step(s):
    """Projection rows -> q, k -> pages -> a tree's attention -> verification -> the kept rows' slots."""
    rows, Hq, Hkv = s["rows"], s["Hq"], s["Hkv"]
    nk1, held1, cu, slots, left = bw.kv_plan_paged(s["nk"], s["nodes"], s["table"], s["held"], s["free"], s["count"], 16, rows.shape[0])
    mask, pos = bw.attn_tree_mask(s["parents"], cu, s["most"], nk=s["nk"])
    q, k = bw.attn_qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hkv], pos, s["freq"], s["w"], s["w"])
    v = rows[:, Hq + Hkv:]
    o, lse = bw.attn_tree_paged(q, s["k"], s["v"], s["table"], k, v, s["nk"], cu, mask, s["most"], workspace=s["ws"])
    acc, counts, nxt = bw.attn_tree_verify(s["tokens"], s["parents"], cu, s["p"], s["u"], s["uw"], s["most"])
    bw.kv_append_paged(k, v, slots, s["k"], s["v"], rows=acc)
    return o, acc, counts, nxt, slots, cu, pos, q, k


def make_step(seed):
    # numbers of 0: the first child of each kept node is kept
    g, Hq, Hkv, d, V = gen(seed), 8, 2, 128, 500
    nk, nodes = [40, 100, 7], [6, 1, 9]
    n = sum(nodes)
    s = {"Hq": Hq, "Hkv": Hkv, "rows": randn((n, Hq + 2 * Hkv, d), g), "nk": i32(nk), "nodes": i32(nodes), "most": 9,
         "parents": i32(trees(nodes, "tree", np.random.default_rng(seed))), "freq": 10000.0 ** (-torch.arange(64, device="cuda") / 64),
         "w": randn((d,), g), "p": probs(n, V, g), "tokens": torch.randint(0, V, (n,), generator=g, device="cuda").to(torch.int32),
         "u": torch.zeros(n, device="cuda"), "uw": torch.rand(3, generator=g, device="cuda"),
         "k": randn((40, 16, Hkv, d), g), "v": randn((40, 16, Hkv, d), g), "held": i32([3, 7, 1]), "free": torch.arange(20, 40, dtype=torch.int32, device="cuda"),
         "count": i32([20]), "ws": torch.empty(bw.tree_workspace_size(3, 9, Hq, Hkv, d), dtype=torch.uint8, device="cuda")}
    s["table"] = torch.full((3, 10), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate([3, 7, 1]):
        s["table"][b, :m] = torch.arange(at, at + m, device="cuda")
        at += m
    return s, nk, nodes


def test_step_together():
    """A verification step, then the next tokens of the kept paths as a chunk over what the step appended."""
    s, nk, nodes = make_step(3)
    o, acc, counts, nxt, slots, cu, pos, q, k = serve_step(s)
    kept, cu = counts.tolist(), cu.tolist()
    assert all(1 <= c <= n for c, n in zip(kept, nodes)) and max(kept) > 1
    for b in range(3):
        for j in range(kept[b]):
            row, slot = int(acc[cu[b] + j]), int(slots[cu[b] + j])
            assert int(pos[row]) == nk[b] + j  # a path's nodes stand behind one another
            assert torch.equal(s["k"].view(-1, 2, 128)[slot], k[row])
            assert torch.equal(s["v"].view(-1, 2, 128)[slot], s["rows"][row, 10:])
    # the path's own rows over the pages give what they gave over the tree
    total = [n + c for n, c in zip(nk, kept)]
    rows = torch.cat([acc[cu[b]:cu[b] + kept[b]] for b in range(3)]).long()
    o2, _ = bw.attn_chunk_paged(q[rows], s["k"], s["v"], s["table"], i32(total), sums(kept), max(kept))
    # both are within their rounding of the exact values: twice 2^-8 (weights, with |o| of order 1) and the output's
    assert float((o2.double() - o[rows].double()).abs().max()) <= 4 * 2.0 ** -8 * float(o.double().abs().max() + s["v"].double().abs().max())


def test_step_captured_and_replayed():
    s, _, _ = make_step(5)
    fresh = {x: s[x].clone() for x in ("k", "v", "table")}
    want = [x.clone() for x in serve_step(s)]
    pools = [s["k"].clone(), s["v"].clone()]
    for x, y in fresh.items():
        s[x].copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = serve_step(s)
    for _ in range(3):
        for x, y in fresh.items():
            s[x].copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(s["k"], pools[0]) and torch.equal(s["v"], pools[1])
    # other inputs in the same buffers
    other, _, _ = make_step(5)
    other["u"].fill_(0.9)
    s["u"].fill_(0.9)
    for x, y in fresh.items():
        s[x].copy_(y)
    graph.replay()
    want = serve_step(other)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_chunk_captured_lengths_change():
    # one capture at bounds, replayed with other lengths, tables and queries in its buffers
    c = Chunk(8, 2, 128, 16, [400, 300, 900], [200, 1, 30], seed=1, pad=0, bound=231)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = c.run()
    for seed, nk, nq in ((2, [300, 500, 31], [1, 199, 31]), (3, [900, 400, 300], [231, 0, 0]), (4, [5, 6, 7], [2, 2, 2])):
        x = Chunk(8, 2, 128, 16, nk, nq, seed=seed, pad=231 - sum(nq))
        m, cols = min(x.k.shape[0], c.k.shape[0]), min(x.table.shape[1], c.table.shape[1])
        assert sum((n + 15) // 16 for n in nk) <= c.k.shape[0] and max(nk) <= (cols - 1) * 16 + 16
        # the same keys in c's pool, page after page
        at = 0
        for b, n in enumerate(nk):
            p = (n + 15) // 16
            j = torch.arange(n, device="cuda")
            c.k[at + j // 16, j % 16], c.v[at + j // 16, j % 16] = x.keys[b]
            c.table[b, :p] = torch.arange(at, at + p, device="cuda")
            at += p
        c.q.copy_(x.q)
        c.nk_t.copy_(x.nk_t)
        c.cu.copy_(x.cu)
        graph.replay()
        torch.cuda.synchronize()
        x.check(o, lse, what=seed)


def test_streams_and_threads():
    cases = [Chunk(8, 2, 128, 16, [700, 90], [300, 1], seed=x) for x in range(4)]
    want = [c.run()[0].clone() for c in cases]
    steps = [make_step(x)[0] for x in range(4)]
    wants = [[x.clone() for x in serve_step(make_step(y)[0])] for y in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(5):
                    o, _ = cases[i].run()
                    table = steps[i]["table"].clone()
                    k, v = steps[i]["k"].clone(), steps[i]["v"].clone()
                    got = serve_step(steps[i])
                    st.synchronize()
                    n = sum(cases[i].nq)
                    assert torch.equal(o[:n], want[i][:n])
                    assert all(torch.equal(a, b) for a, b in zip(got, wants[i]))
                    for x, y in (("table", table), ("k", k), ("v", v)):
                        steps[i][x].copy_(y)
                    st.synchronize()
        except Exception as e:  # noqa: BLE001 - the thread's failure is the test's
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    # a named stream that is not the current one: the inputs are there, the outputs belong to that stream
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = cases[0]
    o, _ = c.run(stream=st)
    st.synchronize()
    assert torch.equal(o[:301], want[0][:301])


def test_refused_tensors():
    c = Chunk(8, 2, 128, 16, [50], [5], pad=0)
    with pytest.raises(ValueError):
        bw.attn_chunk_paged(c.q.float(), c.k, c.v, c.table, c.nk_t, c.cu, 5)
    with pytest.raises(ValueError):
        bw.attn_chunk_paged(c.q, c.k, c.v[:-1], c.table, c.nk_t, c.cu, 5)
    with pytest.raises(ValueError):
        bw.attn_chunk_paged(c.q.transpose(0, 1), c.k, c.v, c.table, c.nk_t, c.cu, 5)
    with pytest.raises(ValueError):
        bw.attn_chunk_paged(c.q, c.k, c.v, c.table, c.nk_t.long(), c.cu, 5)
    with pytest.raises(bw.BwattnError):
        bw.attn_chunk_paged(c.q, c.k, c.v, c.table, c.nk_t, c.cu, 5, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    f = torch.rand(64, device="cuda")
    pos = i32(range(5))
    with pytest.raises(ValueError):
        bw.attn_qk_norm_rope(c.q, c.q[:, :2], pos, f.double())
    with pytest.raises(ValueError):
        bw.attn_qk_norm_rope(c.q, c.q[:, :2], pos[:4], f)
    with pytest.raises(ValueError):
        bw.attn_qk_norm_rope(c.q, c.q[:, :2], pos, f, c.q[0, 0, :64])
    with pytest.raises(bw.BwattnError):
        bw.attn_qk_norm_rope(c.q, c.q[:, :2].contiguous(), pos, torch.rand(65, device="cuda"))
    p, u = torch.rand((5, 30), device="cuda"), torch.rand(5, device="cuda")
    with pytest.raises(ValueError):
        bw.attn_tree_verify(pos, pos, c.cu, p.T, u, u[:1], 5)
    with pytest.raises(ValueError):
        bw.attn_tree_verify(pos, pos, c.cu, p, u, u[:2], 5)
    with pytest.raises(ValueError):
        bw.attn_tree_verify(pos, pos, c.cu, p, u, u[:1], 5, draft_probs=p[:, :29])

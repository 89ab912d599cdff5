"""Speculative decoding on the GPU: tree attention, tree masks, paged plans and appends against plain
64-bit implementations.

Tolerances of tree attention, from the roundings (each at most half a step: bf16 2^-8, fp32 2^-24,
relative). With A = sum_j p_j |v_j| / l of the element and E the largest error of a row's scores:
* the products of bf16 values are exact in fp32 and d of them are summed: E <= (d + 8) 2^-24 sum_c |q_c k_c|
  scale (8 for the scale, the running maximum and the exponential);
* weights may be rounded to bf16 and shift by E in numerator and l: |dO| <= (2^-8 + 4 E) A;
* the output is rounded to bf16 once: 2^-8 (|O| + |dO|);
* LSE: E, the sum of n weights in fp32 (n 2^-24), and 2^-21 (1 + |LSE|) for its logarithm and products.
"""
import math
import threading

import numpy as np
import pytest
import torch

import exact_attention_flashattn_gb300 as bw
import oracle
from exact_attention_flashattn_gb300 import build as bw_build
from exact_attention_flashattn_gb300 import workloads as wl

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
    return i32([0] + list(np.cumsum(lengths)))


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, factor=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * factor).to(torch.bfloat16)


def pack(sees, words):
    """int64 [n, words] of a bool matrix [n, m]."""
    out = np.zeros((sees.shape[0], words), np.uint64)
    for j in range(sees.shape[1]):
        out[:, j // 64] |= sees[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def random_sees(n, kind, r):
    if kind == "tree":
        sees = np.zeros((n, n), bool)
        for i in range(n):
            p = r.integers(-1, i) if i else -1
            if p >= 0:
                sees[i] = sees[p]
            sees[i, i] = True
        return sees
    if kind == "chain":
        return np.tril(np.ones((n, n), bool))
    if kind == "none":
        return np.zeros((n, n), bool)
    if kind == "all":
        return np.ones((n, n), bool)
    sees = r.random((n, n)) < 0.3  # any mask, some rows empty
    sees[r.random(n) < 0.3] = False
    return sees


class Case:
    """Inputs of a tree call; context rows at or past nk and unused pages hold NaN and infinities."""

    def __init__(self, Hq, Hkv, d, page, nk, nodes, kind="tree", seed=0, pad=3, fused=False, bound=None, factor=2.0):
        g, r = gen(seed), np.random.default_rng(seed)
        B, total = len(nk), sum(nodes) + pad
        self.Hq, self.Hkv, self.d, self.page, self.nk, self.nodes, self.total = Hq, Hkv, d, page, nk, nodes, total
        self.max_nodes = bound or max(max(nodes), 1)
        if fused:
            rows = randn((total, Hq + 2 * Hkv, d), g)
            self.q, self.k_new, self.v_new = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
            self.q.mul_(factor)
        else:
            self.q = randn((total, Hq, d), g, factor)
            self.k_new, self.v_new = randn((total, Hkv, d), g), randn((total, Hkv, d), g)
        words = (self.max_nodes + 63) // 64
        self.sees = [random_sees(n, kind, r) for n in nodes]
        mask = np.full((total, words), -1, np.int64)  # bits past a sequence's nodes are set
        at = 0
        for n, s in zip(nodes, self.sees):
            if n:
                wide = np.ones((n, 64 * words), bool)
                wide[:, :n] = s
                mask[at:at + n] = pack(wide, words)
            at += n
        self.mask = torch.from_numpy(mask).cuda()
        self.ctx = [(randn((n, Hkv, d), g), randn((n, Hkv, d), g)) for n in nk]  # keys and values
        bad = torch.tensor([NAN, INF, -INF, 3e38], device="cuda").to(torch.bfloat16)
        if page:
            cols = [(n + page - 1) // page for n in nk]
            mp = max(max(cols), 1) + 1
            pool = sum(cols) + 5
            order = torch.randperm(pool, generator=g, device="cuda")
            self.table = torch.full((B, mp), 1 << 30, dtype=torch.int32, device="cuda")
            self.k = bad[torch.randint(0, 4, (pool, page, Hkv, d), generator=g, device="cuda")]
            self.v = bad[torch.randint(0, 4, (pool, page, Hkv, d), generator=g, device="cuda")]
            at = 0
            for b, (n, c) in enumerate(zip(nk, cols)):
                pages = order[at:at + c]
                self.table[b, :c] = pages.to(torch.int32)
                j = torch.arange(n, device="cuda")
                for dst, src in ((self.k, self.ctx[b][0]), (self.v, self.ctx[b][1])):
                    dst[pages[j // page], j % page] = src
                at += c
        else:
            self.table = None
            cap = max(max(nk), 1) + 7
            self.k = bad[torch.randint(0, 4, (B, Hkv, cap, d), generator=g, device="cuda")]
            self.v = bad[torch.randint(0, 4, (B, Hkv, cap, d), generator=g, device="cuda")]
            for b, n in enumerate(nk):
                self.k[b, :, :n], self.v[b, :, :n] = (x.transpose(0, 1) for x in self.ctx[b])
        self.nk_t, self.cu = i32(nk), sums(nodes)

    def run(self, **kw):
        if self.page:
            return bw.attn_tree_paged(self.q, self.k, self.v, self.table, self.k_new, self.v_new, self.nk_t, self.cu,
                                      self.mask, self.max_nodes, **kw)
        return bw.attn_tree(self.q, self.k, self.v, self.k_new, self.v_new, self.nk_t, self.cu, self.mask, self.max_nodes,
                            **kw)

    def check(self, o, lse, what=""):
        g, at, scale = self.Hq // self.Hkv, 0, 1 / math.sqrt(self.d)
        for b, n in enumerate(self.nodes):
            lo, at = at, at + n
            if n == 0:
                continue
            nk = self.nk[b]
            see = torch.ones((n, nk + n), dtype=torch.bool, device="cuda")
            see[:, nk:] = torch.from_numpy(self.sees[b]).cuda()
            for h in range(self.Hkv):
                k = torch.cat([self.ctx[b][0][:, h], self.k_new[lo:at, h]]).double()
                v = torch.cat([self.ctx[b][1][:, h], self.v_new[lo:at, h]]).double()
                q = self.q[lo:at, h * g:(h + 1) * g].double()
                s = torch.einsum("ngc,jc->ngj", q, k) * scale
                s = s.masked_fill(~see[:, None], -INF)
                z = torch.logsumexp(s, -1)
                p = torch.where(see[:, None], torch.exp(s - torch.where(z == -INF, 0.0, z)[..., None]), 0.0)
                ref = p @ v
                A = p @ v.abs()
                E = (self.d + 8) * 2.0 ** -24 * (torch.einsum("ngc,jc->ngj", q.abs(), k.abs()) * scale)
                E = E.masked_fill(~see[:, None], 0.0).amax(-1)
                dO = (2.0 ** -8 + 4 * E)[..., None] * A
                tol = dO + 2.0 ** -8 * (ref.abs() + dO) + 1e-30
                got = o[lo:at, h * g:(h + 1) * g].double()
                err = (got - ref).abs()
                assert bool((err <= tol).all()), (what, b, h, float((err / tol).max()))
                if lse is not None:
                    gl = lse[lo:at, h * g:(h + 1) * g].double()
                    empty = z == -INF
                    assert torch.equal(torch.isneginf(gl), empty), (what, b, h)
                    lt = E + (nk + n) * 2.0 ** -24 + 2.0 ** -21 * (1 + z.abs())
                    assert bool(((gl - z).abs() <= lt)[~empty].all()), (what, b, h, float((gl - z).abs()[~empty].max()))


SHAPES = [
    # Hq, Hkv, d, page, context lengths, nodes
    (8, 2, 128, 16, [300, 0, 17, 128], [5, 3, 0, 1]),
    (8, 2, 128, 0, [1, 129, 256], [1, 33, 64]),
    (32, 8, 128, 16, [1000, 77], [8, 31]),
    (4, 4, 128, 48, [500, 130], [100, 129]),          # one head a group, two row tiles
    (8, 1, 128, 64, [700], [40]),                     # 320 rows: several row-tile pairs
    (6, 2, 64, 16, [333, 20], [21, 43]),              # group of 3: 126 rows a tile
    (10, 2, 64, 0, [257, 1], [60, 7]),                # group of 5
    (14, 2, 256, 32, [200, 0], [18, 19]),             # group of 7
    (8, 8, 256, 0, [65, 64, 63], [1, 2, 150]),
    (16, 4, 256, 1024, [1500, 3], [32, 33]),
    (71, 1, 64, 16, [100], [3]),                      # one node a tile
    (128, 1, 128, 16, [40], [2]),
    (2, 1, 128, 0, [0, 0], [200, 1]),                 # no context
    (4, 2, 64, 128, [128, 256, 384], [2, 2, 2]),      # whole tiles
    (3, 3, 128, 112, [1000, 111, 112], [4, 1, 9]),
    (4, 1, 128, 16, [5000, 1, 4000], [1, 1, 1]),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_tree(i, kind):
    Hq, Hkv, d, page, nk, nodes = SHAPES[i]
    c = Case(Hq, Hkv, d, page, nk, nodes, kind, seed=100 + i)
    o = torch.full((c.total, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.total, Hq), 7.0, device="cuda")
    ws = torch.full((max(bw.tree_workspace_size(len(nk), c.max_nodes, Hq, Hkv, d), 16),), 255, dtype=torch.uint8, device="cuda")
    c.run(out=o, lse=lse, workspace=ws)  # over a workspace of NaN
    c.check(o, lse, SHAPES[i])
    assert bool((o[sum(nodes):] == 7).all()) and bool((lse[sum(nodes):] == 7).all())  # rows behind the last sequence
    o2, _ = c.run(lse=None)
    assert torch.equal(o2[:sum(nodes)], o[:sum(nodes)])  # no order of arrival in the result


@pytest.mark.parametrize("kind", ["none", "all", "chain"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 0), (256, 16)])
def test_tree_masks(kind, d, page):
    c = Case(8, 2, d, page, [0, 1, 200, 0], [70, 3, 130, 1], kind, seed=7)
    o, lse = c.run()
    c.check(o, lse, kind)
    if kind == "none":
        assert bool((o[:70] == 0).all()) and bool(torch.isneginf(lse[:70]).all())


def test_tree_chain_is_append():
    # drafts in one line are the packed append's causal rule
    nk, n, Hq, Hkv, d = [300, 64], [9, 20], 8, 2, 128
    c = Case(Hq, Hkv, d, 0, nk, n, "chain", seed=21, pad=0)
    o, lse = c.run()
    k = torch.cat([torch.cat([c.ctx[b][0], c.k_new[c.cu[b]:c.cu[b + 1]]]) for b in range(2)])
    v = torch.cat([torch.cat([c.ctx[b][1], c.v_new[c.cu[b]:c.cu[b + 1]]]) for b in range(2)])
    o2, lse2 = bw.attn_varlen(c.q, k, v, c.cu, sums([a + b for a, b in zip(nk, n)]), 20, 309)
    # each is within the weights' and the output's rounding of the exact result
    assert float((o.float() - o2.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())
    assert float((lse - lse2).abs().max()) <= 1e-4


@pytest.mark.parametrize("Hq,Hkv,d,page,nk,nodes", [(8, 2, 128, 16, [150, 300], [40, 6]), (12, 4, 64, 0, [90], [70]),
                                                    (4, 2, 256, 16, [70, 0], [50, 9])])
def test_tree_strided_rows(Hq, Hkv, d, page, nk, nodes):
    c = Case(Hq, Hkv, d, page, nk, nodes, "tree", seed=31, fused=True, bound=200)  # and a loose bound: 4 mask words
    assert not c.q.is_contiguous()
    o, lse = c.run()
    c.check(o, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nodes", [20, 100])
def test_tree_drafts_unseen(d, nodes):
    # what a node does not see changes no bit of its row, whatever it holds
    c = Case(8, 2, d, 16, [100], [nodes], "tree", seed=41)
    o, lse = c.run()
    for j, bad in ((nodes // 2, NAN), (nodes - 1, INF), (3, -INF)):
        for t in (c.k_new, c.v_new):
            keep = t.clone()
            t[j, :, ::3] = bad
            o2, lse2 = c.run()
            blind = ~c.sees[0][:, j]
            rows = torch.from_numpy(np.nonzero(blind)[0]).cuda()
            assert torch.equal(o2[rows], o[rows]) and torch.equal(lse2[rows], lse[rows]), (j, bad)
            seeing = torch.from_numpy(np.nonzero(~blind)[0]).cuda()
            if t is c.v_new:  # a seen value reaches its channels alone
                want = torch.isnan(o2) if bad != bad else torch.isinf(o2) & ((o2 > 0) == (bad > 0))
                assert bool(want[seeing][:, :, ::3].all())
                assert torch.equal(o2[seeing][:, :, 1::3], o[seeing][:, :, 1::3])
                assert torch.equal(lse2[:nodes], lse[:nodes])
            elif bad != bad:
                assert bool(torch.isnan(o2[seeing]).all()) and bool(torch.isnan(lse2[seeing]).all())
            t.copy_(keep)


def test_tree_nan_in_the_context_is_seen():
    c = Case(8, 2, 128, 16, [300, 300], [5, 5], "tree", seed=43)
    c.k[c.table[0, 3], 5] = NAN
    o, lse = c.run()
    assert bool(torch.isnan(o[:5]).all()) and bool(torch.isnan(lse[:5]).all())
    assert bool(torch.isfinite(o[5:10]).all()) and bool(torch.isfinite(lse[5:10]).all())


def test_tree_large_scores():
    # scores of some hundreds: the running maximum moves often and most weights vanish
    c = Case(8, 2, 128, 16, [700, 90], [30, 4], "tree", seed=47, factor=60.0)
    o, lse = c.run()
    c.check(o, lse)


def test_tree_lengths_out_of_range_are_clamped():
    c = Case(8, 2, 128, 16, [100, 60], [6, 5], "chain", seed=51, pad=0)
    o, lse = c.run()
    c.nk_t = i32([100, -5])  # a negative length: no context
    o2, _ = c.run()
    assert torch.equal(o2[:6], o[:6])
    c.nk_t = i32([100, 60])
    c.cu = i32([0, 6, 1 << 30])  # past the packed rows
    o3, _ = c.run()
    assert torch.equal(o3, o)
    c.max_nodes, c.mask = 4, c.mask[:, :1].contiguous()
    c.cu = i32([0, 6, 11])
    out = torch.full_like(o, 7.0)
    c.run(out=out)
    assert bool((out[4:6] == 7).all()) and bool((out[10:] == 7).all())  # nodes past the bound
    assert torch.equal(out[:1], o[:1])


def test_tree_graph_and_streams():
    a = Case(32, 8, 128, 16, [2000, 500], [20, 9], "tree", seed=61)
    b = Case(16, 4, 64, 0, [900], [50], "tree", seed=62)
    want = [x.run() for x in (a, b)]
    torch.cuda.synchronize()
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    ws = [torch.empty(bw.tree_workspace_size(len(x.nk), x.max_nodes, x.Hq, x.Hkv, x.d), dtype=torch.uint8, device="cuda")
          for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for x, (o, l), w in zip((a, b), outs, ws):
            x.run(out=o, lse=l, workspace=w)
    for _ in range(3):
        for o, l in outs:
            o.zero_()
        g.replay()
        # an eager call on another stream beside the replay
        with torch.cuda.stream(side):
            o3, _ = b.run()
        torch.cuda.synchronize()
        for x, (o, l), (wo, wlse) in zip((a, b), outs, want):
            n = sum(x.nodes)
            assert torch.equal(o[:n], wo[:n]) and torch.equal(l[:n], wlse[:n])
        assert torch.equal(o3[:50], want[1][0][:50])
    # the stream argument, with what the call allocates
    o4, _ = a.run(stream=side)
    side.synchronize()
    assert torch.equal(o4[:29], want[0][0][:29])
    # new lengths under the same graph
    a.nk_t.copy_(i32([1500, 500]))
    g.replay()
    torch.cuda.synchronize()
    a.ctx[0] = tuple(x[:1500] for x in a.ctx[0])
    a.nk = [1500, 500]
    a.check(outs[0][0], outs[0][1])


@pytest.mark.parametrize("Hq,Hkv,d,page,nodes", [(8, 8, 128, 0, 9), (8, 8, 128, 16, 9), (32, 8, 128, 16, 64), (8, 8, 64, 0, 9),
                                                 (32, 8, 64, 48, 40), (8, 8, 256, 0, 9), (8, 8, 256, 16, 9)])
def test_tree_runs_of_segments(Hq, Hkv, d, page, nodes):
    # every CTA walks through parts of several units of odd and even tile counts, over and over: the
    # hand-over of ring slots, buffers and streams from unit to unit
    r = np.random.default_rng(d + nodes)
    nk = [int(x) for x in r.integers(0, 6000, 24)]
    n = [int(x) for x in r.integers(1, nodes + 1, 24)]
    c = Case(Hq, Hkv, d, page, nk, n, "tree", seed=73)
    o, lse = c.run()
    c.check(o, lse)
    want = o[:sum(n)].clone()
    for _ in range(40):
        o.zero_()
        c.run(out=o)
        assert torch.equal(o[:sum(n)], want)


def test_tree_many_sequences():
    r = np.random.default_rng(5)
    nk = [int(x) for x in r.integers(0, 60, 700)]
    nodes = [int(x) for x in r.integers(0, 4, 700)]
    c = Case(4, 2, 64, 16, nk, nodes, "tree", seed=71)
    o, lse = c.run()
    c.check(o, lse)


def test_tree_pool_past_32_bits():
    # pages whose elements lie past 2^32 of the pool
    pages, page, Hkv, d = 70000, 64, 8, 128
    g = gen(81)
    k = torch.empty((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 1 << 32
    c = Case(16, Hkv, d, page, [200], [10], "tree", seed=82)
    far = torch.tensor([pages - 1, pages - 3, 65600, 2], device="cuda")
    n = torch.arange(200, device="cuda")
    slots = (far[n // page] * page + n % page).to(torch.int32)
    bw.kv_append_paged(c.ctx[0][0], c.ctx[0][1], slots, k, v)
    assert torch.equal(k[far[n // page], n % page], c.ctx[0][0])
    c.k, c.v, c.table = k, v, far[None].to(torch.int32)
    o, lse = c.run()
    c.check(o, lse)


# ------------------------------------------------------------------ masks from parents


@pytest.mark.parametrize("nodes,bound", [([1], 1), ([5, 0, 64, 65], 65), ([130, 1, 250], 256), ([1024, 1000], 1024), ([9] * 300, 40)])
def test_mask(nodes, bound):
    r = np.random.default_rng(sum(nodes))
    parents, masks, depths = [], [], []
    words = (bound + 63) // 64
    for n in nodes:
        p = np.array([r.integers(-1, i) if i else -1 for i in range(n)], np.int64).reshape(-1)
        if n > 700:
            p = np.arange(n) - 1  # one line
        sees, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
        for i in range(n):
            if p[i] >= 0:
                sees[i], depth[i] = sees[p[i]], depth[p[i]] + 1
            sees[i, i] = True
        # links that are none: negative, the node itself, a later node, far out
        roots = np.nonzero(p < 0)[0]
        p[roots] = r.choice([-1, -7, -(1 << 31), 1 << 30], len(roots))
        if len(roots):
            p[roots[0]] = roots[0]
        parents.append(p), masks.append(pack(sees, words)), depths.append(depth)
    flat = np.concatenate(parents + [np.array([5, 5])]).astype(np.int32)  # two rows of no sequence
    nk = np.arange(len(nodes)) * 10
    mask = torch.full((len(flat), words), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((len(flat),), 77, dtype=torch.int32, device="cuda")
    bw.attn_tree_mask(torch.from_numpy(flat).cuda(), sums(nodes), bound, nk=i32(nk.tolist()), mask=mask, positions=pos)
    want = np.concatenate(masks + [np.full((2, words), 77)])
    assert np.array_equal(mask.cpu().numpy(), want)
    assert np.array_equal(pos.cpu().numpy(), np.concatenate([a + b for a, b in zip(depths, nk)] + [np.array([77, 77])]))
    mask2, pos2 = bw.attn_tree_mask(torch.from_numpy(flat).cuda(), sums(nodes), bound)
    assert torch.equal(mask2[:-2], mask[:-2])
    assert np.array_equal(pos2[:-2].cpu().numpy(), np.concatenate(depths))


def test_mask_past_the_bound():
    parents = i32([-1, 0, 1, 2, 3, -1, 0])
    mask = torch.full((7, 1), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((7,), 77, dtype=torch.int32, device="cuda")
    bw.attn_tree_mask(parents, i32([0, 5, 7]), 3, mask=mask, positions=pos)
    assert mask[:, 0].tolist() == [1, 3, 7, 77, 77, 1, 3] and pos.tolist() == [0, 1, 2, 77, 77, 0, 1]


# ------------------------------------------------------------------ plans


def plan_ref(nk, new, table, held, free, count, P, tokens):
    """The plan from its definition, request by request."""
    table, count = table.copy(), min(max(count, 0), len(free))
    mp, taken, slots, cu = table.shape[1], 0, [], [0]
    held_out, nk_out = [], []
    for b in range(len(nk)):
        n, m, h = max(nk[b], 0), max(new[b], 0), min(max(held[b], 0), mp)
        need = max(0, min(-(-(n + m) // P), mp) - h)
        for i in range(need):
            table[b, h + i] = free[count - 1 - taken] if taken < count else -1
            taken += 1
        held_out.append(h + need), nk_out.append(n + m), cu.append(cu[-1] + m)
        for j in range(n, n + m):
            page = table[b, j // P] if j // P < mp else -1
            slots.append(page * P + j % P if page >= 0 else -1)
    slots = (slots + [-1] * tokens)[:tokens]
    return table, nk_out, held_out, cu, slots, count - taken


def plan_check(nk, new, table, held, free, count, P, tokens):
    want = plan_ref(nk, new, table, held, free, count, P, tokens)
    t = torch.from_numpy(table).cuda()
    args = (i32(nk), i32(new), t, i32(held), i32(free), i32([count]), P, tokens)
    for _ in range(2):  # the same inputs twice: the same plan
        got = bw.kv_plan_paged(*args)
        for x, y in zip((t,) + got, want):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1))


@pytest.mark.parametrize("B,P,most,extra", [(1, 16, 0, 0), (1, 16, 1, 5), (3, 48, 40, 0), (511, 16, 3, 1), (512, 16, 70, 0),
                                            (513, 128, 9, 700), (2000, 16, 6, 3), (40, 1024, 4000, 2)])
def test_plan(B, P, most, extra):
    r = np.random.default_rng(B + P)
    nk = r.integers(0, 300, B)
    new = r.integers(0, most + 1, B)
    held = -(-nk // P) + r.integers(0, 3, B)
    mp = int(max(held.max(), (-(-(nk + new) // P)).max(), 1))
    need = int(np.maximum(0, -(-(nk + new) // P) - held).sum())
    pages = r.permutation(int(held.sum()) + need + 7).astype(np.int32)
    table = np.full((B, mp), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        at += held[b]
    free = pages[at:].tolist()
    plan_check(nk.tolist(), new.tolist(), table, held.tolist(), free, len(free) - 2, P, int(new.sum()) + extra)


def test_plan_short_of_pages_columns_and_slots():
    P, table = 16, np.full((4, 5), -1, np.int32)
    table[0, :2], table[2, :1] = [30, 31], [32]
    args = ([20, 0, 16, 0], [40, 33, 1, 16], table, [2, 0, 1, 0])
    plan_check(*args, [1, 2, 3, 4], 4, P, 90)      # the stack runs out within a request
    plan_check(*args, [1, 2, 3, 4], 0, P, 90)
    plan_check(*args, [], 3, P, 90)                # a count past the stack
    plan_check(*args, list(range(10)), 10, P, 50)  # fewer slots than tokens
    plan_check(*args, list(range(10)), 10, P, 0)
    plan_check([20, 70, 0, 0], [100, 20, 3, 0], table, [2, 0, 1, 0], list(range(20)), 20, P, 130)  # past the columns
    plan_check([-3, 5, 0, 0], [3, -2, 0, -1], table, [2, 0, 9, -4], list(range(20)), 20, P, 5)  # clamped lengths
    plan_check([], [], np.zeros((0, 3), np.int32), [], [4, 5], 2, P, 3)  # no request


# ------------------------------------------------------------------ appends


@pytest.mark.parametrize("n,Hkv,d,page", [(1, 1, 64, 16), (7, 2, 128, 16), (200, 8, 128, 48), (33, 3, 256, 128), (5000, 4, 64, 64)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_append(n, Hkv, d, page, gather, fused, fp8):
    g = gen(n + d)
    rows_in = 2 * n + 3 if gather else n + 2
    if fused:
        x = randn((rows_in, 5 + 2 * Hkv, d), g, 3.0)
        k_new, v_new = x[:, 5:5 + Hkv], x[:, 5 + Hkv:]
    else:
        k_new, v_new = randn((rows_in, Hkv, d), g, 3.0), randn((rows_in, Hkv, d), g, 3.0)
    pages = (n + page - 1) // page + 2
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    rows = torch.randint(0, rows_in, (n,), generator=g, device="cuda").to(torch.int32) if gather else None
    if n > 4:  # skipped: outside the pool, outside the rows
        slots[1], slots[3] = -1, pages * page
        if gather:
            rows[0], rows[4] = -1, rows_in
    src = rows.long() if gather else torch.arange(n, device="cuda")
    ok = (slots >= 0) & (slots < pages * page) & (src >= 0) & (src < rows_in)
    if fp8:
        kp, vp = (torch.randint(0, 255, (pages, page, Hkv, d), generator=g, device="cuda").to(torch.uint8) for _ in range(2))
        ks, vs = (torch.rand((Hkv, d), generator=g, device="cuda") * 0.02 + 1e-3 for _ in range(2))
    else:
        kp, vp = randn((pages, page, Hkv, d), g), randn((pages, page, Hkv, d), g)
        ks = vs = None
    want = []
    for p, new, s in ((kp, k_new, ks), (vp, v_new, vs)):
        w = p.clone().view(-1, Hkv, d)
        r = new[src[ok]]
        w[slots[ok].long()] = codes_of(r, s) if fp8 else r
        want.append(w.view_as(p))
    if fp8:
        got = bw.kv_append_paged_fp8(k_new, v_new, slots, kp, vp, ks, vs, rows=rows)
    else:
        got = bw.kv_append_paged(k_new, v_new, slots, kp, vp, rows=rows)
    assert got[0] is kp and torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def e4m3_values():
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))


def codes_of(x, scale):
    """The nearest E4M3 code of x / scale from the format's definition (exact: the quotient is compared
    with each border as x against border * scale, 24 + 5 bits in 64)."""
    val = e4m3_values()
    x, s = x.double().cpu().numpy(), scale.double().cpu().numpy()
    ax, s = np.abs(x), np.broadcast_to(s, x.shape)
    code = np.zeros(x.shape, np.int64)
    for c in range(126):
        border = (val[c] + val[c + 1]) / 2 * s
        code += (ax > border) | ((ax == border) & (c % 2 == 1))  # a tie goes to the even code
    code = np.where(np.isnan(x), 127, code) | np.where(np.signbit(x), 128, 0)
    return torch.from_numpy(code.astype(np.uint8)).cuda()


def test_append_fp8_every_value():
    # every bf16 bit pattern, over scales that put quotients on and next to the borders
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16).view(512, 1, 128)
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    kp = torch.zeros((32, 16, 1, 128), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    g = gen(5)
    for s in (1.0, 0.01, 3.0, 1 / 3, 448 / 4.5, 4.5 / 448, 1.0000001, 0.99999994, 1e-20, 1e20, None):
        if s is None:
            ks = torch.exp(torch.randn((1, 128), generator=g, device="cuda") * 3)
            vs = torch.exp(torch.randn((1, 128), generator=g, device="cuda") * 20)
        else:
            ks = torch.full((1, 128), s, device="cuda")
            vs = ks * 1.9
        bw.kv_append_paged_fp8(x, x, slots, kp, vp, ks, vs)
        for p, sc in ((kp, ks), (vp, vs)):
            got, want = p.view(512, 1, 128), codes_of(x, sc)
            nan = torch.isnan(x)
            assert torch.equal(got[~nan], want[~nan]), (s, int((got != want).sum()))
            assert bool(((got[nan] & 127) == 127).all())


def test_append_fp8_extreme_scales():
    # the ends of the normal range, where a reciprocal or a remainder runs out of exponents, and powers of
    # two, whose quotients fall on the borders themselves; any two channels of a thread differ
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16).view(256, 1, 256)
    slots = torch.arange(256, dtype=torch.int32, device="cuda")
    kp = torch.zeros((16, 16, 1, 256), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    tops = [1.0, 1.9999999, 1.3333334, 1.0000001, 1.5, 1.0625]
    exps = [-126, -125, -100, -66, -65, -64, -63, -9, 0, 9, 64, 100, 124, 125, 126, 127]
    s = [np.float32(m) * np.float32(2.0) ** np.float32(e) for e in exps for m in tops]
    s = torch.tensor(np.array(s, np.float32), device="cuda")
    assert bool(torch.isfinite(s).all()) and bool((s >= torch.finfo(torch.float32).tiny).all())
    g = gen(6)
    for _ in range(4):
        ks, vs = (s[torch.randint(0, s.numel(), (1, 256), generator=g, device="cuda")] for _ in range(2))
        bw.kv_append_paged_fp8(x, x, slots, kp, vp, ks, vs)
        for p, sc in ((kp, ks), (vp, vs)):
            got, want = p.view(256, 1, 256), codes_of(x, sc)
            nan = torch.isnan(x)
            assert torch.equal(got[~nan], want[~nan]), int((got != want).sum())
            assert bool(((got[nan] & 127) == 127).all())


def test_merge_many_units_and_few():
    # parts of a few units among many CTAs (their records are searched for) and a part at every boundary
    for i, (Hq, Hkv, d, page, nks, nqs) in enumerate([
            (8, 2, 128, 0, [9000, 3], [3, 1]), (12, 3, 64, 48, [9001], [5]), (6, 6, 256, 16, [7000, 1, 0, 5000], [9, 2, 1, 4]),
            (10, 5, 128, 16, [3000] * 7 + [0, 4111], [30] * 9), (7, 7, 64, 0, [1500 + 97 * x for x in range(40)], [2] * 40),
            (11, 11, 64, 16, [700] * 60, [33] * 60), (24, 8, 128, 32, [6000] * 3, [64, 1, 50])]):
        t = Case(Hq, Hkv, d, page, nks, nqs, seed=40 + i)
        t.check(*t.run(), what=(Hq, Hkv, d, page))


@pytest.mark.parametrize("Hq,Hkv,d,page,nk,nodes", [
    (16, 16, 128, 16, [300, 4000], [20, 3]), (12, 12, 64, 48, [2000, 0, 700], [9, 1, 30]), (64, 16, 256, 16, [100, 2500], [5, 7]),
    (36, 9, 64, 16, [900, 33], [40, 2]), (26, 13, 128, 32, [640], [70]), (4, 1, 64, 0, [100, 7], [1024, 1000]),
    (8, 2, 128, 16, [300], [1024])])
def test_tree_heads_and_most_nodes(Hq, Hkv, d, page, nk, nodes):
    # KV heads read side by side in groups of 8, 6, 8, 3 and one by one; and trees of the most nodes
    c = Case(Hq, Hkv, d, page, nk, nodes, "any", seed=Hq + d)
    c.check(*c.run(), what=(Hq, Hkv, d, page))


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_serving_run(page, fp8):
    """Prompts into pages, then steps of drafting a tree, verifying it and keeping the accepted path;
    every attention is checked against the keys and values that the requests have by then."""
    B, Hq, Hkv, d, steps = 3, 8, 2, 128, 4
    g, r = gen(91), np.random.default_rng(91)
    pages, mp = 60, 30
    dt = torch.uint8 if fp8 else torch.bfloat16
    kp, vp = (torch.zeros((pages, page, Hkv, d), dtype=dt, device="cuda") for _ in range(2))
    scales = [(0.5 + torch.rand((Hkv, d), generator=g, device="cuda")) * (4.5 / 448) for _ in range(2)]
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    nk, held, count = i32([0] * B), i32([0] * B), i32([pages])
    have = [[torch.empty((0, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(B)]

    def append(k, v, slots, rows=None):
        if fp8:
            bw.kv_append_paged_fp8(k, v, slots, kp, vp, *scales, rows=rows)
        else:
            bw.kv_append_paged(k, v, slots, kp, vp, rows=rows)

    prompt = [70, 0, 33]
    k, v = randn((sum(prompt), Hkv, d), g), randn((sum(prompt), Hkv, d), g)
    nk, held, cu, slots, count = bw.kv_plan_paged(nk, i32(prompt), table, held, free, count, page, sum(prompt))
    append(k, v, slots)
    for b in range(B):
        have[b] = [x[cu[b]:cu[b + 1]] for x in (k, v)]
    for step in range(steps):
        nodes = [int(x) for x in r.integers(1, 20, B)]
        total, bound = sum(nodes), max(nodes)
        cu = sums(nodes)
        parents = [int(r.integers(max(-1, i - 3), i)) if i else -1 for n in nodes for i in range(n)]
        mask, pos = bw.attn_tree_mask(i32(parents), cu, bound, nk=nk)
        q, k, v = randn((total, Hq, d), g, 2.0), randn((total, Hkv, d), g), randn((total, Hkv, d), g)
        if not fp8:
            c = Case.__new__(Case)
            c.Hq, c.Hkv, c.d, c.nk, c.nodes = Hq, Hkv, d, nk.tolist(), nodes
            c.q, c.k_new, c.v_new, c.ctx = q, k, v, have
            c.sees = []
            at = 0
            for n in nodes:
                s = np.zeros((n, n), bool)
                for i in range(n):
                    if parents[at + i] >= 0:
                        s[i] = s[parents[at + i]]
                    s[i, i] = True
                c.sees.append(s)
                at += n
            o, lse = bw.attn_tree_paged(q, kp, vp, table, k, v, nk, cu, mask, bound)
            c.check(o, lse, step)
        # the path to some node of each tree is accepted
        rows, taken, at = [], [], 0
        for b, n in enumerate(nodes):
            i, path = int(r.integers(0, n)), []
            while i >= 0:
                path.append(at + i)
                i = parents[at + i]
            rows += path[::-1]
            taken.append(len(path))
            assert int(pos[path[0]]) == int(nk[b]) + len(path) - 1
            have[b] = [torch.cat([x, y[path[::-1]]]) for x, y in zip(have[b], (k, v))]
            at += n
        nk, held, _, slots, count = bw.kv_plan_paged(nk, i32(taken), table, held, free, count, page, total)
        assert int(count) >= 0
        append(k, v, slots[:len(rows)].contiguous(), i32(rows))
    assert nk.tolist() == [len(x[0]) for x in have]
    # the paged decode reads what the appends wrote
    q = randn((B, Hq, d), g)
    if fp8:
        o, _ = bw.attn_decode_paged_fp8(q, kp, vp, *scales, table.clamp(min=0), nk, num_splits=2)
        kc, vc = (torch.zeros((B, Hkv, 128, d), dtype=torch.float64) for _ in range(2))
        val = torch.from_numpy(e4m3_values())
        for b in range(B):
            for dst, x, s in ((kc, have[b][0], scales[0]), (vc, have[b][1], scales[1])):
                code = codes_of(x, s).cpu().long()
                dst[b, :, :len(x)] = (val[code & 127] * (1 - 2 * (code >> 7)) * s.double().cpu()).transpose(0, 1)
        ref, _ = oracle.decode(q.double().cpu().numpy(), kc.numpy(), vc.numpy(), nk.cpu().numpy(), method="naive")
    else:
        o, _ = bw.attn_decode_paged(q, kp, vp, table.clamp(min=0), nk, num_splits=2)
        kc, vc = (np.zeros((B, Hkv, 128, d)) for _ in range(2))
        for b in range(B):
            for dst, x in ((kc, have[b][0]), (vc, have[b][1])):
                dst[b, :, :len(x)] = x.double().cpu().numpy().transpose(1, 0, 2)
        ref, _ = oracle.decode(q.double().cpu().numpy(), kc, vc, nk.cpu().numpy(), method="naive")
    assert np.abs(o.double().cpu().numpy() - ref).max() <= 2e-2  # the decode's own bound


@pytest.mark.parametrize("how", ["eager", "graph"])
def test_back_to_back_chain(how):
    """Each kernel reads what the one before it wrote, with nothing in between: the packed prefill's output
    is the trees' queries, their output the rows that are appended, and a decode reads the pages. The same
    calls with a synchronisation behind each give the values."""
    Hq, Hkv, d, page, B = 16, 4, 128, 16, 3
    q_lens, k_lens, nodes, nk = [300, 7, 40], [300, 900, 40], [30, 7, 40], [1000, 17, 300]
    g = gen(77)
    q = randn((sum(q_lens), Hq, d), g)
    k, v = randn((sum(k_lens), Hkv, d), g), randn((sum(k_lens), Hkv, d), g)
    cu_q, cu_k, cu_n = sums(q_lens), sums(k_lens), sums(nodes)
    total = sum(nodes)
    pages0 = [randn((120, page, Hkv, d), g) for _ in range(2)]
    kp, vp = (x.clone() for x in pages0)
    r = np.random.default_rng(3)
    parents = i32(np.concatenate([[r.integers(-1, i) if i else -1 for i in range(n)] for n in nodes]).tolist())
    have = [(n + page - 1) // page for n in nk]
    table0 = torch.full((B, 70), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(have):
        table0[b, :n] = torch.arange(at, at + n, device="cuda")
        at += n
    table = table0.clone()
    free, count, n_new = torch.arange(at, 120, dtype=torch.int32, device="cuda"), i32([120 - at]), i32(nodes)
    lens, held = i32(nk), i32(have)
    ws = torch.empty(bw.tree_workspace_size(B, max(nodes), Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def chain(between):
        kp.copy_(pages0[0]), vp.copy_(pages0[1]), table.copy_(table0)
        between()
        o, _ = bw.attn_varlen(q, k, v, cu_q, cu_k, max(q_lens), max(k_lens), causal=True)
        between()
        nk1, _, cu, slots, left = bw.kv_plan_paged(lens, n_new, table, held, free, count, page, total)
        between()
        mask, _ = bw.attn_tree_mask(parents, cu, max(nodes), nk=lens)
        between()
        qt = o[:total]
        o2, lse2 = bw.attn_tree_paged(qt, kp, vp, table, qt[:, :Hkv], qt[:, Hkv:2 * Hkv], lens, cu, mask, max(nodes), workspace=ws)
        between()
        bw.kv_append_paged(o2[:, :Hkv], o2[:, Hkv:2 * Hkv], slots, kp, vp)
        between()
        mask2, pos = bw.attn_tree_mask(parents, cu, max(nodes), nk=nk1)
        between()
        o3, lse3 = bw.attn_tree_paged(o2, kp, vp, table, o2[:, :Hkv], o2[:, Hkv:2 * Hkv], nk1, cu, mask2, max(nodes), workspace=ws)
        between()
        o4, lse4 = bw.attn_decode_paged(o3[:B], kp, vp, table.clamp(min=0), nk1, num_splits=4)
        return o, o2, lse2, o3, lse3, o4, lse4, kp, vp, table, slots, pos, left

    want = [x.clone() for x in chain(torch.cuda.synchronize)]
    assert int(want[-1]) >= 0
    if how == "graph":
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = chain(lambda: None)
    for _ in range(20):
        if how == "graph":
            graph.replay()
        else:
            got = chain(lambda: None)
        for i, (x, w) in enumerate(zip(got, want)):
            assert torch.equal(x, w), i


def test_fork_and_join_in_a_graph():
    # kernels with dependencies on two streams at once, captured: the append on one, the mask on the other,
    # both joined ahead of the attention that reads the pages and the mask
    t = Case(16, 4, 128, 16, [500, 33], [20, 9], "tree", seed=91)
    n = sum(t.nodes)
    parents = i32([-1] + [(i - 1) // 2 for i in range(1, 20)] + [-1] + [(i - 1) // 2 for i in range(1, 9)] + [0] * (t.total - n))
    slots = torch.cat([t.table[0, :2], t.table[1, :2]]).repeat_interleave(7) * 16 + torch.arange(28, device="cuda").to(torch.int32) % 7
    k0, v0 = t.k.clone(), t.v.clone()
    ws = torch.empty(bw.tree_workspace_size(2, t.max_nodes, 16, 4, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(t.q), torch.empty((t.total, 16), device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        here = torch.cuda.current_stream()
        t.k.copy_(k0), t.v.copy_(v0)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            bw.attn_tree_mask(parents, t.cu, t.max_nodes, mask=t.mask)
        bw.kv_append_paged(t.k_new, t.v_new, slots, t.k, t.v)
        here.wait_stream(side)
        t.run(out=o, lse=lse, workspace=ws)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        calls()
    torch.cuda.synchronize()
    bits = lambda x: x.view(torch.int16)  # unused rows hold NaN
    want = o[:n].clone(), lse[:n].clone(), t.k.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        calls()
    for _ in range(10):
        o.zero_(), lse.zero_(), t.mask.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:n], want[0]) and torch.equal(lse[:n], want[1])
        assert torch.equal(bits(t.k), bits(want[2]))


def test_beside_prefill_and_decode_on_other_streams():
    # three streams at once, each call over and over; the results are those of the calls alone
    t = Case(32, 8, 128, 16, [3000, 40, 900], [64, 5, 20], "tree", seed=95)
    small = Case(12, 4, 64, 0, [700, 90], [9, 3], "tree", seed=96)
    g = gen(97)
    q, k, v = (randn((2, 8, 1000, 128), g) for _ in range(3))
    qd, kc, vc = randn((4, 32, 128), g), randn((4, 8, 2000, 128), g), randn((4, 8, 2000, 128), g)
    nk = i32([2000, 1, 777, 1500])
    calls = [lambda: t.run()[0][:sum(t.nodes)], lambda: small.run()[0][:sum(small.nodes)], lambda: bw.attn_fwd(q, k, v, causal=True)[0],
             lambda: bw.attn_decode(qd, kc, vc, nk, num_splits=8)[0]]
    want = []
    for c in calls:
        want.append(c())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, c, x in zip(streams, calls, got):
            with torch.cuda.stream(s):
                x.append(c())
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert all(torch.equal(w, y) for y in x)


@pytest.mark.parametrize("Hq,Hkv,d,page", [(8, 4, 128, 128), (8, 8, 64, 64), (6, 3, 64, 128), (4, 2, 256, 64), (8, 8, 128, 16), (8, 8, 64, 16)])
def test_tree_tiles_without_copies_for_the_helper(Hq, Hkv, d, page):
    # one row tile over pages: pages so large that the helping producer warp has no copy, contexts so short that
    # it has some in few tiles, and drafts, which it never copies, one after another in every CTA's list
    r = np.random.default_rng(d + page)
    nk = [int(x) for x in r.choice([0, 1, 15, 17, 33, 100, 130, 2000], 300)]
    n = [int(x) for x in r.integers(1, 9, 300)]
    c = Case(Hq, Hkv, d, page, nk, n, "tree", seed=101)
    o, lse = c.run()
    c.check(o, lse)
    want = o[:sum(n)].clone()
    for _ in range(200):
        c.run(out=o)
    assert torch.equal(o[:sum(n)], want)
    assert bw.get_status() == bw.OK  # no wait ran out


def test_mask_calls_of_several_threads():
    # each takes another amount of shared memory; the C calls run side by side
    call, sizes = bw.lib().attn_tree_mask, (1024, 400, 900, 513)
    start, codes = threading.Barrier(len(sizes)), [set() for _ in sizes]
    masks, keep, threads = [], [], []

    def work(i, args):
        start.wait()
        for _ in range(20000):
            codes[i].add(call(*args))

    for i, n in enumerate(sizes):
        parents, cu, stream = i32(range(-1, n - 1)), sums([n]), torch.cuda.Stream()  # one line
        masks.append(torch.zeros((n, (n + 63) // 64), dtype=torch.int64, device="cuda"))
        keep.append((parents, cu, stream))
        args = (parents.data_ptr(), cu.data_ptr(), None, masks[i].data_ptr(), None, 1, n, n, stream.cuda_stream)
        args = [x if x is None else t(x) for x, t in zip(args, call.argtypes)]
        threads.append(threading.Thread(target=work, args=(i, args)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{bw.OK}] * len(sizes)
    for n, m in zip(sizes, masks):
        assert np.array_equal(m.cpu().numpy(), pack(np.tril(np.ones((n, n), bool)), m.shape[1]))


def codes_on_gpu(x, scale):
    """``codes_of`` for many values: the same comparisons, on the GPU."""
    val = e4m3_values()
    ax, s = x.double().abs(), scale.double()
    code = torch.zeros(x.shape, dtype=torch.uint8, device="cuda")
    for c in range(126):
        border = (val[c] + val[c + 1]) / 2 * s
        code += (ax >= border) if c % 2 == 1 else (ax > border)
    return code | torch.signbit(x).to(torch.uint8) << 7


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,d,batches,more", [(64, 256, 1, 0), (64, 256, 2, 1), (64, 256, 5, 77), (8, 128, 3, 1001), (3, 64, 4, 13)])
@pytest.mark.parametrize("how", ["plain", "fused", "gather"])
def test_append_batch_after_batch(fp8, Hkv, d, batches, more, how):
    # every thread goes through several batches of rows, the last of them partly filled: a batch is at most
    # 152 SMs x blocks x 256 threads of 16 output bytes, times its rows
    batch = 152 * 256 * (4 * 16 if fp8 else 32 * 2 * 8) // (Hkv * d)
    n, page = batches * batch + more, 16
    g = gen(n + d)
    rows_in = n + 50
    if how == "fused":
        x = randn((rows_in, 2 + 2 * Hkv, d), g, 3.0)
        k_new, v_new = x[:, 2:2 + Hkv], x[:, 2 + Hkv:]
    else:
        k_new, v_new = randn((rows_in, Hkv, d), g, 3.0), randn((rows_in, Hkv, d), g, 3.0)
    pages = n // page + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    slots[torch.rand(n, generator=g, device="cuda") < 0.05] = -1
    rows = torch.randint(-20, rows_in + 20, (n,), generator=g, device="cuda").to(torch.int32) if how == "gather" else None
    src = torch.arange(n, device="cuda") if rows is None else rows.long()
    ok = (slots >= 0) & (src >= 0) & (src < rows_in)
    ks, vs = (torch.rand((Hkv, d), generator=g, device="cuda") * 0.02 + 1e-3 for _ in range(2))
    kp, vp = (torch.full((pages, page, Hkv, d), 7, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2))
    if fp8:
        bw.kv_append_paged_fp8(k_new, v_new, slots, kp, vp, ks, vs, rows=rows)
    else:
        bw.kv_append_paged(k_new, v_new, slots, kp, vp, rows=rows)
    for p, new, s in ((kp, k_new, ks), (vp, v_new, vs)):
        want = torch.full_like(p, 7).view(-1, Hkv, d)
        r = new[src[ok]]
        want[slots[ok].long()] = codes_on_gpu(r, s) if fp8 else r
        assert torch.equal(p.view(-1, Hkv, d), want)


def test_plan_keys_near_the_end_of_32_bits():
    # the widest table of 48-row pages; the last pages of a request that fills it to within some keys
    P = 48
    columns = 0x7fffffff // P
    table = np.full((1, columns), -1, np.int32)
    for left in (5, 0, -20):  # keys to the table's end
        plan_check([P * columns - left - 45], [45], table, [columns - 2], [5, 6, 7], 3, P, 50)


@pytest.mark.parametrize("B,P,most", [(2047, 16, 5), (2048, 48, 3), (2049, 16, 4), (4096, 16, 2), (5000, 16, 40), (9000, 128, 30)])
def test_plan_of_more_requests_than_a_scan(B, P, most):
    # requests are scanned 2048 at a time: what is carried from scan to scan, a stack and slots that run out
    # behind the first, and (5000 and 9000 requests) the scans' outputs by several blocks
    r = np.random.default_rng(B)
    nk = r.integers(0, 200, B)
    new = r.integers(0, most + 1, B)
    new[r.integers(0, B, 3)] = 300
    held = np.maximum(-(-nk // P) + r.integers(-1, 3, B), 0)
    need = np.maximum(0, -(-(nk + new) // P) - held)
    columns = int((held + need).max())
    pages = r.permutation(int(held.sum() + need.sum()) + 9).astype(np.int32)
    table = np.full((B, columns), -1, np.int32)
    inside = np.arange(columns)[None] < held[:, None]
    table[inside] = pages[:held.sum()]
    free, tokens = pages[held.sum():].tolist(), int(new.sum())
    behind = min(B - 1, 2048 + B // 7)  # a request of a later scan, where there is one
    for count, slots in ((len(free), tokens + 30), (int(need[:behind].sum()), tokens), (len(free), int(new[:behind].sum()) + 1), (0, 17)):
        plan_check(nk.tolist(), new.tolist(), table, held.tolist(), free, count, P, slots)


def test_plan_of_more_tokens_than_threads():
    # above 152 x 1024 tokens a thread takes several, in several scans
    r = np.random.default_rng(8)
    B, P = 2100, 64
    nk, new = r.integers(0, 100, B), r.integers(0, 200, B)
    held = -(-nk // P)
    need = np.maximum(0, -(-(nk + new) // P) - held)
    tokens = int(new.sum())
    assert int(new[:2048].sum()) > 152 * 1024
    table = np.full((B, 8), -1, np.int32)
    table[np.arange(8)[None] < held[:, None]] = np.arange(held.sum())
    free = np.arange(held.sum(), (held + need).sum()).tolist()
    plan_check(nk.tolist(), new.tolist(), table, held.tolist(), free, len(free), P, tokens + 5)


def test_tree_without_a_cache():
    # a cache of no rows (its pointers may be null), whatever the lengths say
    c = Case(8, 2, 128, 0, [0, 0, 0], [9, 0, 150], "any", seed=111)
    c.k = c.v = torch.empty((3, 2, 0, 128), dtype=torch.bfloat16, device="cuda")
    c.nk_t = i32([0, 5, 1 << 30])
    c.check(*c.run())


@pytest.mark.parametrize("d,page", [(64, 16), (128, 0), (256, 16)])
def test_tree_without_nodes(d, page):
    c = Case(8, 2, d, page, [300, 40], [0, 0], seed=113, bound=40)  # rows, but none of a sequence
    o = torch.full((c.total, 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.total, 8), 7.0, device="cuda")
    c.run(out=o, lse=lse)
    assert bool((o == 7).all()) and bool((lse == 7).all())


def test_tree_cache_past_32_bits():
    # contiguous caches whose later sequences' elements lie past 2^32
    B, Hkv, cap, d = 3, 4, 4_500_000, 128
    c = Case(8, Hkv, d, 0, [200, 0, 333], [10, 2, 40], "tree", seed=115)
    k, v = (torch.empty((B, Hkv, cap, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k[:2].numel() > 1 << 32
    for b, n in enumerate(c.nk):
        k[b, :, :n], v[b, :, :n] = (x.transpose(0, 1) for x in c.ctx[b])
    c.k, c.v = k, v
    c.check(*c.run())


def test_tree_most_sequences():
    # 65535 requests of one node, and as many heads as a call of one request may have
    B, d, most = 65535, 64, 20
    g = gen(117)
    nk = torch.randint(0, most + 1, (B,), generator=g, device="cuda").to(torch.int32)
    q, k_new, v_new = randn((B, 2, d), g, 2.0), randn((B, 1, d), g), randn((B, 1, d), g)
    k, v = randn((B, 1, most, d), g), randn((B, 1, most, d), g)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    mask = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    o, lse = bw.attn_tree(q, k, v, k_new, v_new, nk, cu, mask, 1)
    kk, vv = (torch.cat([x[:, 0], y], 1).double() for x, y in ((k, k_new), (v, v_new)))
    see = torch.arange(most + 1, device="cuda")[None] < nk[:, None]
    see[:, most] = True
    s = (q.double() @ kk.transpose(1, 2) / math.sqrt(d)).masked_fill(~see[:, None], -INF)
    p = torch.softmax(s, -1)
    E = (d + 8) * 2.0 ** -24 * (q.double().abs() @ kk.abs().transpose(1, 2) / math.sqrt(d)).amax(-1)
    ref, A = p @ vv, p @ vv.abs()
    dO = (2.0 ** -8 + 4 * E)[..., None] * A
    assert bool(((o.double() - ref).abs() <= dO + 2.0 ** -8 * (ref.abs() + dO) + 1e-30).all())
    z = torch.logsumexp(s, -1)
    assert bool(((lse.double() - z).abs() <= E + 21 * 2.0 ** -24 + 2.0 ** -21 * (1 + z.abs())).all())
    c = Case(2048, 512, 64, 16, [70], [3], "tree", seed=118)
    c.check(*c.run())


def test_append_rows_of_the_pool():
    # rows moved within the pool: none of those read is written
    g = gen(119)
    pages, page, Hkv, d = 40, 16, 2, 128
    kp, vp = randn((pages, page, Hkv, d), g), randn((pages, page, Hkv, d), g)
    order = torch.randperm(pages * page, generator=g, device="cuda").to(torch.int32)
    rows, slots = order[:300].contiguous(), order[300:600].contiguous()
    want = []
    for p in (kp, vp):
        w = p.clone().view(-1, Hkv, d)
        w[slots.long()] = w[rows.long()]
        want.append(w.view_as(p))
    bw.kv_append_paged(kp.view(-1, Hkv, d), vp.view(-1, Hkv, d), slots, kp, vp, rows=rows)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_append_to_pages_of_a_float8_type():
    g = gen(121)
    k_new, v_new = randn((50, 2, 64), g), randn((50, 2, 64), g)
    ks, vs = (torch.rand((2, 64), generator=g, device="cuda") * 0.02 + 1e-3 for _ in range(2))
    kp, vp = (torch.zeros((4, 16, 2, 64), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    slots = torch.randperm(64, generator=g, device="cuda")[:50].to(torch.int32)
    bw.kv_append_paged_fp8(k_new, v_new, slots, kp, vp, ks, vs)
    for p, x, s in ((kp, k_new, ks), (vp, v_new, vs)):
        assert torch.equal(p.view(torch.uint8).view(-1, 2, 64)[slots.long()], codes_of(x, s))


def test_tree_captured_without_a_workspace():
    # what a captured call allocates lives in the graph's memory, and two graphs replayed at once have their own
    cases = [Case(16, 4, 128, 16, [3000, 5], [20, 9], "tree", seed=123), Case(16, 4, 128, 16, [40, 2500], [7, 30], "any", seed=124)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(30):
        for g, s, (o, l) in zip(graphs, streams, outs):
            with torch.cuda.stream(s):
                o.zero_(), l.zero_()
                g.replay()
    torch.cuda.synchronize()
    for c, (o, l), (wo, wl) in zip(cases, outs, want):
        n = sum(c.nodes)
        assert torch.equal(o[:n], wo[:n]) and torch.equal(l[:n], wl[:n])


def test_refusals_of_the_binding():
    c = Case(8, 2, 128, 16, [40, 3], [5, 2], "tree", seed=127)
    t = dict(q=c.q, k=c.k, v=c.v, table=c.table, k_new=c.k_new, v_new=c.v_new, nk=c.nk_t, cu=c.cu, mask=c.mask, max_nodes=c.max_nodes)
    wide = torch.zeros((c.total, 2, 132), dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        x = {**t, **kw}
        return bw.attn_tree_paged(x["q"], x["k"], x["v"], x["table"], x["k_new"], x["v_new"], x["nk"], x["cu"], x["mask"],
                                  x["max_nodes"], **{n: kw[n] for n in ("out", "lse", "workspace") if n in kw})
    call()
    for kw in (dict(q=c.q.float()), dict(q=c.q[:, :, ::2]), dict(q=c.q.transpose(0, 1)), dict(k=c.k[:, :, :1]), dict(v=c.v[1:]),
               dict(k=c.k.half()), dict(k_new=c.k_new[1:]), dict(k_new=wide[:, :, :128]), dict(v_new=c.v_new.cpu()),
               dict(v_new=c.v_new[:1].expand(c.total, 2, 128)), dict(table=c.table.long()), dict(table=c.table[:, ::2]),
               dict(nk=c.nk_t[:1]), dict(nk=c.nk_t.long()), dict(cu=c.cu[:2]), dict(mask=c.mask[:-1]), dict(mask=c.mask.to(torch.int32)),
               dict(max_nodes=65), dict(out=c.q[:-1].clone()), dict(lse=torch.zeros((c.total, 7), device="cuda")),
               dict(workspace=torch.zeros(1 << 26, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(bw.BwattnError):
        call(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    slots = i32(range(c.total))
    for args in ((c.k_new.float(), c.v_new, slots, c.k, c.v), (c.k_new, c.v_new[:-1], slots, c.k, c.v), (c.k_new, c.v_new, slots.long(), c.k, c.v),
                 (c.k_new, c.v_new, slots, c.k, c.v[:-1]), (c.k_new, c.v_new, slots, c.k.float(), c.v.float())):
        with pytest.raises(ValueError):
            bw.kv_append_paged(*args)
    with pytest.raises(ValueError):
        bw.kv_append_paged(c.k_new, c.v_new, slots, c.k, c.v, rows=slots[1:])
    with pytest.raises(bw.BwattnError):
        bw.kv_append_paged(c.k_new[1:], c.v_new[1:], slots, c.k, c.v)  # more slots than rows
    with pytest.raises(ValueError):
        bw.kv_append_paged_fp8(c.k_new, c.v_new, slots, c.k, c.v, torch.ones((2, 128), device="cuda"), torch.ones((2, 128), device="cuda"))
    with pytest.raises(ValueError):
        bw.attn_tree_mask(i32([0]).long(), i32([0, 1]), 1)
    with pytest.raises(ValueError):
        bw.attn_tree_mask(i32([0]), i32([0, 1]), 1, nk=i32([1, 2]))
    with pytest.raises(bw.BwattnError):
        bw.attn_tree_mask(i32([0]), i32([0, 1]), 1025)
    for a, b in ((i32([1]), i32([0, 1])), (i32([1, 2]), i32([0]))):
        with pytest.raises(ValueError):
            bw.kv_plan_paged(a, b, c.table, i32([1, 1]), i32([3, 4]), i32([2]), 16, 4)
    with pytest.raises(bw.BwattnError):
        bw.kv_plan_paged(i32([1, 2]), i32([0, 1]), c.table, i32([1, 1]), i32([3, 4]), i32([2]), 24, 4)

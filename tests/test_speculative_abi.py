"""Argument checks of the speculative-decoding calls: rejected on the host before any CUDA call, so
these run without a GPU."""
import pytest
import torch

import exact_attention_flashattn_gb300 as bw
from exact_attention_flashattn_gb300 import build as bw_build

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    bw_build.build()
    return bw.lib()


def tree(L, paged=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, kn=FAKE, vn=FAKE, o=FAKE, lse=None, nk=FAKE, cu=FAKE, mask=FAKE, n=2, tq=9,
             mn=8, cap=64, ps=16, npg=10, mp=4, Hq=8, Hkv=2, d=128, qs=1024, ks=256, vs=256, scale=0.1, ws=FAKE,
             wsb=1 << 40, stream=None)
    a.update(kw)
    if paged:
        return L.attn_tree_paged(a["q"], a["k"], a["v"], a["table"], a["kn"], a["vn"], a["o"], a["lse"], a["nk"], a["cu"],
                                 a["mask"], a["n"], a["tq"], a["mn"], a["ps"], a["npg"], a["mp"], a["Hq"], a["Hkv"], a["d"],
                                 a["qs"], a["ks"], a["vs"], a["scale"], a["ws"], a["wsb"], a["stream"])
    return L.attn_tree(a["q"], a["k"], a["v"], a["kn"], a["vn"], a["o"], a["lse"], a["nk"], a["cu"], a["mask"], a["n"],
                       a["tq"], a["mn"], a["cap"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["ks"], a["vs"], a["scale"],
                       a["ws"], a["wsb"], a["stream"])


@pytest.mark.parametrize("paged", [False, True])
def test_tree_refusals(L, paged):
    for name in ("q", "k", "v", "kn", "vn", "o", "nk", "cu", "mask", "ws"):
        assert tree(L, paged, **{name: None}) == bw.ERR_INVALID_ARG, name
    for name, off in (("q", 8), ("k", 8), ("v", 8), ("kn", 2), ("vn", 2), ("o", 8), ("nk", 2), ("cu", 1), ("mask", 4),
                      ("lse", 2), ("ws", 8)):
        assert tree(L, paged, **{name: FAKE + off}) == bw.ERR_INVALID_ARG, name
    for kw in (dict(n=-1), dict(tq=-1), dict(mn=-1), dict(Hq=0), dict(Hkv=0), dict(d=0), dict(Hq=7), dict(n=65536),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=1016), dict(qs=1028),
               dict(ks=255), dict(ks=128), dict(vs=250), dict(ks=-256), dict(vs=1 << 38)):
        assert tree(L, paged, **kw) == bw.ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(d=32, qs=1024), dict(mn=1025), dict(Hq=258, qs=258 * 128)):
        assert tree(L, paged, **kw) == bw.ERR_UNSUPPORTED, kw
    need = L.attn_tree_workspace_size(2, 8, 8, 2, 128)
    assert need > 0 and tree(L, paged, wsb=need - 1) == bw.ERR_INVALID_ARG
    for kw in (dict(n=0), dict(tq=0), dict(mn=0)):  # no work
        assert tree(L, paged, q=None, kn=None, **kw) == bw.OK


def test_tree_paged_refusals(L):
    for kw in (dict(table=None), dict(table=FAKE + 2), dict(ps=8), dict(ps=24), dict(ps=1040), dict(npg=0), dict(mp=0),
               dict(npg=1 << 28), dict(mp=1 << 28)):
        assert tree(L, True, **kw) == bw.ERR_INVALID_ARG, kw
    assert tree(L, False, cap=-1) == bw.ERR_INVALID_ARG


def test_tree_workspace_size(L):
    f = L.attn_tree_workspace_size
    assert f(0, 8, 8, 2, 128) == f(1, 0, 8, 2, 128) == f(1, 8, 8, 3, 128) == f(1, 8, 8, 2, 96) == 0
    sizes = [f(n, m, 32, 8, d) for d in (64, 128, 256) for m in (1, 33, 1024) for n in (1, 500, 65535)]
    assert all(s > 0 and s % 256 == 0 for s in sizes)


def test_tree_mask_refusals(L):
    def call(p=FAKE, cu=FAKE, nk=None, mask=FAKE, pos=None, n=2, tq=9, mn=8):
        return L.attn_tree_mask(p, cu, nk, mask, pos, n, tq, mn, None)
    for kw in (dict(p=None), dict(cu=None), dict(mask=None), dict(mask=FAKE + 4), dict(p=FAKE + 2), dict(nk=FAKE + 1),
               dict(pos=FAKE + 2), dict(n=-1), dict(tq=-1), dict(mn=-1)):
        assert call(**kw) == bw.ERR_INVALID_ARG, kw
    assert call(mn=1025) == bw.ERR_UNSUPPORTED
    assert call(n=0, p=None) == call(tq=0, p=None) == call(mn=0, p=None) == bw.OK


def test_plan_refusals(L):
    base = [0x1000 * (i + 16) for i in range(11)]
    names = ("nk", "new", "table", "held", "free", "count", "nk_out", "held_out", "cu", "slots", "free_out")

    def call(B=3, ps=16, mp=8, fc=20, nt=30, **kw):
        p = [kw.get(n, b) for n, b in zip(names, base)]
        return L.kv_plan_paged(*p, B, ps, mp, fc, nt, None)
    for n in names:
        assert call(**{n: None}) == bw.ERR_INVALID_ARG, n
        assert call(**{n: FAKE + 2}) == bw.ERR_INVALID_ARG, n
    for kw in (dict(B=-1), dict(ps=8), dict(ps=20), dict(ps=2048), dict(mp=0), dict(mp=1 << 28), dict(fc=-1), dict(nt=-1)):
        assert call(**kw) == bw.ERR_INVALID_ARG, kw
    ins, outs = (0, 1, 3, 4, 5), (2, 6, 7, 8, 9, 10)
    for i in ins:
        for o in outs:  # an output in an input's place
            assert call(**{names[o]: base[i]}) == bw.ERR_INVALID_ARG, (names[i], names[o])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(L, fp8):
    def call(kn=FAKE, vn=FAKE, slots=FAKE, rows=None, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, n=4, nr=4, ps=16, npg=3, Hkv=2,
             d=128, s0=256, s1=256):
        if fp8:
            return L.kv_append_paged_fp8(kn, vn, slots, rows, kp, vp, ks, vs, n, nr, ps, npg, Hkv, d, s0, s1, None)
        return L.kv_append_paged(kn, vn, slots, rows, kp, vp, n, nr, ps, npg, Hkv, d, s0, s1, None)
    for name in ("kn", "vn", "slots", "kp", "vp") + (("ks", "vs") if fp8 else ()):
        assert call(**{name: None}) == bw.ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == bw.ERR_INVALID_ARG, name
    for kw in (dict(rows=FAKE + 2), dict(n=-1), dict(nr=-1), dict(n=5), dict(ps=8), dict(ps=1040), dict(npg=0),
               dict(npg=1 << 28), dict(Hkv=0), dict(d=0), dict(s0=255), dict(s1=260), dict(s0=128)):
        assert call(**kw) == bw.ERR_INVALID_ARG, kw
    assert call(d=96) == bw.ERR_UNSUPPORTED
    assert call(n=0, kn=None) == call(nr=0, n=0, kn=None) == bw.OK


def test_python_checks():
    q, c, t = torch.zeros(3, 8, 128), torch.zeros(1, 2, 16, 128), torch.zeros(3, dtype=torch.int32)
    new = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError):
        bw.attn_tree(q, c, c, new, new, t, t, t, 3)
    with pytest.raises(ValueError):
        bw.attn_tree_mask(t, t, 3)
    with pytest.raises(ValueError):
        bw.kv_plan_paged(t, t, t[None], t, t, t[:1], 16, 4)
    with pytest.raises(ValueError):
        bw.kv_append_paged(new, new, t, c, c)


def test_tree_workspace_size_of_refused_sizes(L):
    # 0 for every size that the calls refuse, at the limits' two sides
    f = L.attn_tree_workspace_size
    for n, mn, Hq, Hkv, d in ((2, 1025, 8, 2, 128), (2, 8, 258, 2, 128), (2, 8, 129, 1, 64), (65536, 8, 8, 2, 128), (2, 8, 65536, 8192, 64),
                              (2, 8, 8, 2, 512), (-1, 8, 8, 2, 64), (2, -1, 8, 2, 64), (2, 8, 0, 2, 64), (2, 8, 8, 0, 64)):
        assert f(n, mn, Hq, Hkv, d) == 0, (n, mn, Hq, Hkv, d)
        if min(Hq, Hkv) > 0:
            assert tree(L, n=n, mn=mn, Hq=Hq, Hkv=Hkv, d=d, qs=Hq * d, ks=Hkv * d, vs=Hkv * d) in (bw.ERR_INVALID_ARG, bw.ERR_UNSUPPORTED)
    for n, mn, Hq, Hkv, d in ((2, 1024, 8, 2, 128), (2, 8, 256, 2, 128), (65535, 8, 8, 2, 128), (2, 8, 65520, 8190, 64)):
        assert f(n, mn, Hq, Hkv, d) > 0, (n, mn, Hq, Hkv, d)

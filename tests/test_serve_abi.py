"""Argument checks of the chunk, rotation and verification calls: rejected on the host before any CUDA call, so
these run without a GPU."""
import pytest
import torch

import exact_attention_flashattn_gb300 as bw
from exact_attention_flashattn_gb300 import build as bw_build

FAKE = 0x10000  # aligned, never dereferenced
BAD = bw.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    bw_build.build()
    return bw.lib()


def chunk(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, o=FAKE, lse=None, nk=FAKE, cu=FAKE, n=2, tq=9, mq=8, ps=16, npg=10, mp=4, Hq=8,
             Hkv=2, d=128, qs=1024, causal=1, scale=0.1, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return L.attn_chunk_paged(*[a[x] for x in ("q", "k", "v", "table", "o", "lse", "nk", "cu", "n", "tq", "mq", "ps", "npg", "mp",
                                               "Hq", "Hkv", "d", "qs", "causal", "scale", "ws", "wsb", "stream")])


def test_chunk_refusals(L):
    for name in ("q", "k", "v", "table", "o", "nk", "cu", "ws"):
        assert chunk(L, **{name: None}) == BAD, name
    for name, off in (("q", 8), ("k", 8), ("v", 2), ("table", 2), ("o", 8), ("nk", 2), ("cu", 1), ("lse", 2), ("ws", 8)):
        assert chunk(L, **{name: FAKE + off}) == BAD, name
    for kw in (dict(n=-1), dict(n=65536), dict(tq=-1), dict(mq=-1), dict(Hq=0), dict(Hkv=0), dict(d=0), dict(Hq=7), dict(ps=8),
               dict(ps=24), dict(ps=1040), dict(npg=0), dict(mp=0), dict(npg=1 << 28), dict(mp=1 << 28), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=1016), dict(qs=1028), dict(qs=1 << 38), dict(causal=2)):
        assert chunk(L, **kw) == BAD, kw
    for kw in (dict(d=96), dict(d=32), dict(Hq=258, qs=258 * 128)):
        assert chunk(L, **kw) == bw.ERR_UNSUPPORTED, kw
    # lengths whose sum, or whose tiles, pass 31 bits
    assert chunk(L, ps=1024, npg=1, mp=(1 << 21) - 1, tq=4096, mq=4096) == bw.ERR_UNSUPPORTED
    need = L.attn_chunk_workspace_size(2, 8, 8, 2, 128)
    assert need > 0 and chunk(L, wsb=need - 1) == BAD
    for kw in (dict(n=0), dict(tq=0), dict(mq=0)):  # no work
        assert chunk(L, q=None, **kw) == bw.OK


def test_chunk_workspace_size(L):
    f = L.attn_chunk_workspace_size
    for sizes in ((0, 8, 8, 2, 128), (2, 0, 8, 2, 128), (2, 8, 8, 3, 128), (2, 8, 8, 2, 96), (-1, 8, 8, 2, 64), (2, -1, 8, 2, 64),
                  (65536, 8, 8, 2, 128), (2, 8, 258, 2, 128), (2, 8, 0, 2, 64), (2, 8, 8, 0, 64), (2, 8, 8, 2, 512)):
        assert f(*sizes) == 0, sizes
        if sizes[0] != 0 and sizes[1] != 0:
            n, mq, Hq, Hkv, d = sizes
            assert chunk(L, n=n, mq=mq, Hq=Hq, Hkv=Hkv, d=d, qs=max(Hq, 1) * d) in (BAD, bw.ERR_UNSUPPORTED), sizes
    for sizes in ((1, 1, 1, 1, 64), (65535, 1 << 30, 256, 2, 128), (2, 8, 65520, 8190, 256)):
        assert f(*sizes) > 0, sizes


def rope(L, **kw):
    a = dict(q=FAKE, k=2 * FAKE, qo=3 * FAKE, ko=4 * FAKE, pos=FAKE, axes=None, freq=FAKE, qw=None, kw=None, eps=1e-6, n=5, na=1,
             pairs=64, inter=0, Hq=8, Hkv=2, d=128, qs=1024, ks=256, qos=1024, kos=256, stream=None)
    a.update(kw)
    return L.attn_qk_norm_rope(*[a[x] for x in ("q", "k", "qo", "ko", "pos", "axes", "freq", "qw", "kw", "eps", "n", "na", "pairs",
                                                "inter", "Hq", "Hkv", "d", "qs", "ks", "qos", "kos", "stream")])


def test_rope_refusals(L):
    for name in ("q", "k", "qo", "ko", "pos", "freq"):
        assert rope(L, **{name: None}) == BAD, name
    for name, off in (("q", 8), ("k", 2), ("qo", 8), ("ko", 8), ("pos", 2), ("axes", 1), ("freq", 2), ("qw", 8), ("kw", 2)):
        assert rope(L, **{name: 5 * FAKE + off}) == BAD, name
    for kw in (dict(n=-1), dict(na=0), dict(pairs=-1), dict(pairs=65), dict(inter=2), dict(Hq=0), dict(Hkv=0), dict(d=0),
               dict(Hq=65536, qs=65536 * 128, qos=65536 * 128), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(qs=1016), dict(ks=252), dict(qos=1028), dict(kos=128), dict(qs=1 << 38),
               dict(q=3 * FAKE, qs=2048), dict(k=4 * FAKE, ks=512), dict(q=4 * FAKE), dict(k=3 * FAKE), dict(ko=3 * FAKE)):
        assert rope(L, **kw) == BAD, kw
    assert rope(L, d=96) == bw.ERR_UNSUPPORTED
    assert rope(L, n=0, q=None, k=None) == bw.OK


def verify(L, **kw):
    names = ("tok", "par", "cu", "p", "q", "u", "w", "acc", "cnt", "nxt")
    a = {x: FAKE * (i + 1) for i, x in enumerate(names)}
    a.update(n=2, tq=9, mn=8, V=100, ps=100, qs=100, stream=None)
    a.update(kw)
    return L.attn_tree_verify(*[a[x] for x in names + ("n", "tq", "mn", "V", "ps", "qs", "stream")])


def test_verify_refusals(L):
    for name in ("tok", "par", "cu", "p", "u", "w", "acc", "cnt", "nxt"):
        assert verify(L, **{name: None}) == BAD, name
    for name in ("tok", "par", "cu", "p", "q", "u", "w", "acc", "cnt", "nxt"):
        assert verify(L, **{name: 20 * FAKE + 2}) == BAD, name
    for kw in (dict(n=-1), dict(n=65536), dict(tq=-1), dict(mn=-1), dict(V=0), dict(ps=99), dict(qs=99), dict(ps=1 << 38)):
        assert verify(L, **kw) == BAD, kw
    for kw in (dict(mn=1025), dict(V=500001, ps=1 << 20, qs=1 << 20)):
        assert verify(L, **kw) == bw.ERR_UNSUPPORTED, kw
    for i, out in enumerate(("acc", "cnt", "nxt")):  # an output in an input's place
        for j in range(7):
            assert verify(L, **{out: FAKE * (j + 1)}) == BAD, (out, j)
    for kw in (dict(acc=FAKE * 9), dict(acc=FAKE * 10), dict(cnt=FAKE * 10)):  # or in another output's
        assert verify(L, **kw) == BAD, kw
    assert verify(L, n=0, tq=0, tok=None, p=None, acc=None, cnt=None) == bw.OK


def test_python_checks():
    q, c, t = torch.zeros(3, 8, 128), torch.zeros(4, 16, 2, 128), torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(3, 10)
    with pytest.raises(ValueError):
        bw.attn_chunk_paged(q, c, c, t[None], t, t, 3)
    with pytest.raises(ValueError):
        bw.attn_qk_norm_rope(q, q[:, :2], t, f[0])
    with pytest.raises(ValueError):
        bw.attn_tree_verify(t, t, t, f, f[:, 0], f[:2, 0], 3)

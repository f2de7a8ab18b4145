"""Host-side checks of packed attention with grouped heads and of caches in pages that need no GPU: refusals at the C ABI
(before anything is launched) and in the Python layer, workspace sizes, overlaps, and whether the tests' bounds notice one
wrong tile."""
import itertools
import math

import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import pages_plain as P

BAD, NO, OK = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_OK
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# every call's arguments in the order of the C ABI, with values that pass every check but for the device
FWD = dict(q=1 * MB, k=2 * MB, v=3 * MB, cu=4 * MB, nseq=3, T=100, longest=60, out=5 * MB, lse=6 * MB, ws=7 * MB, wsb=1 << 19, Hq=4, Hkv=2, d=64,
           qs=256, ks=128, vs=128, causal=1, scale=0.0, dtype=_lib.ATTN_BF16, flags=0)
BWD = dict(q=1 * MB, k=2 * MB, v=3 * MB, out=4 * MB, dout=5 * MB, lse=6 * MB, cu=7 * MB, nseq=3, T=100, longest=60, dq=8 * MB, dk=9 * MB, dv=10 * MB,
           ws=11 * MB, wsb=1 << 19, Hq=4, Hkv=2, d=64, qs=256, ks=128, vs=128, causal=1, scale=0.0, dtype=_lib.ATTN_BF16, flags=0)
PAGED = dict(q=1 * MB, k=2 * MB, v=3 * MB, table=4 * MB, lens=5 * MB, o=6 * MB, lse=7 * MB, ws=8 * MB, wsb=1 << 19, B=2, Hq=4, Hkv=2, Nq=3, M=200,
             pages=20, page=64, longest=0, d=64, causal=1, scale=0.0, dtype=_lib.ATTN_BF16, flags=0)
APPEND = dict(k=1 * MB, v=2 * MB, table=3 * MB, kn=4 * MB, vn=5 * MB, cu=6 * MB, lens=None, B=2, T=9, Hkv=2, M=4, pages=20, page=32, d=64, ks=128,
              vs=128, dtype=_lib.ATTN_BF16)
FREE = dict(table=1 * MB, lens=2 * MB, refs=3 * MB, keep=4 * MB, to=5 * MB, lo=6 * MB, ro=7 * MB, B=4, M=8, pages=40, page=16)
FORK = dict(table=1 * MB, lens=2 * MB, refs=3 * MB, src=4 * MB, dst=5 * MB, to=6 * MB, lo=7 * MB, ro=8 * MB, copies=9 * MB, n=2, B=4, M=8, pages=40,
            page=16)
RESERVE = dict(table=1 * MB, lens=2 * MB, refs=3 * MB, new=4 * MB, to=5 * MB, ro=6 * MB, B=4, M=8, pages=40, page=16)
COMPACT = dict(table=1 * MB, refs=2 * MB, to=3 * MB, ro=4 * MB, copies=5 * MB, used=6 * MB, B=4, M=8, pages=40)
COPY = dict(k=1 * MB, v=2 * MB, copies=3 * MB, n=5, Hkv=2, pages=20, page=32, d=64, dtype=_lib.ATTN_BF16)
CALLS = {"fwd": (_lib.attn_fwd_varlen_gqa, FWD), "bwd": (_lib.attn_bwd_varlen_gqa, BWD), "paged": (_lib.attn_fwd_kvpages, PAGED),
         "append": (_lib.attn_kvpages_append, APPEND), "free": (_lib.attn_kvpages_free, FREE), "fork": (_lib.attn_kvpages_fork, FORK),
         "reserve": (_lib.attn_kvpages_reserve, RESERVE), "compact": (_lib.attn_kvpages_compact, COMPACT), "copy": (_lib.attn_kvpages_copy, COPY)}


def call(name, **kw):
    f, a = CALLS[name]
    assert not set(kw) - set(a)
    return f(*{**a, **kw}.values(), None)


def pointers(name):
    return [x for x, y in CALLS[name][1].items() if isinstance(y, int) and y >= MB or y is None]


OPTIONAL = {"fwd": {"lse"}, "bwd": set(), "paged": {"lse"}, "append": {"lens"}, "free": set(), "fork": set(), "reserve": set(), "compact": set(), "copy": set()}


@pytest.mark.parametrize("name", list(CALLS))
def test_pointers(lib, name):
    """Null and misaligned pointers."""
    for p in pointers(name):
        at = CALLS[name][1][p] or 50 * MB
        if p not in OPTIONAL[name]:
            assert call(name, **{p: None}) == BAD, p
        assert call(name, **{p: at + 2}) == BAD, p


@pytest.mark.parametrize("name,wrong", [
    ("fwd", [dict(nseq=-1), dict(T=-1), dict(longest=-1), dict(longest=0), dict(nseq=0), dict(Hq=3), dict(Hkv=0), dict(d=0), dict(qs=255), dict(qs=252),
             dict(ks=120), dict(vs=0), dict(qs=-256), dict(ks=132), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(dtype=3),
             dict(flags=2), dict(flags=4), dict(ws=7 * MB + 128), dict(wsb=100), dict(q=1 * MB + 8), dict(out=5 * MB + 8)]),
    ("bwd", [dict(nseq=-1), dict(T=-1), dict(longest=0), dict(Hq=5), dict(qs=248), dict(vs=64), dict(scale=-2.0), dict(flags=4), dict(dtype=-1),
             dict(wsb=1000), dict(dk=9 * MB + 8), dict(dout=5 * MB + 8)]),
    ("paged", [dict(B=-1), dict(Nq=-1), dict(Hq=3), dict(M=-1), dict(pages=-1), dict(page=0), dict(page=48), dict(page=256), dict(longest=-1),
               dict(d=0), dict(scale=-1.0), dict(flags=2), dict(dtype=9), dict(wsb=64), dict(ws=8 * MB + 64), dict(k=2 * MB + 8)]),
    ("append", [dict(B=-1), dict(T=-1), dict(Hkv=0), dict(M=0), dict(B=0), dict(pages=0), dict(page=8), dict(ks=64), dict(vs=132), dict(dtype=4), dict(d=0)]),
    ("free", [dict(B=-1), dict(M=-1), dict(pages=-1), dict(page=24)]),
    ("fork", [dict(n=-1), dict(B=-1), dict(page=1), dict(copies=9 * MB + 4)]),
    ("reserve", [dict(B=-1), dict(pages=-3), dict(page=512)]),
    ("compact", [dict(B=-1), dict(M=-1), dict(pages=-1), dict(copies=5 * MB + 4)]),
    ("copy", [dict(n=-1), dict(Hkv=0), dict(pages=-1), dict(page=100), dict(dtype=5), dict(d=-16), dict(k=1 * MB + 8)])])
def test_arguments(lib, name, wrong):
    for kw in wrong:
        assert call(name, **kw) == BAD, kw


@pytest.mark.parametrize("name,much", [
    ("fwd", [dict(d=24), dict(d=144, qs=1024, ks=1024, vs=1024), dict(nseq=65536), dict(longest=2 ** 31 - 1), dict(T=2 ** 30, longest=60),
             dict(qs=1 << 37)]),
    ("bwd", [dict(d=40), dict(nseq=70000), dict(T=2 ** 30)]),
    ("paged", [dict(d=24), dict(d=256), dict(M=2 ** 25, page=128), dict(pages=2 ** 30), dict(B=2 ** 24, M=200), dict(Nq=2 ** 30)]),
    ("append", [dict(d=24), dict(M=2 ** 28), dict(pages=2 ** 30), dict(T=2 ** 31 - 1)]),
    ("free", [dict(B=65537), dict(M=2 ** 28), dict(pages=2 ** 31 - 1)]), ("fork", [dict(n=65537), dict(B=70000)]), ("reserve", [dict(B=65537)]),
    ("compact", [dict(B=65537), dict(pages=2 ** 31 - 1)]), ("copy", [dict(d=72), dict(pages=2 ** 30)])])
def test_sizes(lib, name, much):
    for kw in much:
        assert call(name, **kw) == NO, kw


def test_nothing_to_do(lib):
    assert call("fwd", T=0, q=None, out=None, ws=None) == OK and call("fwd", T=0, nseq=0, cu=None) == OK
    assert call("bwd", T=0, q=None, ws=None) == OK
    assert call("paged", B=0) == OK and call("paged", Nq=0, ws=None) == OK
    assert call("append", T=0, k=None) == OK and call("copy", n=0, copies=None) == OK
    assert call("free", B=0, pages=0, table=None, refs=None, to=None, ro=None, lens=None, lo=None, keep=None) == OK


def test_workspaces(lib):
    f, b, p = _lib.attn_fwd_varlen_gqa_workspace_bytes, _lib.attn_bwd_varlen_gqa_workspace_bytes, _lib.attn_fwd_kvpages_workspace_bytes
    assert f(3, 1000, 500, 8, 2) % 256 == 0 and f(3, 1000, 500, 8, 2) >= 256 + 16 * (1000 // 128)
    # a list for every tile that there may be: a sequence's last one is not full, and long ones take whole levels
    assert f(60000, 60000, 9, 8, 2) >= 16 * 60000
    assert f(1, 10 ** 6, 10 ** 6, 16, 1) >= 16 * (10 ** 6 // 8)
    assert b(3, 1000, 500, 8, 2, 64) > _lib.attn_bwd_workspace_bytes(1, 8, 1000, 64)
    for bad in ((0, 10, 5, 4, 2), (2, 0, 5, 4, 2), (2, 10, 0, 4, 2), (2, 10, 5, 4, 3), (2, 10, 5, 0, 2)):
        assert f(*bad) == 0 and b(*bad, 64) == 0
    assert p(1, 8, 2, 1, 10, 64, 0, 128, 2) == 0       # a cluster per head joins its parts on chip
    assert p(8, 32, 8, 1, 512, 64, 0, 128, 2) > 0
    assert p(8, 32, 8, 1, 512, 64, 640, 128, 2) == 0   # planned for short ones
    assert p(2, 8, 2, 100, 100, 64, 0, 64, 0) > 0      # fp32
    for bad in ((0, 8, 2, 1, 10, 64, 0, 64, 2), (1, 8, 3, 1, 10, 64, 0, 64, 2), (1, 8, 2, 0, 10, 64, 0, 64, 2), (1, 8, 2, 1, -1, 64, 0, 64, 2),
                (1, 8, 2, 1, 10, 63, 0, 64, 2), (1, 8, 2, 1, 10, 64, -1, 64, 2), (1, 8, 2, 1, 10, 64, 0, 0, 2), (1, 8, 2, 1, 2 ** 30, 64, 0, 64, 2)):
        assert p(*bad) == 0


# sizes in bytes of the arrays above, outputs first
SPANS = {
    "fwd": (("out", "lse"), dict(out=100 * 256 * 2, lse=100 * 16, q=100 * 256 * 2, k=100 * 128 * 2, v=100 * 128 * 2, cu=16)),
    "bwd": (("dq", "dk", "dv"), dict(dq=100 * 256 * 2, dk=100 * 128 * 2, dv=100 * 128 * 2, q=100 * 256 * 2, k=100 * 128 * 2, v=100 * 128 * 2,
                                     out=100 * 256 * 2, dout=100 * 256 * 2, lse=1600, cu=16)),
    "paged": (("o", "lse"), dict(o=2 * 4 * 3 * 64 * 2, lse=96, q=2 * 4 * 3 * 64 * 2, k=20 * 2 * 64 * 64 * 2, v=20 * 2 * 64 * 64 * 2, table=1600, lens=16)),
    "append": (("k", "v"), dict(k=20 * 2 * 32 * 64 * 2, v=20 * 2 * 32 * 64 * 2, kn=9 * 256, vn=9 * 256, table=32, cu=16)),
    "free": (("to", "lo", "ro"), dict(to=128, lo=16, ro=160, table=128, lens=16, refs=160, keep=16)),
    "fork": (("to", "lo", "ro", "copies"), dict(to=128, lo=16, ro=160, copies=16, table=128, lens=16, refs=160, src=8, dst=8)),
    "reserve": (("to", "ro"), dict(to=128, ro=160, table=128, lens=16, refs=160, new=16)),
    "compact": (("to", "ro", "copies", "used"), dict(to=128, ro=160, copies=160, used=4, table=128, refs=160)),
    "copy": (("k", "v"), dict(k=20 * 2 * 32 * 64 * 2, v=20 * 2 * 32 * 64 * 2, copies=40))}
FOLLOWS = {("to", "table"), ("lo", "lens"), ("ro", "refs")}


@pytest.mark.parametrize("name", list(SPANS))
def test_overlaps(lib, name):
    """Every output on the last bytes of every input and of every other output, and the other way round; an output of the
    books may be the array that it follows, but not a part of it."""
    outs, sizes = SPANS[name]
    ins = [x for x in sizes if x not in outs]
    for a, b in itertools.chain(itertools.combinations(outs, 2), itertools.product(outs, ins)):
        for x, y in ((a, b), (b, a)):
            at = {n: CALLS[name][1][n] + 20 * MB for n in sizes}
            step = (sizes[y] - 1) // 16 * 16
            if step == 0 and ((x, y) in FOLLOWS or (y, x) in FOLLOWS):
                continue
            at[x] = at[y] + step
            assert call(name, **at) == BAD, (x, y)



def test_python_refusals():
    t = torch.zeros(4, 2, 16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        A.fwd_varlen_gqa(t, t, t, i, 4, True)
    with pytest.raises(TypeError):
        A.fwd_varlen_gqa(None, t, t, i, 4, True)
    with pytest.raises(ValueError, match="CUDA"):
        A.bwd_varlen_gqa(t, t, t, t, t, t, i, 4, True)
    x = torch.zeros(1, 2, 3, 16)
    with pytest.raises(ValueError, match="CUDA"):
        A.fwd_kvpages(x, x, x, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        A.kvpages_append(x, x, i[None], t, t, i)
    for f in (lambda: A.kvpages_free(i[None], i, i, i, 16), lambda: A.kvpages_fork(i[None], i, i, i, i, 16),
              lambda: A.kvpages_reserve(i[None], i, i, i, 16), lambda: A.kvpages_compact(i[None], i), lambda: A.kvpages_copy(x, x, i[None])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(TypeError):
        A.kvpages_free([[0]], i, i, i, 16)


def test_the_bounds_notice_a_wrong_tile():
    """16 keys left out of 1500, a value taken from its neighbour, a gradient without one query: all outside the bounds."""
    g = torch.Generator().manual_seed(0)
    G, Nq, L, d = 2, 3, 1500, 64
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((G, Nq, d), (L, d), (L, d)))
    o, lse, p, size = P.attend(q, k, v, L - Nq, True)
    for rho, half in ((P.HALF[torch.bfloat16], 2.0 ** -24), (2.0 ** -15, 2.0 ** -24), (P.HALF[torch.float16], P.HALF[torch.float16])):
        bo, be = P.attend_bounds(v, p, size, o, d, rho, half)
        keep = torch.ones(L, dtype=torch.bool)
        keep[700:716] = False
        o2, lse2, _, _ = P.attend(q, k[keep], v[keep], L - 16 - Nq, True)
        assert ((o2 - o).abs() > bo).any() and ((lse2 - lse).abs() > be).any()
        v2 = v.clone()
        v2[700:716] = v[684:700]
        o3 = P.attend(q, k, v2, L - Nq, True)[0]
        assert ((o3 - o).abs() > bo).any()
    do = torch.randn(G, L, d, generator=g, dtype=torch.float64)
    q = torch.randn(G, L, d, generator=g, dtype=torch.float64)
    h = P.HALF[torch.bfloat16]
    want, bounds = P.grads(q, k, v, do, 0, True, h, h, h ** 2 * 2)
    do2 = do.clone()
    do2[1, 900] = 0
    got, _ = P.grads(q, k, v, do2, 0, True, h, h, h ** 2 * 2)
    for w, y, b in zip(want, got, bounds):
        assert ((w - y).abs() > b).any()


def test_the_plain_books():
    """The plain implementation's own arithmetic on a state that is checked by hand."""
    table, lens, refs = [[4, 1, -1], [4, 6, -1], [-1, -1, -1]], [20, 32, 0], [0, 1, 0, 0, 2, 0, 1]
    t, n, r, bad = P.free(table, lens, refs, [0, 16, 5], 16)
    assert (t, n, r, bad) == ([[-1, -1, -1], [4, -1, -1], [-1, -1, -1]], [0, 16, 0], [0, 0, 0, 0, 1, 0, 0], False)
    t, n, r, c, bad = P.fork(table, lens, refs, [0], [2], 16)
    assert (t[2], n[2], r, c, bad) == ([4, 0, -1], 20, [1, 1, 0, 0, 3, 0, 1], [[1, 0]], False)
    t, r, bad = P.reserve(table, lens, refs, [12, 1, 17], 16)
    assert (t, r, bad) == ([[4, 1, -1], [4, 6, 0], [2, 3, -1]], [1, 1, 1, 1, 2, 0, 1], False)
    t, r, c, U, bad = P.compact(table, refs)
    assert (t, r, c, U, bad) == ([[0, 1, -1], [0, 2, -1], [-1, -1, -1]], [2, 1, 1, 0, 0, 0, 0], [[4, 0], [6, 2], [-1, -1]], 3, False)

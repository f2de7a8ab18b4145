"""Host-side refusals of the cache calls where an output lies over an input or over another output."""
import itertools

import pytest

from exact_attention_50_gb300 import _lib, build

MB = 1 << 20
BAD = _lib.ATTN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def apart(names):
    return {n: (i + 1) * MB for i, n in enumerate(names)}


def over(sizes, outs, ins):
    """Every output on the last 16 bytes of every input and of every other output, and the other way round."""
    for a, b in itertools.chain(itertools.combinations(outs, 2), itertools.product(outs, ins)):
        for x, y in ((a, b), (b, a)):
            at = apart(sizes)
            at[x] = at[y] + (sizes[y] - 1) // 16 * 16
            yield (x, y), at


def test_append(lib):
    B, H, Nn, Nk, d, block = 4, 2, 4, 100, 64, 64
    codes, scales, new = B * H * Nk * d, B * H * 2 * 4, B * H * Nn * d * 2
    sizes = dict(k8=codes, v8=codes, ks=scales, vs=scales, k=new, v=new, lens=16, new=16)
    for what, a in over(sizes, ("k8", "v8", "ks", "vs"), ("k", "v", "lens", "new")):
        st = _lib.attn_kvcache8_append(a["k8"], a["v8"], a["ks"], a["vs"], a["k"], a["v"], a["lens"], a["new"], B, H, Nn, Nk, d,
                                       block, _lib.ATTN_BF16, _lib.ATTN_CACHE_I8, None)
        assert st == BAD, what


@pytest.mark.parametrize("Nq", [3, 0])
def test_weights(lib, Nq):
    B, Hq, H, Nk, d = 4, 4, 2, 100, 64
    sizes = dict(out=B * H * Nk * 4, w=B * H * Nk * 4, lens=16, k=B * H * Nk * d * 2)
    if Nq:
        sizes.update(q=B * Hq * Nq * d * 2, lse=B * Hq * Nq * 4)
    for what, a in over(sizes, ("out",), [n for n in sizes if n != "out"]):
        st = _lib.attn_kvcache_weights(a.get("q", 50 * MB), a["k"], a.get("lse", 51 * MB), a["lens"], a["w"], a["out"], B, Hq, H, Nq, Nk, d, 1,
                                       0.0, _lib.ATTN_BF16, None)
        assert st == BAD, what


def test_evict(lib):
    B, H, Nk, cap, d, keep, recent = 4, 2, 100, 40, 64, 24, 16
    cache, out = B * H * Nk * d * 2, B * H * cap * d * 2
    sizes = dict(k=cache, v=cache, w=B * H * Nk * 4, lens=16, ko=out, vo=out, wo=B * H * cap * 4, idx=B * H * 40 * 4, lo=16)
    for what, a in over(sizes, ("ko", "vo", "wo", "idx", "lo"), ("k", "v", "w", "lens")):
        st = _lib.attn_kvcache_evict(a["k"], a["v"], a["w"], a["lens"], a["ko"], a["vo"], a["wo"], a["idx"], a["lo"], B, H, Nk, cap, d,
                                     keep, recent, _lib.ATTN_BF16, None)
        assert st == BAD, what

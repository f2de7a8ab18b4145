"""Host-side checks of the 8-bit cache and eviction calls that need no GPU: argument refusals at
the C ABI (before anything is launched) and in the Python layer, workspace sizes, and the plain
implementations that the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import cache_plain as P

BAD, NO, OK = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_append_refusals(lib):
    def f(**kw):
        a = dict(k8=4096, v8=8192, ks=4096, vs=4096, k=4096, v=4096, lens=None, new=None, B=2, Hkv=2, Nn=4, Nk=100, d=64,
                 block=64, dtype=_lib.ATTN_BF16, cache=_lib.ATTN_CACHE_I8)
        a.update(kw)
        return _lib.attn_kvcache8_append(a["k8"], a["v8"], a["ks"], a["vs"], a["k"], a["v"], a["lens"], a["new"], a["B"],
                                         a["Hkv"], a["Nn"], a["Nk"], a["d"], a["block"], a["dtype"], a["cache"], None)
    assert f(B=0) == OK and f(Nn=0) == OK
    for kw in (dict(B=-1), dict(Hkv=0), dict(Nn=-1), dict(Nk=-1), dict(Nn=101), dict(d=0), dict(block=0), dict(block=48),
               dict(block=256), dict(dtype=7), dict(cache=2), dict(k8=None), dict(v8=4100), dict(ks=None), dict(vs=4098),
               dict(k=4104), dict(v=None), dict(lens=4098), dict(new=4098)):
        assert f(**kw) == BAD, kw
    for kw in (dict(d=24), dict(d=144), dict(B=1 << 30, Hkv=1 << 10), dict(B=1 << 20, Hkv=1 << 10, block=16)):
        assert f(**kw) == NO, kw


def test_attend_refusals_and_workspace(lib):
    ws = _lib.attn_fwd_kvcache8_workspace_bytes(2, 4, 2, 3, 100000, 64)
    assert ws >= 256 and ws % 256 == 0
    assert _lib.attn_fwd_kvcache8_workspace_bytes(2, 4, 2, 3, 100, 64) == 0  # a cluster per head joins its parts on chip
    # many rows: K and V in 16 bits, and what the key ranges leave
    assert _lib.attn_fwd_kvcache8_workspace_bytes(2, 4, 2, 300, 1000, 64) >= 2 * 2 * 2 * 1000 * 64 * 2
    for bad in ((0, 4, 2, 3, 1000, 64), (2, 3, 2, 3, 1000, 64), (2, 4, 2, 0, 1000, 64), (2, 4, 2, 3, -1, 64), (2, 4, 2, 3, 9, 0)):
        assert _lib.attn_fwd_kvcache8_workspace_bytes(*bad) == 0

    def f(**kw):
        a = dict(q=4096, k8=4096, v8=4096, ks=4096, vs=4096, lens=None, o=4096, lse=None, ws=4096, wsb=ws, B=2, Hq=4, Hkv=2,
                 Nq=3, Nk=100000, d=64, block=64, causal=1, scale=0.0, dtype=_lib.ATTN_BF16, cache=_lib.ATTN_CACHE_I8, flags=0)
        a.update(kw)
        return _lib.attn_fwd_kvcache8(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], a["lens"], a["o"], a["lse"], a["ws"],
                                      a["wsb"], a["B"], a["Hq"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["block"],
                                      a["causal"], a["scale"], a["dtype"], a["cache"], a["flags"], None)
    assert f(B=0) == OK and f(Nq=0) == OK
    for kw in (dict(q=None), dict(o=None), dict(k8=None), dict(v8=None), dict(ks=None), dict(vs=None), dict(q=4104),
               dict(k8=4104), dict(ks=4098), dict(lse=4098), dict(lens=4098), dict(ws=None), dict(ws=4224), dict(wsb=ws - 1),
               dict(Hq=3), dict(Nk=-1), dict(Nq=-1), dict(block=8), dict(scale=-1.0), dict(scale=math.nan), dict(flags=2),
               dict(cache=5), dict(dtype=9), dict(d=0)):
        assert f(**kw) == BAD, kw
    for kw in (dict(d=40), dict(d=256), dict(dtype=_lib.ATTN_F32)):
        assert f(**kw) == NO, kw


def test_weights_refusals(lib):
    def f(**kw):
        a = dict(q=4096, k=4096, lse=4096, lens=None, w=None, out=4096, B=2, Hq=4, Hkv=2, Nq=3, Nk=100, d=64, causal=1,
                 scale=0.0, dtype=_lib.ATTN_BF16)
        a.update(kw)
        return _lib.attn_kvcache_weights(a["q"], a["k"], a["lse"], a["lens"], a["w"], a["out"], a["B"], a["Hq"], a["Hkv"],
                                         a["Nq"], a["Nk"], a["d"], a["causal"], a["scale"], a["dtype"], None)
    assert f(B=0) == OK and f(Nk=0) == OK
    for kw in (dict(q=None), dict(k=None), dict(lse=None), dict(out=None), dict(q=4104), dict(k=4104), dict(lse=4098),
               dict(out=4098), dict(w=4098), dict(lens=4098), dict(Hq=3), dict(Nq=-1), dict(Nk=-1), dict(scale=-1.0),
               dict(dtype=3), dict(d=-16)):
        assert f(**kw) == BAD, kw
    assert f(d=72) == NO and f(d=144) == NO


def test_evict_refusals(lib):
    MB = 1 << 20

    def f(**kw):
        a = dict(k=MB, v=2 * MB, w=3 * MB, lens=None, ko=4 * MB, vo=5 * MB, wo=6 * MB, idx=7 * MB, lo=8 * MB, B=2, Hkv=2, Nk=100,
                 cap=40, d=64, keep=24, recent=16, dtype=_lib.ATTN_BF16)
        a.update(kw)
        return _lib.attn_kvcache_evict(a["k"], a["v"], a["w"], a["lens"], a["ko"], a["vo"], a["wo"], a["idx"], a["lo"],
                                       a["B"], a["Hkv"], a["Nk"], a["cap"], a["d"], a["keep"], a["recent"], a["dtype"], None)
    assert f(B=0) == OK
    for kw in (dict(k=None), dict(v=None), dict(w=None), dict(ko=None), dict(vo=None), dict(wo=None), dict(idx=None),
               dict(lo=None), dict(k=MB + 8), dict(ko=4 * MB + 8), dict(w=3 * MB + 2), dict(lens=4098), dict(keep=-1),
               dict(recent=-1), dict(keep=0, recent=0), dict(cap=39), dict(B=-1), dict(Nk=-1), dict(dtype=4),
               dict(ko=MB), dict(vo=2 * MB + 256), dict(ko=5 * MB), dict(wo=3 * MB + 400)):
        assert f(**kw) == BAD, kw
    assert f(d=20) == NO
    assert f(keep=2 ** 31 - 1, recent=2 ** 31 - 1) == BAD  # their sum does not wrap


def test_sizes_whose_tile_numbers_leave_32_bits_are_refused(lib):
    """Lengths and row counts are rounded up to tiles and stepped over in 32 bits on the device."""
    MB, big = 1 << 20, 0x7fff0001
    assert _lib.attn_kvcache8_append(MB, 1 << 50, 1 << 51, 1 << 52, MB, MB, None, None, 1, 1, 1, big, 16, 64, _lib.ATTN_BF16, 0, None) == NO
    for Nq in (1, 100):
        assert _lib.attn_fwd_kvcache8(MB, MB, MB, MB, MB, None, MB, None, MB, 1 << 60, 1, 1, 1, Nq, big, 16, 64, 1, 0.0,
                                      _lib.ATTN_BF16, 0, 0, None) == NO
    assert _lib.attn_fwd_kvcache8(MB, MB, MB, MB, MB, None, MB, None, MB, 1 << 60, 1, 1, 1, big, 64, 16, 64, 1, 0.0,
                                  _lib.ATTN_BF16, 0, 0, None) == NO
    for dtype in (_lib.ATTN_BF16, _lib.ATTN_F32):
        for Nq, Nk in ((1, big), (big, 64)):
            assert _lib.attn_kvcache_weights(MB, MB, MB, None, None, 1 << 50, 1, 1, 1, Nq, Nk, 16, 1, 0.0, dtype, None) == NO
    for Nk, cap, keep in ((big, 40, 24), (100, big, 24), (100, big, big - 1)):
        assert _lib.attn_kvcache_evict(MB, 1 << 42, 1 << 44, None, 1 << 46, 1 << 48, 1 << 50, 1 << 52, 1 << 54, 1, 1, Nk, cap,
                                       16, keep, 1, _lib.ATTN_BF16, None) == NO


def test_outputs_that_overlap_what_is_read_are_refused(lib):
    MB = 1 << 20

    def append(**kw):
        a = dict(k8=MB, v8=2 * MB, ks=3 * MB, vs=4 * MB)
        a.update(kw)
        return _lib.attn_kvcache8_append(a["k8"], a["v8"], a["ks"], a["vs"], 5 * MB, 6 * MB, None, None, 2, 2, 4, 100, 64, 64,
                                         _lib.ATTN_BF16, _lib.ATTN_CACHE_I8, None)
    for kw in (dict(v8=MB), dict(v8=MB + 25584), dict(vs=3 * MB), dict(vs=3 * MB + 28)):
        assert append(**kw) == BAD, kw

    def weights(out, w=4 * MB, Nq=3):
        return _lib.attn_kvcache_weights(MB, 2 * MB, 3 * MB, None, w, out, 2, 4, 2, Nq, 100, 64, 1, 0.0, _lib.ATTN_BF16, None)
    for Nq in (3, 0):
        assert weights(4 * MB + 4, Nq=Nq) == BAD and weights(4 * MB - 1596, Nq=Nq) == BAD
    assert weights(3 * MB) == BAD and weights(3 * MB - 4, None) == BAD
    for lo in (9 * MB, 9 * MB + 4):  # the new lengths over the old ones, which other heads still read
        assert _lib.attn_kvcache_evict(MB, 2 * MB, 3 * MB, 9 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, lo, 2, 2, 100, 40, 64, 24, 16,
                                       _lib.ATTN_BF16, None) == BAD


def test_the_python_layer_refuses_sizes_that_c_would_cut(lib):
    A._check_sizes((1, 2, 2 ** 31 - 1), (4,))
    with pytest.raises(ValueError, match="2\\*\\*31"):
        A._check_sizes((1, 2), (1, 2 ** 31, 16))


def test_python_layer_wants_cuda_tensors_of_the_right_kind():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    k8 = torch.zeros(1, 1, 64, 64, dtype=torch.int8)
    s = torch.zeros(1, 1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        A.fwd_kvcache8(q, k8, k8, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        A.kvcache8_append(k8, k8, s, s, q[:, :1], q[:, :1])
    with pytest.raises(ValueError, match="CUDA"):
        A.kvcache_weights(q, q, torch.zeros(1, 2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        A.kvcache_evict(q, q, torch.zeros(1, 2, 1), 1, 0)
    with pytest.raises(TypeError):
        A.kvcache_weights(None, q, q)


@pytest.mark.parametrize("cache", ["i8", "e4m3"])
def test_plain_codes_round_like_torch(cache):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4096, generator=g) * torch.exp(2 * torch.randn(4096, generator=g)) * (20 if cache == "e4m3" else 40)
    x = torch.cat((x, torch.arange(-140, 140) / 2.0, torch.arange(-64, 64) * 2.0 ** -10))
    ours = P.round_code(x.numpy(), cache)
    if cache == "i8":
        ref = torch.round(x).clamp(-127, 127).numpy()
    else:
        ref = x.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ours, ref)


def test_plain_append_is_idempotent_and_bounded():
    """Appending token by token: every value reads back within the steps that its scale's growth
    allows (one half step per recoding), and writing the last token again changes nothing."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((70, 16)) * np.exp(rng.standard_normal((70, 1)))).astype(np.float32)
    codes, scale = np.zeros((70, 16), np.float32), np.full(5, 9e9, np.float32)
    grown = np.zeros(5, int)
    for t in range(70):
        before = scale[t // 16]
        P.append(codes, scale, x[t:t + 1], t, 1, 16, "i8")
        grown[t // 16] += t % 16 > 0 and scale[t // 16] > before
    back = codes * np.repeat(scale, 16)[:70, None]
    steps = np.repeat(scale * (0.5 + 0.5 * grown + 1e-4), 16)[:70, None]
    assert np.all(np.abs(back - x) <= steps)
    again, s2 = codes.copy(), scale.copy()
    P.append(again, s2, x[69:70], 69, 1, 16, "i8")
    assert np.array_equal(again, codes) and np.array_equal(s2, scale)


def test_plain_attend_is_softmax():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, h, n, 16, generator=g, dtype=torch.float64) for h, n in ((4, 3), (2, 20), (2, 20)))
    o, lse, a, _ = P.attend(q, k, v, None, False)
    ref = torch.nn.functional.scaled_dot_product_attention(q, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1))
    assert (o - ref).abs().max() < 1e-13 and bool((a >= o.abs() - 1e-15).all())
    w, _ = P.weights(q, k, lse, None, False, None)
    assert (w.sum(-1) - 6).abs().max() < 1e-12  # two heads of three queries, each of weight one


def test_plain_evict_ties_and_nan():
    w = np.array([1, 5, 5, np.nan, 0, 5, np.inf, 7, 0, 0], np.float32)
    assert P.evict(None, None, w, 10, 3, 2).tolist() == [3, 6, 7, 8, 9]
    assert P.evict(None, None, w, 6, 2, 1).tolist() == [1, 3, 5]
    assert P.evict(None, None, w, 3, 2, 1).tolist() == [0, 1, 2]
    assert P.evict(None, None, w, 10, 0, 4).tolist() == [6, 7, 8, 9]

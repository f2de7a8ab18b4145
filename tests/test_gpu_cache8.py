"""GPU tests of the 8-bit KV cache: codes and scales bit by bit against the definition in single
float32 operations, attention against 64 bits with bounds from the roundings that the kernels
make, and what a serving program does with them (graphs, streams, ragged and padded batches)."""
import numpy as np
import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import cache_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    _lib.load()
    return torch.device("cuda:0")


def rows(seed, shape, dev, dtype=torch.float32):
    """Keys or values with columns and tokens of different magnitude."""
    g = torch.Generator(dev).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(shape[:2] + (1, shape[3]), generator=g, device=dev))
    x *= torch.exp(0.5 * torch.randn(shape[:3] + (1,), generator=g, device=dev))
    return x.to(dtype)


def status_ok():
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_OK


# ------------------------------------------------------------------------------------- append
def values(x8):
    return x8.float().cpu().numpy()


@pytest.mark.parametrize("cache", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 64), ("f16", 64, 32), ("f32", 80, 16), ("bf16", 16, 128), ("f32", 128, 128)])
def test_append_matches_the_definition_bit_by_bit(dev, cache, dtype, d, block):
    """Ragged lengths around the blocks' edges, one batch that appends nothing, one that fills its
    cache; everything outside the touched blocks, and the scales of untouched ones, stays."""
    Nk, Nn = 301, 150
    lens, new = [0, 1, block - 1, block, block + 5, 151, 301, 70], [150, 1, 2, block, 77, 150, 0, 0]
    B, H = len(lens), 3
    k8, v8 = ((torch.randint(-120, 120, (B, H, Nk, d), device=dev).to(torch.int8) if cache == "i8"
               else torch.randn(B, H, Nk, d, device=dev).mul(60).to(torch.float8_e4m3fn)) for _ in range(2))
    nb = -(-Nk // block)
    ks, vs = (torch.rand(B, H, nb, device=dev) * (0.02 if cache == "i8" else 0.005) for _ in range(2))
    kn, vn = (rows(i, (B, H, Nn, d), dev, DT[dtype]) for i in (1, 2))
    kn[4, 1] *= 0.001   # a block's present scale stays
    vn[3] = 0           # a block of zeros: scale 0
    vn[1] *= 1e-38 if dtype == "f32" else 1  # scales below the smallest normal number
    want = []
    for x8, s, x in ((k8, ks, kn), (v8, vs, vn)):
        c, sc, xn = values(x8), s.cpu().numpy().copy(), x.float().cpu().numpy()
        for b in range(B):
            for h in range(H):
                P.append(c[b, h], sc[b, h], xn[b, h], lens[b], new[b], block, cache)
        want.append((c, sc))
    cl, nl = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (lens, new))
    for _ in range(2):  # the second time changes nothing
        A.kvcache8_append(k8, v8, ks, vs, kn, vn, cl, nl, block=block)
        status_ok()
        for x8, s, (c, sc) in ((k8, ks, want[0]), (v8, vs, want[1])):
            assert np.array_equal(s.cpu().numpy(), sc)
            assert np.array_equal(values(x8), c)


def test_append_defaults_empty_cache_and_whole_lengths(dev):
    kn, vn = (rows(i, (2, 2, 40, 64), dev, torch.bfloat16) for i in (3, 4))
    k8, v8 = (torch.zeros(2, 2, 64, 64, dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.full((2, 2, 1), float("nan"), device=dev) for _ in range(2))  # never read
    A.kvcache8_append(k8, v8, ks, vs, kn, vn)
    status_ok()
    c, s = P.quantise(torch.nn.functional.pad(kn.float(), (0, 0, 0, 24)), 64, "i8")
    assert float((ks - s).abs().max() / s.max()) < 2.0 ** -22
    assert float((k8.float() - c.float()).abs().max()) <= 1


def test_append_keeps_infinities_and_nan_visible(dev):
    k8, v8 = (torch.zeros(1, 1, 128, 16, dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(1, 1, 2, device=dev) for _ in range(2))
    kn = torch.ones(1, 1, 3, 16, device=dev)
    vn = kn.clone()
    kn[0, 0, 1, 3], vn[0, 0, 2, 0] = float("nan"), float("-inf")
    A.kvcache8_append(k8, v8, ks, vs, kn, vn, torch.tensor([63], dtype=torch.int32, device=dev))
    status_ok()
    assert float(ks[0, 0, 0]) == pytest.approx(1 / 127) and bool(torch.isnan(ks[0, 0, 1])) and bool(torch.isinf(vs[0, 0, 1]))
    # a block that holds a NaN keeps it
    A.kvcache8_append(k8, v8, ks, vs, torch.ones_like(kn), vn, torch.tensor([66], dtype=torch.int32, device=dev))
    status_ok()
    assert bool(torch.isnan(ks[0, 0, 1]))


@pytest.mark.parametrize("lens,new", [([100, 10], [4, 1]), ([-1, 10], [1, 1]), ([5, 10], [-1, 1]), ([5, 10], [5, 1]),
                                      ([2 ** 31 - 1, 10], [4, 1])])
def test_append_reports_bad_lengths_and_leaves_the_batch(dev, lens, new):
    k8, v8 = (torch.full((2, 2, 103, 32), 7, dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.full((2, 2, 4), 0.5, device=dev) for _ in range(2))
    x = torch.full((2, 2, 4, 32), 200.0, device=dev)
    cl, nl = (torch.tensor(t, dtype=torch.int32, device=dev) for t in (lens, new))
    A.kvcache8_append(k8, v8, ks, vs, x, x, cl, nl, block=32)
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_ERR_DEVICE_INPUT and A.get_device_status() == _lib.ATTN_OK
    assert bool((k8[0] == 7).all()) and bool((v8[0] == 7).all()) and bool((ks[0] == 0.5).all())
    assert bool((k8[1, :, 10] == 127).all()) and bool((k8[1, :, 11:] == 7).all())


# ------------------------------------------------------------------------------------- attend
def check_attend(o32, o, lse, q, k8, v8, ks, vs, block, lens, causal, scale=None):
    """o32: with out_f32.  Bounds: the weights, and where the kernel keeps 16-bit copies of the values
    those, are each rounded once to the output's type: 2 u P|V| (u half a step); the scores' float32
    sums give E twice (numerator and denominator), the exponential 2^-18; a weight below the 16-bit
    range is off by at most 2^-24 of the largest value; the stored output adds u |o|."""
    u = P.HALF[q.dtype]
    kd, vd = P.dequantise(k8, ks, block), P.dequantise(v8, vs, block)
    ro, rl, A_, E = P.attend(q, kd, vd, lens, causal, scale)
    top = torch.zeros(q.shape[0], 1, 1, 1, dtype=torch.float64, device=q.device)
    for b in range(q.shape[0]):
        L = k8.shape[2] if lens is None else int(lens[b])
        if L:
            top[b] = vd[b, :, :L].abs().max() * L * 2.0 ** -24
    bound = A_ * (2 * u + 2 * E[..., None] + 2.0 ** -18) + top
    assert bool(torch.isfinite(o32).all())
    assert bool(((o32.double() - ro).abs() <= bound).all()), float(((o32.double() - ro).abs() - bound).max())
    assert bool(((o.double() - ro).abs() <= bound + u * (ro.abs() + bound) + 2.0 ** -24).all())
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((o32[empty] == 0).all())
    err = (lse.double() - rl).abs().masked_fill(empty, 0)
    assert bool((err <= E + 2.0 ** -18 + rl.abs().masked_fill(empty, 0) * 2.0 ** -22).all()), float(err.max())


def run_attend(dev, B, Hq, Hkv, Nq, Nk, d, block, dtype, cache, lens, causal, seed, poison=True, scale=None):
    q = torch.randn(B, Hq, Nq, d, generator=torch.Generator(dev).manual_seed(seed), device=dev).to(DT[dtype])
    k8, ks = P.quantise(rows(seed + 1, (B, Hkv, Nk, d), dev), block, cache)
    v8, vs = P.quantise(rows(seed + 2, (B, Hkv, Nk, d), dev), block, cache)
    cl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    if poison and lens is not None:  # what lies behind a length may hold anything
        for b, L in enumerate(lens):
            for x8 in (k8, v8):
                x8.view(torch.uint8)[b, :, L:] = 0x7f  # 127, or e4m3's NaN
            first = -(-L // block)
            ks[b, :, first:], vs[b, :, first:] = float("nan"), float("inf")
    o32, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, scale, block, out_f32=True)
    o, lse2 = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, scale, block)
    status_ok()
    assert torch.equal(lse, lse2)
    check_attend(o32, o, lse, q, k8, v8, ks, vs, block, lens, causal, scale)
    return q, k8, v8, ks, vs, cl, o


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,cache,d,block", [("bf16", "i8", 128, 64), ("f16", "e4m3", 64, 32), ("bf16", "e4m3", 128, 128),
                                                 ("f16", "i8", 80, 16), ("bf16", "i8", 16, 64), ("f16", "i8", 48, 128)])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (4, 4, 1), (8, 1, 2), (6, 2, 5), (16, 2, 5), (4, 1, 37), (8, 2, 130)])
def test_attend_ragged(dev, causal, dtype, cache, d, block, Hq, Hkv, Nq):
    """Row counts of 1 to 520 per kv head; caches that are empty, of one token, shorter than the
    queries, ending inside a block or a tile, and full."""
    run_attend(dev, 7, Hq, Hkv, Nq, 700, d, block, dtype, cache, [700, 333, 64, 3, 1, 0, 513], causal, seed=Nq)


@pytest.mark.parametrize("Nk", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1025, 5000])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 1, 1), (2, 2, 9), (32, 1, 8)])
def test_attend_lengths(dev, Nk, Hq, Hkv, Nq):
    run_attend(dev, 2, Hq, Hkv, Nq, Nk, 128, 64, "bf16", "i8", None, True, seed=Nk)
    run_attend(dev, 2, Hq, Hkv, Nq, Nk, 64, 16, "f16", "e4m3", [Nk, Nk // 2], True, seed=Nk)


@pytest.mark.parametrize("cache", ["i8", "e4m3"])
@pytest.mark.parametrize("Nq,Nk", [(300, 300), (1000, 2500), (129, 4100), (700, 130)])
def test_attend_prefill(dev, cache, Nq, Nk):
    run_attend(dev, 2, 4, 2, Nq, Nk, 128, 64, "bf16", cache, [Nk, max(1, Nk - 77)], True, seed=5)
    run_attend(dev, 1, 4, 4, Nq, Nk, 64, 16, "f16", cache, None, False, seed=6)


def test_attend_many_rows_on_long_caches(dev):
    """More tokens than the expansion has CTAs for at once."""
    run_attend(dev, 2, 142, 2, 1, 100001, 16, 16, "bf16", "i8", [100001, 80000], False, seed=1)
    run_attend(dev, 3, 16, 4, 20, 40001, 64, 32, "f16", "e4m3", [40001, 1, 39000], True, seed=2)


def test_attend_many_short_sequences(dev):
    lens = [(37 * b) % 130 for b in range(120)]
    run_attend(dev, 120, 8, 4, 1, 130, 128, 64, "bf16", "i8", lens, True, seed=7)
    run_attend(dev, 700, 2, 1, 1, 40, 64, 16, "f16", "e4m3", [(7 * b) % 41 for b in range(700)], True, seed=8)


@pytest.mark.parametrize("cache", ["i8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (33, 1), (64, 1), (71, 1), (128, 1), (142, 2)])
def test_attend_many_heads_share_a_cache(dev, cache, Hq, Hkv):
    """One query each: row blocks that two, four or all warps share, and the kernel of many rows."""
    run_attend(dev, 3, Hq, Hkv, 1, 900, 64, 64, "bf16", cache, [900, 1, 333], True, seed=Hq)
    run_attend(dev, 2, Hq, Hkv, 1, 9000, 112, 16, "f16", cache, [9000, 77], False, seed=Hq)


def test_attend_and_append_with_thousands_of_sequences(dev):
    B = 5000
    lens = [(13 * b) % 34 for b in range(B)]
    q, k8, v8, ks, vs, cl, _ = run_attend(dev, B, 2, 2, 1, 40, 16, 16, "bf16", "i8", lens, True, seed=3, poison=False)
    x = rows(9, (B, 2, 3, 16), dev).bfloat16()
    codes, scales = k8.clone(), ks.clone()
    A.kvcache8_append(k8, v8, ks, vs, x, x, cl, block=16)
    status_ok()
    for b in (0, 1, 2, 33, 1234, 2500, 4097, B - 1):
        for h in range(2):
            c, s = codes[b, h].float().cpu().numpy(), scales[b, h].cpu().numpy()
            P.append(c, s, x[b, h].float().cpu().numpy(), lens[b], 3, 16, "i8")
            assert torch.equal(k8[b, h].float().cpu(), torch.from_numpy(c)) and torch.equal(ks[b, h].cpu(), torch.from_numpy(s))


def test_attend_two_graphs_at_once(dev):
    """Two captured calls, each with its own workspace, replayed on two streams at the same time."""
    calls = []
    for i, (Nq, Nk) in enumerate(((1, 20000), (20, 3000), (100, 2000))):
        q = torch.randn(3, 8, Nq, 128, generator=torch.Generator(dev).manual_seed(i), device=dev).bfloat16()
        k8, ks = P.quantise(rows(i + 1, (3, 2, Nk, 128), dev), 64, "i8")
        v8, vs = P.quantise(rows(i + 2, (3, 2, Nk, 128), dev), 64, "i8")
        want = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True)
        calls.append((g, got, want, torch.cuda.Stream(), (q, k8, v8, ks, vs)))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, got, _, s, _ in calls:
            with torch.cuda.stream(s):
                got[0].zero_()
                g.replay()
    status_ok()
    for _, got, want, _, _ in calls:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("Hq,Nq,block,dtype", [(8, 1, 64, "bf16"), (8, 3, 16, "f16"), (32, 4, 32, "bf16")])
def test_attend_long_caches_of_64_columns(dev, Hq, Nq, block, dtype):
    """Enough tiles for 64 keys each."""
    lens = [30011, 1, 64, 29000, 65, 30011, 7]
    run_attend(dev, 7, Hq, 8, Nq, 30011, 64, block, dtype, "i8", lens, True, seed=Nq)
    run_attend(dev, 7, Hq, 8, Nq, 30011, 48, block, dtype, "e4m3", lens, False, seed=Nq)


@pytest.mark.parametrize("cache,d", [("i8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("Hq,Nq", [(8, 1), (32, 1), (32, 5), (32, 10)])
def test_attend_long_runs_behind_short_sequences(dev, cache, d, Hq, Nq):
    """Many tiles per CTA, long sequences next to sequences of one tile: a CTA's warps take very
    unequal numbers of them, and the ring turns many times."""
    lens = [9000, 1, 1, 40, 12321, 2, 3, 1, 1, 5, 8000]
    q, k8, v8, ks, vs, cl, o = run_attend(dev, len(lens), Hq, 8, Nq, 12321, d, 64, "bf16", cache, lens, True, seed=Nq)
    for _ in range(20):
        assert torch.equal(A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True, None, 64)[0], o)
    status_ok()


@pytest.mark.parametrize("cache", ["i8", "e4m3"])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("dtype,Nq", [("f16", 100), ("bf16", 100), ("f16", 1), ("bf16", 5)])
def test_attend_error_is_that_of_two_roundings_at_most(dev, cache, block, dtype, Nq):
    """Root mean square: the outputs' rounding and that of P, independent and of one size in fp16 (where
    codes add none): sqrt(2) times the former; in bf16 P's, and with many rows V's, are an eighth each.
    A twentieth over that for the sample (102400 outputs at Nq = 100, at least 2048)."""
    k8, ks = P.quantise(rows(1, (2, 2, 3000, 128), dev), block, cache)
    v8, vs = P.quantise(rows(2, (2, 2, 3000, 128), dev), block, cache)
    q = torch.randn(2, 8, Nq, 128, generator=torch.Generator(dev).manual_seed(3), device=dev).to(DT[dtype])
    o, _ = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True, None, block)
    status_ok()
    ro = P.attend(q, P.dequantise(k8, ks, block), P.dequantise(v8, vs, block), None, True, None)[0]
    alone = (ro.to(q.dtype).double() - ro).norm()
    assert float((o.double() - ro).norm() / alone) <= 1.05 * (2 ** 0.5 if dtype == "f16" else (1 + 2 / 64) ** 0.5)


@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_many_rows_scales_of_very_different_size(dev, block, dtype):
    """Values' scales over 2^-20 .. 1, some of them and a key's 0."""
    k8, ks = P.quantise(rows(1, (2, 2, 1500, 64), dev), block, "i8")
    v8, vs = P.quantise(rows(2, (2, 2, 1500, 64), dev), block, "i8")
    vs = vs * torch.exp2(-(torch.arange(vs.shape[2], device=dev) * 7 % 21).float())
    vs[:, :, 3], vs[0, 0, 5], ks[:, :, 4] = 0, 0, 0
    q = torch.randn(2, 8, 60, 64, generator=torch.Generator(dev).manual_seed(3), device=dev).to(DT[dtype])
    cl = torch.tensor([1500, 1111], dtype=torch.int32, device=dev)
    for causal in (True, False):
        o32, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, None, block, out_f32=True)
        o, _ = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, None, block)
        status_ok()
        check_attend(o32, o, lse, q, k8, v8, ks, vs, block, [1500, 1111], causal)
    none = torch.zeros_like(vs)
    o, _ = A.fwd_kvcache8(q, k8, v8, ks, none, cl, True, None, block)
    status_ok()
    assert bool((o == 0).all())


def test_attend_scales_of_very_different_size(dev):
    """Blocks whose value scales lie many powers of two apart, the weights concentrated on the
    small ones and on the large ones; a block of zeros; rows of large and of tiny queries."""
    B, H, Nk, d, block = 2, 2, 512, 64, 16
    for dtype in ("bf16", "f16"):
        q = torch.randn(B, H, 3, d, device=dev)
        q[:, :, 1] *= 20.0
        q[:, :, 2] *= 1e-4
        q = q.to(DT[dtype])
        k8, ks = P.quantise(rows(11, (B, H, Nk, d), dev), block, "i8")
        v8, vs = P.quantise(rows(12, (B, H, Nk, d), dev), block, "i8")
        vs *= torch.exp2(torch.arange(vs.shape[2], device=dev) % 14 - 13.0)
        vs[:, :, 5] = 0
        ks[:, :, 9] = 0
        o32, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, None, False, None, block, out_f32=True)
        o, _ = A.fwd_kvcache8(q, k8, v8, ks, vs, None, False, None, block)
        status_ok()
        check_attend(o32, o, lse, q, k8, v8, ks, vs, block, None, False)


def test_attend_scale_argument_and_without_lse(dev):
    q, k8, v8, ks, vs, cl, o = run_attend(dev, 2, 4, 2, 3, 200, 64, 64, "bf16", "i8", [200, 90], True, 8, scale=0.3)
    o2, none = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True, 0.3, 64, with_lse=False)
    assert none is None and torch.equal(o, o2)


def test_attend_empty_cache_and_no_queries(dev):
    q = torch.randn(2, 4, 3, 64, device=dev).bfloat16()
    k8, s = torch.zeros(2, 2, 0, 64, dtype=torch.int8, device=dev), torch.zeros(2, 2, 0, device=dev)
    o, lse = A.fwd_kvcache8(q, k8, k8, s, s)
    assert torch.count_nonzero(o).item() == 0 and bool(torch.isneginf(lse).all())
    o, lse = A.fwd_kvcache8(q[:, :, :0].contiguous(), k8, k8, s, s)
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    status_ok()


@pytest.mark.parametrize("Nq", [1, 200])
def test_attend_reports_bad_lengths(dev, Nq):
    q = torch.randn(2, 4, Nq, 64, device=dev).bfloat16()
    k8 = torch.ones(2, 2, 300, 64, dtype=torch.int8, device=dev)
    s = torch.ones(2, 2, 5, device=dev)
    for bad in (301, -1):
        o, lse = A.fwd_kvcache8(q, k8, k8, s, s, torch.tensor([100, bad], dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        assert A.get_device_status() == _lib.ATTN_ERR_DEVICE_INPUT and A.get_device_status() == _lib.ATTN_OK
        assert bool(torch.isneginf(lse[1]).all()) and bool((o[1] == 0).all()) and bool((o[0] == 1).all())


@pytest.mark.parametrize("Nq,Nk", [(1, 2000), (1, 30000), (100, 2000)])
def test_attend_in_graphs_and_on_other_streams(dev, Nq, Nk):
    """Captured once and replayed with other lengths and other codes; two streams at a time, each
    call with its own workspace; a caller's workspace."""
    B, Hq, Hkv, d = 3, 8, 2, 128
    q = torch.randn(B, Hq, Nq, d, device=dev).bfloat16()
    k8, ks = P.quantise(rows(21, (B, Hkv, Nk, d), dev), 64, "i8")
    v8, vs = P.quantise(rows(22, (B, Hkv, Nk, d), dev), 64, "i8")
    cl = torch.tensor([Nk, 700, 1], dtype=torch.int32, device=dev)
    ws = torch.empty(max(1, A.kvcache8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)), dtype=torch.uint8, device=dev)
    A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True, workspace=ws)
    for lens in ([Nk, 700, 1], [5, Nk - 1, 0], [64, 65, 1500]):
        cl.copy_(torch.tensor(lens, dtype=torch.int32))
        v8.neg_()
        ws.fill_(255)  # what it holds does not matter
        graph.replay()
        want, wl = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(A.fwd_kvcache8(q, k8, v8, ks, vs, cl, True)[0])
    torch.cuda.synchronize()
    for x in outs:
        assert torch.equal(x, want)
    status_ok()


def test_attend_refusals_of_the_python_layer(dev):
    q = torch.randn(2, 4, 1, 64, device=dev).bfloat16()
    k8 = torch.ones(2, 2, 128, 64, dtype=torch.int8, device=dev)
    s = torch.ones(2, 2, 2, device=dev)
    cl = torch.tensor([1, 2], dtype=torch.int32, device=dev)
    ok = lambda **kw: A.fwd_kvcache8(**{**dict(q=q, k8=k8, v8=k8, k_scale=s, v_scale=s, cache_seqlens=cl), **kw})
    ok()
    for kw in (dict(q=q[:1]), dict(q=q[:, :3].contiguous()), dict(k8=k8[..., :32]), dict(v8=k8[:, :1].contiguous()), dict(block=48),
               dict(block=32), dict(k_scale=s[:, :, :1].contiguous()), dict(cache_seqlens=cl[:1]), dict(cache_seqlens=cl.cpu()),
               dict(scale=-1.0), dict(q=q.transpose(1, 2))):
        with pytest.raises((ValueError, _lib.AttnError)):
            ok(**kw)
    big, sb = torch.ones(2, 2, 20000, 64, dtype=torch.int8, device=dev), torch.ones(2, 2, 313, device=dev)
    need = A.kvcache8_workspace_bytes(2, 4, 2, 1, 20000, 64)
    assert need > 0
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device=dev), torch.empty(need + 256, dtype=torch.uint8, device=dev)[128:]):
        with pytest.raises(_lib.AttnError):
            ok(k8=big, v8=big, k_scale=sb, v_scale=sb, workspace=ws)
    assert A.kvcache8_workspace_bytes(2, 4, 2, 1, 128, 64) == 0  # small: none is used
    ok(workspace=torch.empty(8, dtype=torch.uint8, device=dev))
    for kw in (dict(k8=k8.float()), dict(v8=k8.to(torch.float8_e4m3fn)), dict(k_scale=s.half()), dict(cache_seqlens=cl.long())):
        with pytest.raises(TypeError):
            ok(**kw)
    with pytest.raises(_lib.AttnError):
        ok(q=q.float())
    x = torch.ones(2, 2, 3, 64, device=dev)
    for kw in (dict(k_new=x[:, :1].contiguous()), dict(k_new=torch.ones(2, 2, 129, 64, device=dev), v_new=torch.ones(2, 2, 129, 64, device=dev)),
               dict(new_seqlens=cl[:1])):
        with pytest.raises((ValueError, _lib.AttnError)):
            A.kvcache8_append(**{**dict(k8=k8, v8=k8.clone(), k_scale=s, v_scale=s.clone(), k_new=x, v_new=x), **kw})
    status_ok()


def test_offsets_past_32_bits(dev):
    """A cache of more than 2^32 bytes per tensor: the last sequence's codes are found and written."""
    B, Nk, d = 3, 2 ** 23 * 3 // 2 + 100, 128  # 12.6 M tokens: 1.6 GB of codes each, the last from 3.2 GB on
    Hkv = 3                                    # 14.5 GB per tensor
    k8, v8 = (torch.zeros(B, Hkv, Nk, d, dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(B, Hkv, -(-Nk // 128), device=dev) for _ in range(2))
    L = [5, 40, Nk - 3]
    x, y = (rows(i, (B, Hkv, 3, d), dev, torch.bfloat16) for i in (31, 32))
    A.kvcache8_append(k8, v8, ks, vs, x, y, torch.tensor(L, dtype=torch.int32, device=dev), block=128)
    q = torch.randn(B, Hkv, 1, d, device=dev).bfloat16()
    cl = torch.tensor([8, 43, Nk], dtype=torch.int32, device=dev)
    o, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, False, 4.0, 128, out_f32=True)
    status_ok()
    # every earlier key is zero: scores 0, weight exp(0), values 0
    back = lambda x8, s, b, h: x8[b, h, L[b]:L[b] + 3].double() * torch.stack([s[b, h, (L[b] + i) // 128] for i in range(3)]).double()[:, None]
    for b in range(B):
        for h in range(Hkv):
            kk, vv = back(k8, ks, b, h), back(v8, vs, b, h)
            assert float((kk - x[b, h].double()).abs().max()) <= float(x[b, h].abs().max()) / 250
            s = 4.0 * (kk @ q[b, h, 0].double())
            m = s.max().clamp(min=0)
            z = torch.exp(s - m).sum() + L[b] * torch.exp(-m)
            want = (torch.exp(s - m) / z) @ vv
            assert float((o[b, h, 0].double() - want).abs().max()) <= 2.0 ** -6 * float(vv.abs().max())
            assert abs(float(lse[b, h, 0]) - float(m + torch.log(z))) <= 1e-4 * max(1.0, float(m))

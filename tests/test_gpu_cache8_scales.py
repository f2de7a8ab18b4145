"""GPU tests of attention over an 8-bit cache whose value scales lie far apart: a row's error is
relative to the values that it sees, whatever the scales of other blocks."""
import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import cache_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ROWS = [(4, 30), (4, 90)]  # query heads over two kv heads, queries: 60 and 180 rows


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    _lib.load()
    return torch.device("cuda:0")


def randn(seed, shape, dev):
    return torch.randn(shape, generator=torch.Generator(dev).manual_seed(seed), device=dev)


def cache_of(dev, shape, block, cache, seed=1):
    return P.quantise(randn(seed, shape, dev), block, cache) + P.quantise(randn(seed + 1, shape, dev), block, cache)


def check(q, k8, v8, ks, vs, block, lens, causal, scale=None):
    cl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=q.device)
    o32, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, scale, block, out_f32=True)
    o, _ = A.fwd_kvcache8(q, k8, v8, ks, vs, cl, causal, scale, block)
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_OK
    P.check_attend8(o32, o, lse, q, k8, v8, ks, vs, block, lens, causal, scale)
    return o32, lse


@pytest.mark.parametrize("Hq,Nq", ROWS)
@pytest.mark.parametrize("dtype,cache", [("bf16", "i8"), ("f16", "i8"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("power", [8, 16, 22, 28, 40])
def test_causal_rows_that_see_small_scales_only(dev, Hq, Nq, dtype, cache, block, power):
    """The first block's values 2^-power of those behind it, which the first rows do not see."""
    L = block + 20
    k8, ks, v8, vs = cache_of(dev, (2, 2, L, 64), block, cache)
    vs[:, :, 0] *= 2.0 ** -power
    q = randn(3, (2, Hq, Nq, 64), dev).to(DT[dtype])
    check(q, k8, v8, ks, vs, block, [L, L - 3], True)


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (8, 1), (4, 30), (4, 90)])
@pytest.mark.parametrize("dtype,d,block", [("bf16", 128, 16), ("f16", 64, 64), ("f16", 128, 32), ("bf16", 64, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_scales_in_no_order_over_forty_powers_of_two(dev, Hq, Nq, dtype, d, block, causal):
    """Every power in turn, some blocks of scale 0 with codes that are not, in short and in long caches."""
    for Nk, lens in ((700, [700, 333]), (9000, [9000, 8191])):
        k8, ks, v8, vs = cache_of(dev, (2, 2, Nk, d), block, "i8")
        vs *= torch.exp2(-(torch.arange(vs.shape[2], device=dev) * 5 % 41).float())
        vs[:, :, 3], vs[0, 0, 5 % vs.shape[2]], ks[:, :, 4] = 0, 0, 0
        q = randn(3, (2, Hq, Nq, d), dev).to(DT[dtype])
        check(q, k8, v8, ks, vs, block, lens, causal)


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (4, 30), (4, 90)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_values_of_no_weight(dev, Hq, Nq, dtype):
    """Blocks of values 2^20 times the others', with weights of about 2^-36: the others decide the output."""
    block, Nk, d = 16, 640, 64
    k = randn(1, (1, 2, Nk, d), dev) * 0.1
    q = (randn(3, (1, Hq, Nq, d), dev) * 0.1 + 1).to(DT[dtype])
    k[:, :, 320:352] = -25.0 / 8  # q.k / 8 = -25
    k8, ks = P.quantise(k, block, "i8")
    v8, vs = P.quantise(randn(2, (1, 2, Nk, d), dev), block, "i8")
    vs[:, :, 20:22] *= 2.0 ** 20
    for causal in (True, False):
        check(q, k8, v8, ks, vs, block, None, causal)


@pytest.mark.parametrize("Hq,Nq", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [16, 128])
def test_rows_that_see_a_scale_of_zero_only(dev, Hq, Nq, dtype, block):
    """Codes that are not 0 stand for 0 with a scale of 0."""
    L = block + 20
    k8, ks, v8, vs = cache_of(dev, (1, 2, L, 64), block, "i8")
    vs[:, :, 0] = 0
    q = randn(3, (1, Hq, Nq, 64), dev).to(DT[dtype])
    o, lse = check(q, k8, v8, ks, vs, block, None, True)
    seen = torch.arange(Nq, device=dev) + L - Nq < block
    assert bool((o[:, :, seen] == 0).all()) and bool(seen.any())


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (4, 30), (4, 90)])
@pytest.mark.parametrize("Nk", [90, 700, 9000])
def test_the_lse_does_not_depend_on_the_values(dev, Hq, Nq, Nk):
    """Scales of zero, and one large scale at the front of small ones: a row sum 2^60 or 2^50 times its usual
    size, and an LSE as exact as ever: small queries, so E is next to nothing."""
    for seed in range(5):
        k8, ks, v8, vs = cache_of(dev, (3, 2, Nk, 64), 16, "i8", seed)
        vs[0], vs[1, :, 1:] = 0, vs[1, :, 1:] * 2.0 ** -50
        q = (1e-3 * randn(seed + 9, (3, Hq, Nq, 64), dev)).half()
        check(q, k8, v8, ks, vs, 16, [Nk, Nk, Nk - 13], True)


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (4, 30), (4, 90)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("power", [-100, 100])
def test_heads_of_very_small_and_very_large_values(dev, Hq, Nq, dtype, power):
    """All of a head's scales far from one: fp32 outputs to the same relative error."""
    for Nk in (300, 20000):
        k8, ks, v8, vs = cache_of(dev, (1, 2, Nk, 64), 64, "i8")
        q = randn(3, (1, Hq, Nq, 64), dev).to(DT[dtype])
        cl = torch.tensor([Nk - 1], dtype=torch.int32, device=dev)
        o, lse = A.fwd_kvcache8(q, k8, v8, ks, vs * 2.0 ** power, cl, True, out_f32=True)
        P.check_attend8(o, None, lse, q, k8, v8, ks, vs * 2.0 ** power, 64, [Nk - 1], True)


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (4, 30), (4, 90)])
@pytest.mark.parametrize("order", [(-100, 0, 100), (100, 0, -100), (0, -100, 100), (-100, -100, 0)])
def test_scales_beyond_the_range_count_as_zero(dev, Hq, Nq, order):
    """Blocks whose scales lie more than 2^60 apart, in any order, and a first one of scale 0: the LSE, and what
    the small ones add to the outputs is below 2^-50 of the largest."""
    block = 16
    for Nk in (4 * block, 6000):
        k8, ks, v8, vs = cache_of(dev, (2, 2, Nk, 64), block, "i8")
        n = vs.shape[2]
        power = torch.tensor([order[min(2, 3 * i // n)] for i in range(n)], device=dev)
        vs = vs * torch.exp2(power.float())
        vs[1, :, 0] = 0
        q = randn(3, (2, Hq, Nq, 64), dev).bfloat16()
        o, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True, None, block, out_f32=True)
        ro, rl, bound, _, E = P.attend8(q, k8, v8, ks, vs, block, None, True)
        torch.cuda.synchronize()
        assert A.get_device_status() == _lib.ATTN_OK
        most = float(vs.max()) * 127
        assert bool(((o.double() - ro).abs() <= bound + 2.0 ** -50 * most).all())
        none = torch.isneginf(rl)
        assert torch.equal(torch.isneginf(lse), none)
        assert bool(((lse.double() - rl).abs().masked_fill(none, 0) <= E + 2.0 ** -18 + rl.abs().masked_fill(none, 0) * 2.0 ** -22).all())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 50.0])
@pytest.mark.parametrize("Nq", [1, 100])
def test_scales_of_the_scores_at_the_ends_of_their_range(dev, scale, Nq):
    """Products of the scale and a key's that leave float's normal range: even weights, nothing masked that is seen."""
    for block in (16, 128):
        k8, ks, v8, vs = cache_of(dev, (2, 2, 500, 64), block, "i8")
        if scale < 1:
            ks = ks * 1e-9
        q = randn(3, (2, 4, Nq, 64), dev).half()
        check(q, k8, v8, ks, vs, block, [500, 130], True, scale)


def long_case(dev, B, Hq, Hkv, Nq, Nk, d, block, dtype, cache, lens, causal, seed):
    g = torch.Generator(dev).manual_seed(seed)
    rows = lambda: (torch.randn(B, Hkv, Nk, d, generator=g, device=dev) * torch.exp(0.5 * torch.randn(B, Hkv, Nk, 1, generator=g, device=dev)))
    k8, ks = P.quantise(rows(), block, cache)
    v8, vs = P.quantise(rows(), block, cache)
    q = (0.25 * torch.randn(B, Hq, Nq, d, generator=g, device=dev)).to(DT[dtype])  # weights of one size
    for b, L in enumerate(lens):  # behind a length: anything
        k8.view(torch.uint8)[b, :, L:], v8.view(torch.uint8)[b, :, L:] = 0x7f, 0x7f
        ks[b, :, -(-L // block):], vs[b, :, -(-L // block):] = float("nan"), float("inf")
    check(q, k8, v8, ks, vs, block, lens, causal)


@pytest.mark.parametrize("Hq,Nq,block,dtype", [(8, 1, 64, "bf16"), (8, 3, 16, "f16"), (32, 4, 32, "bf16")])
def test_every_key_of_long_caches_of_64_columns_counts(dev, Hq, Nq, block, dtype):
    long_case(dev, 7, Hq, 8, Nq, 30011, 64, block, dtype, "i8", [30011, 1, 64, 29000, 65, 30011, 7], True, Nq)
    long_case(dev, 7, Hq, 8, Nq, 30011, 48, block, dtype, "e4m3", [30011, 1, 64, 29000, 65, 30011, 7], False, Nq)


@pytest.mark.parametrize("cache,d", [("i8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("Hq,Nq", [(8, 1), (32, 1), (32, 5), (32, 10), (32, 30)])
def test_every_key_of_long_caches_behind_short_ones_counts(dev, cache, d, Hq, Nq):
    lens = [9000, 1, 1, 40, 12321, 2, 3, 1, 1, 5, 8000]
    for dtype in ("bf16", "f16"):
        long_case(dev, len(lens), Hq, 8, Nq, 12321, d, 64, dtype, cache, lens, True, Nq)


def test_every_key_of_long_caches_counts_with_many_rows(dev):
    long_case(dev, 2, 142, 2, 1, 100001, 16, 16, "bf16", "i8", [100001, 80000], False, 1)
    long_case(dev, 3, 16, 4, 20, 40001, 64, 32, "f16", "e4m3", [40001, 1, 39000], True, 2)
    long_case(dev, 2, 71, 1, 1, 9000, 112, 16, "f16", "i8", [9000, 77], False, 3)


@pytest.mark.parametrize("B,Hkv,Nk,d,dtype", [(9, 4, 120000, 64, "bf16"), (2, 5, 700001, 112, "f16")])
def test_many_rows_by_groups_of_batches_and_of_heads(dev, B, Hkv, Nk, d, dtype):
    """More keys than are held in 16 bits at a time: five batches and then four, three heads and then two; a batch
    in the last group with a bad length."""
    lens = [Nk, 1000, 0, Nk - 77, 5, 65536, 70001, 80, Nk - 1][:B]
    long_case(dev, B, 2 * Hkv, Hkv, 40, Nk, d, 64, dtype, "i8", lens, True, 1)
    q, k8 = randn(1, (B, 2 * Hkv, 40, d), dev).to(DT[dtype]), torch.ones(B, Hkv, Nk, d, dtype=torch.int8, device=dev)
    s = torch.ones(B, Hkv, -(-Nk // 64), device=dev)
    o, lse = A.fwd_kvcache8(q, k8, k8, s, s, torch.tensor([40] * (B - 1) + [Nk + 1], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_ERR_DEVICE_INPUT and A.get_device_status() == _lib.ATTN_OK
    assert bool((o[:-1] == 1).all()) and bool((o[-1] == 0).all()) and bool(torch.isneginf(lse[-1]).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,cache,d,block", [("bf16", "i8", 128, 64), ("f16", "e4m3", 64, 32), ("f16", "i8", 80, 16), ("bf16", "e4m3", 112, 128)])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (8, 1, 2), (6, 2, 5), (16, 2, 5), (4, 1, 13), (4, 1, 37), (8, 2, 130)])
def test_every_key_of_ragged_caches_counts(dev, causal, dtype, cache, d, block, Hq, Hkv, Nq):
    long_case(dev, 7, Hq, Hkv, Nq, 700, d, block, dtype, cache, [700, 333, 64, 3, 1, 0, 513], causal, Nq)

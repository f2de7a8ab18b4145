"""GPU tests of attention over an 8-bit cache with bounds that a tile of wrong values would break."""
import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import cache_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


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


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,cache,d,block", [("bf16", "i8", 128, 64), ("f16", "e4m3", 64, 32), ("f16", "i8", 80, 16), ("bf16", "e4m3", 112, 128)])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (8, 1, 2), (6, 2, 5), (16, 2, 5), (4, 1, 13), (4, 1, 37), (8, 2, 130)])
def test_every_key_of_ragged_caches_counts(dev, causal, dtype, cache, d, block, Hq, Hkv, Nq):
    long_case(dev, 7, Hq, Hkv, Nq, 700, d, block, dtype, cache, [700, 333, 64, 3, 1, 0, 513], causal, Nq)

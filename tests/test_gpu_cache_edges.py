"""GPU tests of the cache operators where inputs are NaN, infinite or signed zeros."""
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


def status_ok():
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_OK


def randn(seed, shape, dev, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(dev).manual_seed(seed), device=dev).to(dtype)


# -------------------------------------------------------------------------------------- evict
@pytest.mark.parametrize("Nk", [700, 3000, 40000, 300000])
def test_evict_hands_weights_on_as_they_are(dev, Nk):
    """Bit by bit, in every form of the selection: zeros of both signs, NaN of both signs and other payloads."""
    k = randn(1, (1, 2, Nk, 16), dev, torch.bfloat16)
    w = randn(2, (1, 2, Nk), dev)
    bits = w.view(torch.int32)
    w[..., ::5] = -0.0
    w[..., 1::50] = 0.0
    bits[..., 3::97], bits[..., 4::101] = 0x7fc01234, -0x3ffedc  # 0xffc00124
    for keep, recent in ((Nk // 2, 10), (Nk // 3, 0), (20, Nk // 2)):
        _, _, wo, index, lens = A.kvcache_evict(k, k, w, keep, recent)
        status_ok()
        for h in range(2):
            at = torch.from_numpy(P.evict(None, None, w[0, h].cpu().numpy(), Nk, keep, recent)).to(dev)
            assert torch.equal(index[0, h].long(), at)
            assert torch.equal(wo.view(torch.int32)[0, h], bits[0, h, at])

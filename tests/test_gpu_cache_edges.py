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


# ------------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Nq", [1, 3, 30, 200, 600])
def test_a_row_whose_lse_is_nan_reaches_the_keys_that_it_sees_alone(dev, dtype, Nq):
    """As for a query of NaN: the keys behind its causal limit keep the other rows' weights."""
    q, k = randn(1, (2, 4, Nq, 64), dev, DT[dtype]), randn(2, (2, 2, 700, 64), dev, DT[dtype])
    cl = torch.tensor([700, 650], dtype=torch.int32, device=dev)
    lse = torch.full((2, 4, Nq), 12.0, device=dev)
    i = Nq // 3
    without = lse.clone()
    without[0, 1, i] = without[1, 2, i] = float("-inf")
    want, err = P.weights(q, k, without, cl.tolist(), True, None)
    lse[0, 1, i] = float("nan")
    q[1, 2, i] = float("nan")
    got = A.kvcache_weights(q, k, lse, cl, True)
    status_ok()
    seen = torch.zeros(2, 2, 700, dtype=torch.bool, device=dev)
    seen[0, 0, :700 - Nq + i + 1], seen[1, 1, :650 - Nq + i + 1] = True, True
    assert torch.equal(got.isnan(), seen)
    assert bool(((got.double() - want).abs() <= err)[~seen].all())


# --------------------------------------------------------------------------------- key ranges
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("splits", [1, 2, 5])
def test_nan_in_some_or_all_ranges_of_a_cache(dev, dtype, splits):
    """A query of NaN, and a key that some rows see: NaN in O and LSE of those rows, not an empty row's 0 and -inf."""
    q = randn(1, (2, 4, 6, 64), dev, DT[dtype])
    k, v = (randn(i, (2, 2, 900, 64), dev, DT[dtype]) for i in (2, 3))
    cl = torch.tensor([900, 3], dtype=torch.int32, device=dev)
    want, wl = A.fwd_kvcache(q, k, v, cl, True, num_splits=splits)
    q[0, 1, 2] = float("nan")
    k[0, 1, 897] = float("nan")  # seen by the queries from 3 on, of heads 2 and 3
    o, lse = A.fwd_kvcache(q, k, v, cl, True, num_splits=splits)
    status_ok()
    bad = torch.zeros(2, 4, 6, dtype=torch.bool, device=dev)
    bad[0, 1, 2] = bad[0, 2:, 3:] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse[~bad], wl[~bad]) and torch.equal(o[~bad], want[~bad])
    assert bool(torch.isneginf(lse[1, :, :3]).all()) and bool((o[1, :, :3] == 0).all())


@pytest.mark.parametrize("Nq", [1, 12, 100])
@pytest.mark.parametrize("Nk", [200, 30000])
def test_nan_scores_over_an_8_bit_cache(dev, Nq, Nk):
    """A query of NaN (every row of its tile keeps its own scores) and a key scale of NaN: O and LSE of the rows
    that see it are NaN, with one key range and with several."""
    q = randn(1, (2, 4, Nq, 64), dev, torch.bfloat16)
    k8, ks = P.quantise(randn(2, (2, 2, Nk, 64), dev), 16, "i8")
    v8, vs = P.quantise(randn(3, (2, 2, Nk, 64), dev), 16, "i8")
    want, wl = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True, block=16)
    q[0, 1, Nq // 2] = float("nan")
    ks[1, 0, 0] = float("nan")
    o, lse = A.fwd_kvcache8(q, k8, v8, ks, vs, None, True, block=16)
    status_ok()
    bad = torch.zeros(2, 4, Nq, dtype=torch.bool, device=dev)
    bad[0, 1, Nq // 2] = bad[1, :2] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse[~bad], wl[~bad]) and torch.equal(o[~bad], want[~bad])


@pytest.mark.parametrize("Nq", [1, 12, 100])
@pytest.mark.parametrize("Nk", [200, 30000])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_value_scales_that_are_not_finite_leave_the_lse(dev, Nq, Nk, dtype, what):
    """O of the rows that see such a block is not finite; the LSE is that of the keys, and other heads are as they were."""
    q = randn(1, (2, 4, Nq, 64), dev, DT[dtype])
    k8, ks = P.quantise(randn(2, (2, 2, Nk, 64), dev), 16, "i8")
    v8, vs = P.quantise(randn(3, (2, 2, Nk, 64), dev), 16, "i8")
    want, wl = A.fwd_kvcache8(q, k8, v8, ks, vs, None, False, block=16)
    for block in (0, 5, -1):
        bad = vs.clone()
        bad[1, 0, block] = float(what)
        o, lse = A.fwd_kvcache8(q, k8, v8, ks, bad, None, False, block=16)
        status_ok()
        assert bool((lse - wl).abs().max() <= 2.0 ** -18 * wl.abs().max())
        assert not bool(o[1, :2].isfinite().all(-1).any())
        assert torch.equal(o[0], want[0]) and torch.equal(o[1, 2:], want[1, 2:])

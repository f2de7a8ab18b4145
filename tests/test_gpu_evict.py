"""GPU tests of the accumulated attention weights and of eviction by them, and of the run of the
cache operators together: prompt, weights, eviction, 8-bit cache, decode."""
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


def status_ok():
    torch.cuda.synchronize()
    assert A.get_device_status() == _lib.ATTN_OK


def randn(seed, shape, dev, dtype):
    return torch.randn(shape, generator=torch.Generator(dev).manual_seed(seed), device=dev).to(dtype)


# ------------------------------------------------------------------------------------ weights
def run_weights(dev, B, Hq, Hkv, Nq, Nk, d, dtype, lens, causal, seed, with_in=True, scale=None):
    q, k = randn(seed, (B, Hq, Nq, d), dev, DT[dtype]), randn(seed + 1, (B, Hkv, Nk, d), dev, DT[dtype])
    cl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    _, lse64, _, _ = P.attend(q, k.double(), k.double(), lens, causal, scale)
    lse = lse64.float()
    w_in = randn(seed + 2, (B, Hkv, Nk), dev, torch.float32).abs() if with_in else None
    want, err = P.weights(q, k, lse, lens, causal, w_in, scale)
    if lens is not None:  # what lies behind a length may hold anything
        for b, L in enumerate(lens):
            k[b, :, L:] = float("nan")
    got = A.kvcache_weights(q, k, lse, cl, causal, scale, w_in)
    status_ok()
    bad = (got.double() - want).abs() - err
    assert bool((bad <= 0).all()), (float(bad.max()), float((got.double() - want).abs().max()))
    if w_in is not None:  # in place, and the same bits again
        out = A.kvcache_weights(q, k, lse, cl, causal, scale, w_in, out=w_in)
        status_ok()
        assert out.data_ptr() == w_in.data_ptr() and torch.equal(out, got)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 80), ("f16", 16), ("f32", 128)])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (4, 4, 1), (6, 2, 5), (8, 2, 37), (4, 1, 100), (4, 2, 300)])
def test_weights_ragged(dev, causal, dtype, d, Hq, Hkv, Nq):
    run_weights(dev, 7, Hq, Hkv, Nq, 700, d, dtype, [700, 333, 128, 3, 1, 0, 513], causal, seed=Nq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nk", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1025])
def test_weights_lengths(dev, dtype, Nk):
    run_weights(dev, 2, 4, 2, 1, Nk, 64, dtype, None, False, seed=Nk, with_in=False)
    run_weights(dev, 2, 4, 2, Nk, Nk, 128, dtype, None, True, seed=Nk)
    run_weights(dev, 1, 8, 1, 33, Nk, 128, dtype, [max(0, Nk - 5)], True, seed=Nk)


def test_weights_scale_and_many_rows(dev):
    run_weights(dev, 2, 4, 4, 600, 520, 64, "bf16", [520, 400], True, seed=3, scale=0.4)
    run_weights(dev, 1, 32, 1, 129, 1111, 128, "f16", None, True, seed=4)
    run_weights(dev, 4, 16, 4, 1200, 1200, 64, "bf16", [1200, 1100, 300, 0], True, seed=5)  # two CTAs per 256 keys
    run_weights(dev, 20, 8, 8, 300, 700, 128, "bf16", [700 - 30 * b for b in range(20)], True, seed=6)  # several items a CTA


@pytest.mark.parametrize("Hq,Nq,d", [(8, 1, 128), (8, 30, 128), (4, 200, 64), (8, 1, 64)])
def test_weights_long_caches(dev, Hq, Nq, d):
    """Dozens of items per CTA, some of them with keys in their first half only: every ring turns
    many times, and its readers at different speeds.  The same bits each time."""
    lens = [200001, 130, 77000, 100, 256 * 300 + 128, 1, 199999]
    run_weights(dev, 7, Hq, 4, Nq, 200001, d, "bf16", lens, True, seed=Nq)
    q, k = randn(1, (7, Hq, Nq, d), dev, torch.bfloat16), randn(2, (7, 4, 200001, d), dev, torch.bfloat16)
    lse = torch.full((7, Hq, Nq), 11.0, device=dev)
    cl = torch.tensor(lens, dtype=torch.int32, device=dev)
    want = A.kvcache_weights(q, k, lse, cl)
    for _ in range(20):
        assert torch.equal(A.kvcache_weights(q, k, lse, cl), want)
    status_ok()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Nq", [127, 128, 129, 257, 1000])
def test_weights_walk_over_heads(dev, causal, Nq):
    """Heads a little shorter, as long as and longer than a tile, caches shorter and longer than the
    queries: which tiles see a key, for whole items and for those that several CTAs share."""
    run_weights(dev, 20, 6, 2, Nq, 1100, 64, "bf16", [1100 - 53 * b for b in range(20)], causal, seed=Nq)
    run_weights(dev, 2, 3, 1, Nq, 1100, 128, "f16", [1100, Nq // 2], causal, seed=Nq)


def test_weights_and_evict_with_thousands_of_sequences(dev):
    B = 5000
    lens = [(13 * b) % 34 for b in range(B)]
    run_weights(dev, B, 4, 2, 1, 33, 16, "bf16", lens, True, seed=4)
    k, w = randn(1, (B, 2, 33, 16), dev, torch.bfloat16), randn(2, (B, 2, 33), dev, torch.float32)
    got = A.kvcache_evict(k, k, w, 9, 4, torch.tensor(lens, dtype=torch.int32, device=dev))
    status_ok()
    some = [0, 1, 33, 1234, 2500, 4097, B - 1]
    check_evict(k[some], k[some], w[some], 9, 4, [lens[b] for b in some], tuple(x[some] for x in got),
                tuple(torch.zeros_like(x[some]) for x in got[:2]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Nq", [1, 9, 200, 600])
def test_weights_of_rows_that_a_caller_leaves_out(dev, dtype, causal, Nq):
    """Padded queries: an LSE of -inf, and q whatever was there.  Such rows add nothing, nor do the
    rows that fill up a tile, against keys with infinities either."""
    q, k = randn(1, (3, 4, Nq, 64), dev, DT[dtype]), randn(2, (3, 2, 400, 64), dev, DT[dtype])
    cl = torch.tensor([400, 390, 0], dtype=torch.int32, device=dev)
    lse = torch.full((3, 4, Nq), 12.0, device=dev)
    lse[0, 1], lse[1, :, Nq // 2:] = float("-inf"), float("-inf")
    want, err = P.weights(q, k, lse, cl.tolist(), causal, None)
    q[0, 1], q[1, 2, Nq // 2:], q[1, 3, Nq // 2:] = float("nan"), float("inf"), float("-inf")
    got = A.kvcache_weights(q, k, lse, cl, causal)
    status_ok()
    assert bool(((got.double() - want).abs() <= err).all())
    # one component of a key infinite, all queries on its other side: a score of -inf, a weight of 0
    q = randn(1, (3, 4, Nq, 64), dev, DT[dtype]).abs()
    k[:, :, 7, 3] = float("-inf")
    got = A.kvcache_weights(q, k, lse, cl, causal)
    status_ok()
    assert bool((got[:, :, 7] == 0).all()) and bool(got.isfinite().all())


def test_weights_sum_to_the_number_of_rows_after_the_forward(dev):
    """With the forward's own LSE: each row's weights add up to one, so the sum over the keys is the
    number of (head, query) rows that see any key."""
    q, k = randn(1, (3, 8, 40, 128), dev, torch.bfloat16), randn(2, (3, 2, 900, 128), dev, torch.bfloat16)
    cl = torch.tensor([900, 17, 0], dtype=torch.int32, device=dev)
    _, lse = A.fwd_kvcache(q, k, k, cl, True)
    w = A.kvcache_weights(q, k, lse, cl, True)
    status_ok()
    for b, rows in enumerate((40, 17, 0)):
        assert float((w[b].double().sum(-1) - 4 * rows).abs().max()) <= 4 * rows * 1e-4
    assert bool((w[1, :, 17:] == 0).all())
    _, lse = A.fwd(k, k, k, True)
    w = A.kvcache_weights(k, k, lse, None, True)
    status_ok()
    assert float((w.double().sum(-1) - 900).abs().max()) <= 0.09


def test_weights_empty_calls_and_bad_lengths(dev):
    q, k = randn(1, (2, 4, 3, 64), dev, torch.bfloat16), randn(2, (2, 2, 100, 64), dev, torch.bfloat16)
    lse = torch.zeros(2, 4, 3, device=dev)
    w_in = torch.rand(2, 2, 100, device=dev)
    none = q[:, :, :0].contiguous()
    assert torch.equal(A.kvcache_weights(none, k, lse[..., :0].contiguous(), weights=w_in), w_in)
    assert bool((A.kvcache_weights(none, k, lse[..., :0].contiguous()) == 0).all())
    assert A.kvcache_weights(q, k[:, :, :0].contiguous(), lse).shape == (2, 2, 0)
    status_ok()
    for bad in (101, -7):
        w = A.kvcache_weights(q, k, lse, torch.tensor([bad, 100], dtype=torch.int32, device=dev), weights=w_in)
        torch.cuda.synchronize()
        assert A.get_device_status() == _lib.ATTN_ERR_DEVICE_INPUT and A.get_device_status() == _lib.ATTN_OK
        assert torch.equal(w[0], w_in[0]) and bool((w[1] > w_in[1]).all())
    for kw in (dict(lse=lse[:, :, :2].contiguous()), dict(k_cache=k[:1]), dict(weights=w_in[:, :1].contiguous()), dict(out=w_in[:1]),
               dict(q=q[:, :3].contiguous()), dict(k_cache=k.transpose(1, 2))):
        with pytest.raises((ValueError, _lib.AttnError)):
            A.kvcache_weights(**{**dict(q=q, k_cache=k, lse=lse[:, :3].contiguous() if "q" in kw else lse), **kw})
    with pytest.raises(TypeError):
        A.kvcache_weights(q, k.half(), lse)


# -------------------------------------------------------------------------------------- evict
def check_evict(k, v, w, keep, recent, lens, out, before):
    ko, vo, wo, index, nl = out
    B, Hkv, Nk, _ = k.shape
    M, cap = keep + recent, ko.shape[2]
    wn = w.cpu().numpy()
    for b in range(B):
        L = Nk if lens is None else lens[b]
        n = min(L, M)
        assert int(nl[b]) == n
        for h in range(Hkv):
            at = torch.from_numpy(P.evict(None, None, wn[b, h], L, keep, recent)).to(k.device)
            assert torch.equal(index[b, h, :n].long(), at) and bool((index[b, h, n:] == -1).all())
            assert torch.equal(wo[b, h, :n].nan_to_num(-1), w[b, h, at].nan_to_num(-1)) and bool((wo[b, h, n:] == 0).all())
            for x, y, z in ((k, ko, before[0]), (v, vo, before[1])):
                assert torch.equal(y[b, h, :n], x[b, h, at])
                assert torch.equal(y[b, h, n:], z[b, h, n:])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 80), ("f32", 16)])
@pytest.mark.parametrize("keep,recent,extra", [(100, 30, 0), (1, 0, 5), (0, 17, 0), (600, 100, 64), (255, 1, 3), (64, 701, 0)])
def test_evict(dev, dtype, d, keep, recent, extra):
    B, Hkv, Nk = 6, 2, 700
    k, v = randn(1, (B, Hkv, Nk, d), dev, DT[dtype]), randn(2, (B, Hkv, Nk, d), dev, DT[dtype])
    w = randn(3, (B, Hkv, Nk), dev, torch.float32).abs()
    w[0] = (w[0] * 4).floor()          # few different weights: ties
    w[1] = 0.25                        # all equal
    w[2, 0, ::7], w[2, 1, 5], w[2, 1, 9] = float("nan"), float("inf"), -0.0
    w[3] = -w[3]
    for lens in (None, [700, 131, 699, 400, 1, 0]):
        out = tuple(torch.full((B, Hkv, keep + recent + extra, d), 3.0, dtype=k.dtype, device=dev) for _ in range(2))
        before = tuple(x.clone() for x in out)
        cl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
        got = A.kvcache_evict(k, v, w, keep, recent, cl, out=out)
        status_ok()
        check_evict(k, v, w, keep, recent, lens, got, before)


@pytest.mark.parametrize("Nk,keep,recent", [(1, 1, 0), (2, 1, 0), (1023, 511, 2), (1024, 1, 1), (1025, 1024, 0), (40000, 4001, 128), (200000, 30000, 1)])
def test_evict_lengths(dev, Nk, keep, recent):
    k, v = randn(4, (1, 3, Nk, 32), dev, torch.bfloat16), randn(5, (1, 3, Nk, 32), dev, torch.bfloat16)
    w = torch.exp(2 * randn(6, (1, 3, Nk), dev, torch.float32))
    w[0, 1] = (w[0, 1] * 2).floor()
    got = A.kvcache_evict(k, v, w, keep, recent)
    status_ok()
    check_evict(k, v, w, keep, recent, None, got, tuple(torch.zeros_like(x) for x in got[:2]))


@pytest.mark.parametrize("Nk", [3000, 40000, 300000])
def test_evict_many_equal_weights(dev, Nk):
    """More keys of one weight, or of nearly one, than any list holds."""
    k, v = randn(4, (1, 2, Nk, 16), dev, torch.bfloat16), randn(5, (1, 2, Nk, 16), dev, torch.bfloat16)
    w = torch.full((1, 2, Nk), 0.5, device=dev)
    w[0, 1] += 1e-6 * torch.randint(0, 30, (Nk,), generator=torch.Generator(dev).manual_seed(1), device=dev)
    w[0, 0, 100:120] = 2.0
    got = A.kvcache_evict(k, v, w, Nk // 3, 10)
    status_ok()
    check_evict(k, v, w, Nk // 3, 10, None, got, tuple(torch.zeros_like(x) for x in got[:2]))


def test_offsets_past_32_bits(dev):
    """Caches of more than 2^32 bytes, the keys that matter in the last head's last rows."""
    Hkv, Nk, d = 3, 2 ** 23, 128  # 2.1 GB of keys a head
    k = torch.zeros(1, Hkv, Nk, d, dtype=torch.bfloat16, device=dev)
    k[0, :, -2:] = randn(7, (Hkv, 2, d), dev, torch.bfloat16)
    q = randn(8, (1, 6, 2, d), dev, torch.bfloat16)
    lse = torch.full((1, 6, 2), 3.0, device=dev)
    w = A.kvcache_weights(q, k, lse, None, False)
    status_ok()
    for h in range(Hkv):
        s = q[0, 2 * h:2 * h + 2].double().reshape(4, d) @ k[0, h, -2:].double().T / d ** 0.5
        want = torch.exp(s - 3.0).sum(0)
        assert float((w[0, h, -2:].double() / want - 1).abs().max()) < 1e-5
        assert float((w[0, h, :-2].double() / (4 * np.exp(-3.0)) - 1).abs().max()) < 1e-5
    w.zero_()
    w[0, :, 5], w[0, :, -3], w[0, :, -2] = 1.0, 2.0, 3.0
    v = k.clone()
    v[0, :, -3] = 7.0
    ko, vo, wo, index, lens = A.kvcache_evict(k, v, w, 3, 1)
    status_ok()
    at = [5, Nk - 3, Nk - 2, Nk - 1]
    assert index[0].tolist() == [at] * Hkv and lens.tolist() == [4]
    for h in range(Hkv):
        assert torch.equal(ko[0, h], k[0, h, at]) and torch.equal(vo[0, h], v[0, h, at])


def test_evict_bad_lengths_empty_cache_and_refusals(dev):
    k = randn(4, (2, 2, 50, 32), dev, torch.bfloat16)
    w = torch.rand(2, 2, 50, device=dev)
    for bad in (51, -1):
        got = A.kvcache_evict(k, k, w, 10, 5, torch.tensor([bad, 50], dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        assert A.get_device_status() == _lib.ATTN_ERR_DEVICE_INPUT and A.get_device_status() == _lib.ATTN_OK
        check_evict(k, k, w, 10, 5, [0, 50], got, tuple(torch.zeros_like(x) for x in got[:2]))
    none = k[:, :, :0].contiguous()
    got = A.kvcache_evict(none, none, w[:, :, :0].contiguous(), 3, 0)
    status_ok()
    assert got[4].tolist() == [0, 0] and bool((got[3] == -1).all()) and bool((got[0] == 0).all())
    big = torch.zeros(2, 2, 15, 32, dtype=torch.bfloat16, device=dev)
    for kw in (dict(keep=-1), dict(keep=0, recent=0), dict(weights=w[:, :1].contiguous()), dict(out=(big[:, :, :14].contiguous(), big)),
               dict(out=(k, big)), dict(out=(big, big)), dict(v_cache=k[:1])):
        with pytest.raises((ValueError, _lib.AttnError)):
            A.kvcache_evict(**{**dict(k_cache=k, v_cache=k, weights=w, keep=10, recent=5), **kw})
    with pytest.raises(TypeError):
        A.kvcache_evict(k, k.half(), w, 10, 5)


def test_evict_and_weights_in_a_graph(dev):
    q, k, v = (randn(i, (2, h, n, 64), dev, torch.bfloat16) for i, h, n in ((1, 4, 3), (2, 2, 500), (3, 2, 500)))
    cl = torch.tensor([500, 20], dtype=torch.int32, device=dev)
    w = torch.rand(2, 2, 500, device=dev)
    out = tuple(torch.zeros(2, 2, 80, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))

    def step():
        _, lse = A.fwd_kvcache(q, k, v, cl, True)
        w2 = A.kvcache_weights(q, k, lse, cl, True, weights=w)
        return (w2,) + A.kvcache_evict(k, v, w2, 50, 10, cl, out=out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for lens in ([500, 20], [61, 500], [60, 0]):
        cl.copy_(torch.tensor(lens, dtype=torch.int32))
        w.uniform_()
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    status_ok()


# ----------------------------------------------------------------------------------- together
@pytest.mark.parametrize("cache,block", [("i8", 32), ("e4m3", 64)])
def test_prompt_weights_eviction_and_decode_together(dev, cache, block):
    """A padded batch of prompts of different lengths; its last queries judge the keys; each cache is
    cut to 96 + 32 keys, held in 8 bits, and six tokens are decoded on top.  Every step is compared
    with 64 bits on the step's own inputs, and the end with the decode over the evicted cache in 16 bits."""
    from tests.test_gpu_cache8 import check_attend
    B, Hq, Hkv, N, d, win = 3, 8, 2, 600, 128, 24
    lens = [600, 411, 90]
    cl = torch.tensor(lens, dtype=torch.int32, device=dev)
    k, v = (randn(i, (B, Hkv, N, d), dev, torch.bfloat16) for i in (1, 2))
    q = randn(3, (B, Hq, win, d), dev, torch.bfloat16)
    _, lse = A.fwd_kvcache(q, k, v, cl, True)
    w = A.kvcache_weights(q, k, lse, cl, True)
    kc, vc, wc, index, nl = A.kvcache_evict(k, v, w, 96, 32, cl)
    status_ok()
    check_evict(k, v, w, 96, 32, lens, (kc, vc, wc, index, nl), tuple(torch.zeros_like(kc) for _ in range(2)))
    cap = 150
    k8, v8 = (torch.zeros(B, Hkv, cap, d, dtype=P.C8[cache], device=dev) for _ in range(2))
    ks, vs = (torch.zeros(B, Hkv, -(-cap // block), device=dev) for _ in range(2))
    A.kvcache8_append(k8, v8, ks, vs, kc, vc, None, nl, block=block)
    k16, v16 = (torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    k16[:, :, :128], v16[:, :, :128] = kc, vc
    now = nl.clone()
    for t in range(6):
        kt, vt = (randn(10 * t + i, (B, Hkv, 1, d), dev, torch.bfloat16) for i in (5, 6))
        qt = randn(10 * t + 7, (B, Hq, 1, d), dev, torch.bfloat16)
        A.kvcache8_append(k8, v8, ks, vs, kt, vt, now, block=block)
        for b in range(B):
            k16[b, :, int(now[b])], v16[b, :, int(now[b])] = kt[b, :, 0], vt[b, :, 0]
        now += 1
        o32, l8 = A.fwd_kvcache8(qt, k8, v8, ks, vs, now, True, block=block, out_f32=True)
        o8, _ = A.fwd_kvcache8(qt, k8, v8, ks, vs, now, True, block=block)
        status_ok()
        check_attend(o32, o8, l8, qt, k8, v8, ks, vs, block, now.tolist(), True)
    o16, _ = A.fwd_kvcache(qt, k16, v16, now, True)
    status_ok()
    # steps of max|x| / 254 per value (int8) or 2^-4 of it (e4m3): well within a tenth of the outputs
    assert float((o8.double() - o16.double()).norm() / o16.double().norm()) < 0.1

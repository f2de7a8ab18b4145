"""GPU tests of packed attention with grouped heads, forward and backward, against 64 bits, with bounds from the roundings
that the kernels make."""
import random

import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import pages_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    _lib.load()
    return torch.device("cuda:0")


def status(bad=False):
    torch.cuda.synchronize()
    assert A.get_device_status() == (_lib.ATTN_ERR_DEVICE_INPUT if bad else _lib.ATTN_OK)


def make(dev, dtype, Hq, Hkv, d, lens, seed=0, fused=True, behind=0):
    """q, k, v, dout, cu; tokens behind the last sequence are NaN."""
    g = torch.Generator(dev).manual_seed(seed)
    T = sum(lens) + behind
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=dev)
    x[:, Hq:] *= torch.exp(0.4 * torch.randn(1, 2 * Hkv, d, generator=g, device=dev))
    dout = torch.randn(T, Hq, d, generator=g, device=dev)
    x[sum(lens):], dout[sum(lens):] = float("nan"), float("nan")
    x = x.to(DT[dtype])
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, dout.to(DT[dtype]), torch.tensor(cu, dtype=torch.int32, device=dev)


def check_fwd(o, lse, q, k, v, lens, causal, out_f32, scale=None):
    Hq, Hkv, d, dt = q.shape[1], k.shape[1], q.shape[2], q.dtype
    G, at = Hq // Hkv, 0
    for L in lens:
        t = slice(at, at + L)
        at += L
        for h in range(Hkv):
            g = slice(h * G, (h + 1) * G)
            x, kh, vh = q[t, g].double().transpose(0, 1), k[t, h].double(), v[t, h].double()
            want, e, p, size = P.attend(x, kh, vh, 0, causal, scale)
            if L == 0:
                continue
            half = 2.0 ** -24 if out_f32 or dt == torch.float32 else P.HALF[dt]
            bo, be = P.attend_bounds(vh, p, size, want, d, P.HALF[dt], half)
            go = o[t, g].double().transpose(0, 1)
            assert ((go - want).abs() <= bo).all(), (L, h, float(((go - want).abs() - bo).max()))
            assert ((lse[g, t].double() - e).abs() <= be + e.abs() * 2.0 ** -22).all(), (L, h)
    assert (o[at:] == 0).all() and (lse[:, at:] == -INF).all()


def check_bwd(got, q, k, v, dout, lens, causal, out_f32, scale=None, few=None):
    Hq, Hkv, dt = q.shape[1], k.shape[1], q.dtype
    G, at = Hq // Hkv, 0
    half = 2.0 ** -24 if out_f32 or dt == torch.float32 else P.HALF[dt]
    rho = 2.0 ** -24 if dt == torch.float32 else P.HALF[dt] ** 2 * 2
    dq, dk, dv = (x.double() for x in got)
    for L in lens:
        t = slice(at, at + L)
        at += L
        for h in range(Hkv):
            g = slice(h * G, (h + 1) * G)
            if L == 0:
                continue
            x, kh, vh, do = q[t, g].double().transpose(0, 1), k[t, h].double(), v[t, h].double(), dout[t, g].double().transpose(0, 1)
            want, bounds = P.grads(x, kh, vh, do, 0, causal, P.HALF[dt], half, rho, scale, few(L) if few else 0)
            for name, y, w, b in zip(("dq", "dk", "dv"), (dq[t, g].transpose(0, 1), dk[t, h], dv[t, h]), want, bounds):
                assert ((y - w).abs() <= b).all(), (name, L, h, float(((y - w).abs() - b).max()))
    assert all((x[at:] == 0).all() for x in (dq, dk, dv))


LENS = [[1], [200, 0, 1, 17, 128, 129], [3, 5, 2, 9, 31, 1, 1, 60], [300, 40, 257, 512]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [
    ("bf16", 8, 2, 128), ("f16", 4, 4, 64), ("bf16", 3, 1, 80), ("f16", 12, 1, 16), ("bf16", 10, 2, 64), ("f16", 32, 2, 128), ("bf16", 7, 1, 48),
    ("f32", 4, 2, 64), ("f32", 3, 1, 128)])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: str(len(x)))
def test_against_64_bits(dev, dtype, Hq, Hkv, d, lens, causal):
    q, k, v, dout, cu = make(dev, dtype, Hq, Hkv, d, lens, seed=Hq + d, behind=5)
    for out_f32 in (True, False):
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, max(lens), causal, out_f32=out_f32)
        status()
        check_fwd(o, lse, q, k, v, lens, causal, out_f32)
    for out_f32, det in ((True, False), (False, True)):
        got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, max(lens), causal, out_f32=out_f32, deterministic=det)
        status()
        check_bwd(got, q, k, v, dout, lens, causal, out_f32)


@pytest.mark.parametrize("dtype,Hq,Hkv,d,lens", [
    ("bf16", 8, 2, 128, [1500, 3, 700]), ("f16", 17, 1, 64, [130, 40]), ("bf16", 71, 1, 64, [50, 20, 9]), ("bf16", 4, 2, 128, [2500]),
    ("f16", 16, 1, 64, [1, 2, 3, 4, 5, 6, 7, 8] * 40), ("bf16", 34, 2, 112, [90, 200])])
def test_group_sizes_and_lengths(dev, dtype, Hq, Hkv, d, lens):
    """Groups that no divisor packs, one head group beside another, hundreds of short sequences, a bound far above the
    longest."""
    q, k, v, dout, cu = make(dev, dtype, Hq, Hkv, d, lens, seed=1, fused=False)
    for bound in (max(lens), 5000):
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, bound, True, scale=0.2)
        check_fwd(o, lse, q, k, v, lens, True, False, 0.2)
        got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, bound, True, scale=0.2)
        status()
        check_bwd(got, q, k, v, dout, lens, True, False, 0.2)


def test_agrees_with_the_packed_qkv_call(dev):
    """Heads without groups: the other packed call's outputs, within both calls' roundings."""
    lens, H, d = [333, 64, 5], 4, 64
    qkv = torch.randn(sum(lens), 3, H, d, device=dev, dtype=torch.float16)
    cu = torch.tensor([0, 333, 397, 402], dtype=torch.int32, device=dev)
    a, la = A.fwd_varlen(qkv, cu, 333, True, out_f32=True)
    b, lb = A.fwd_varlen_gqa(qkv[:, 0], qkv[:, 1], qkv[:, 2], cu, 333, True, out_f32=True)
    status()
    bound = 2 * P.HALF[torch.float16] * qkv[:, 2].float().abs().max()  # P rounded once in each, weights that sum to one
    assert (a - b).abs().max() <= bound and (la - lb).abs().max() <= 2.0 ** -18 * la.abs().max()


def test_a_nan_stays_in_its_sequence(dev):
    """NaN and infinities in one sequence's tokens, and behind the last: the others' outputs and gradients keep their bits."""
    lens, Hq, Hkv, d = [70, 50, 133, 20], 4, 2, 64
    q, k, v, dout, cu = make(dev, "bf16", Hq, Hkv, d, lens, seed=2, fused=False, behind=9)
    for causal in (True, False):
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, 133, causal)
        want = (o, lse.t()) + A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 133, causal, deterministic=True)
        q2, k2, v2, d2 = (x.clone() for x in (q, k, v, dout))
        at = slice(70, 120)
        q2[at], k2[at], v2[at], d2[at] = float("nan"), INF, float("nan"), -INF
        o, lse = A.fwd_varlen_gqa(q2, k2, v2, cu, 133, causal)
        got = (o, lse.t()) + A.bwd_varlen_gqa(q2, k2, v2, o, lse, d2, cu, 133, causal, deterministic=True)
        status()
        keep = torch.ones(q.shape[0], dtype=torch.bool, device=dev)
        keep[at] = False
        for x, y in zip(want, got):
            assert torch.equal(x[keep], y[keep])


def test_bad_cu_seqlens(dev):
    """Broken sequences are left out and reported; the call stays in bounds."""
    q, k, v, dout, cu = make(dev, "bf16", 4, 2, 64, [100, 60, 40], seed=3)
    good = A.fwd_varlen_gqa(q, k, v, cu, 100, True)
    status()
    for bad, fine in (([0, 100, 160, 201], slice(0, 160)), ([1, 100, 160, 200], slice(100, 200)), ([0, 100, 90, 200], None),
                      ([0, 200, 0, 200], None), ([-5, 100, 160, 200], slice(100, 200))):
        c = torch.tensor(bad, dtype=torch.int32, device=dev)
        o, lse = A.fwd_varlen_gqa(q, k, v, c, 100, True)
        status(True)
        if fine:
            assert torch.equal(o[fine], good[0][fine]) and torch.equal(lse[:, fine], good[1][:, fine])
        A.bwd_varlen_gqa(q, k, v, good[0], good[1], dout, c, 100, True)
        status(True)
    o, lse = A.fwd_varlen_gqa(q, k, v, cu, 99, True)  # the first is longer than it may be
    status(True)
    assert torch.equal(o[100:], good[0][100:])


def test_one_sequence(dev):
    """The path without a list: lengths below the bound, tokens behind the end, an empty and a broken sequence."""
    for L, T, bound in ((300, 300, 300), (129, 140, 500), (1, 9, 1), (16, 16, 16), (1000, 1003, 1001)):
        q, k, v, dout, cu = make(dev, "bf16", 8, 2, 64, [L], seed=L, behind=T - L)
        for causal in (True, False):
            o, lse = A.fwd_varlen_gqa(q, k, v, cu, bound, causal)
            check_fwd(o, lse, q, k, v, [L], causal, False)
            for det in (False, True):
                check_bwd(A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, bound, causal, deterministic=det), q, k, v, dout, [L], causal, False)
            status()
    for bad in ([1, 100], [0, 1004], [0, -1], [0, 1002]):
        c = torch.tensor(bad, dtype=torch.int32, device=dev)
        A.fwd_varlen_gqa(q, k, v, c, 1001, True)
        status(True)
        A.bwd_varlen_gqa(q, k, v, o, lse, dout, c, 1001, True)
        status(True)
    none = torch.zeros(2, dtype=torch.int32, device=dev)
    o, lse = A.fwd_varlen_gqa(q, k, v, none, 1001, True)
    assert (o == 0).all() and (lse == -INF).all()
    assert all((x == 0).all() for x in A.bwd_varlen_gqa(q, k, v, o, lse, dout.nan_to_num(), none, 1001, True))
    status()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 8, 2, 128), ("f16", 4, 4, 64), ("bf16", 5, 1, 80), ("f16", 71, 1, 16), ("f16", 32, 2, 112)])
def test_gradients_without_the_rounding_of_o(dev, dtype, Hq, Hkv, d, causal):
    """D is a sum over the keys: where a row sees one key its gradients are zero but for fp32's errors, and not what
    rounding O leaves."""
    for lens in ([1] * 20 + [2, 3, 1, 5, 8], [32, 33, 1, 31, 64, 300], [40], [129, 700]):
        q, k, v, dout, cu = make(dev, dtype, Hq, Hkv, d, lens, seed=d, behind=3)
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, max(lens), causal)
        got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, max(lens), causal, out_f32=True)
        status()
        check_bwd(got, q, k, v, dout, lens, causal, True, few=lambda L: L)
        if lens[0] == 1:  # dS = P (dP - D), dP of two summations, P from an LSE of fp32
            size = dout[:20].double().norm(dim=-1) * v[:20].double().norm(dim=-1).repeat_interleave(Hq // Hkv, 1)
            bound = size[..., None] * 2.0 ** -16 * k[:20].double().abs().repeat_interleave(Hq // Hkv, 1) / d ** 0.5
            assert (got[0][:20].double().abs() <= bound + 2.0 ** -20).all()


def test_deterministic_gradients(dev):
    q, k, v, dout, cu = make(dev, "bf16", 8, 2, 128, [900, 77, 400], seed=4)
    o, lse = A.fwd_varlen_gqa(q, k, v, cu, 900, True)
    first = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 900, True, deterministic=True)
    for _ in range(5):
        again = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 900, True, deterministic=True)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd(dev, dtype):
    """loss.backward() through parts of one projection, against the explicit calls and (fp32) against differences."""
    lens, Hq, Hkv, d = [40, 3, 25], 4, 2, 32
    T = sum(lens)
    g = torch.Generator(dev).manual_seed(5)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=dev).to(DT[dtype]).requires_grad_()
    cu = torch.tensor([0, 40, 43, 68], dtype=torch.int32, device=dev)
    w = torch.randn(T, Hq, d, generator=g, device=dev).to(DT[dtype])

    def loss(y):
        q, k, v = y.split((Hq, Hkv, Hkv), 1)
        return A.flash_attn_varlen_gqa_func(q, k, v, cu, 40, causal=True)

    o = loss(x)
    o.backward(w)
    q, k, v = x.detach().split((Hq, Hkv, Hkv), 1)
    ref, lse = A.fwd_varlen_gqa(q, k, v, cu, 40, True)
    assert torch.equal(ref, o)
    check_bwd(x.grad.split((Hq, Hkv, Hkv), 1), q, k, v, w, lens, True, False)
    status()
    if dtype != "f32":
        return
    # central differences: errors of eps^2 times the third derivative (below 1e-3 of the norms here) and of fp32 sums over eps
    eps = 1e-2
    for s in range(4):
        u = torch.randn(x.shape, generator=g, device=dev)
        u /= u.norm()
        with torch.no_grad():
            slope = float(((loss(x + eps * u).double() - loss(x - eps * u).double()) * w.double()).sum()) / (2 * eps)
        want = float((x.grad.double() * u.double()).sum())
        noise = 2.0 ** -22 * float((o.detach().double().abs() * w.double().abs()).sum()) / eps
        assert abs(slope - want) <= noise + 1e-3 * float(x.grad.norm())


def test_same_call_in_a_graph_and_on_two_streams(dev):
    """Captured forward and backward, replayed after the lengths have changed (fewer tokens than were captured), and two
    calls at once."""
    Hq, Hkv, d = 8, 2, 64
    q, k, v, dout, cu = make(dev, "bf16", Hq, Hkv, d, [120, 60, 200], seed=6)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, 300, True)
        A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 300, True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            o, lse = A.fwd_varlen_gqa(q, k, v, cu, 300, True)
            got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 300, True)
    for lens in ([120, 60, 200], [280, 0, 33], [1, 2, 3]):
        c = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(3)], dtype=torch.int32)
        cu.copy_(c)
        graph.replay()
        status()
        n = sum(lens)
        check_fwd(o, lse, q, k, v, lens, True, False)
        check_bwd(got, q, k, v, dout, lens, True, False)
        assert (o[n:] == 0).all()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    want = A.fwd_varlen_gqa(q, k, v, cu, 300, True)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s):
            x = A.fwd_varlen_gqa(q, k, v, cu, 300, True)
        with torch.cuda.stream(t):
            y = A.fwd_varlen_gqa(q, k, v, cu, 300, True)
        status()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, x, y))


def test_thousands_of_sequences(dev):
    """5000 sequences of 0 to 7 tokens and one of 900: the list of tiles."""
    rng = random.Random(7)
    lens = [rng.randint(0, 7) for _ in range(5000)] + [900]
    rng.shuffle(lens)
    Hq, Hkv, d = 4, 1, 64
    q, k, v, dout, cu = make(dev, "f16", Hq, Hkv, d, lens, seed=8)
    o, lse = A.fwd_varlen_gqa(q, k, v, cu, 900, True)
    got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, 900, True)
    status()
    at, pick = [0], set(rng.sample(range(len(lens)), 60)) | {lens.index(900)}
    for L in lens:
        at.append(at[-1] + L)
    for i in pick:
        t = slice(at[i], at[i + 1])
        check_fwd(o[t], lse[:, t], q[t], k[t], v[t], [lens[i]], True, False)
        check_bwd([x[t] for x in got], q[t], k[t], v[t], dout[t], [lens[i]], True, False)


def test_long_sequences_over_many_levels(dev):
    """Tiles of eight tokens (16 heads on one): 17000 tokens are more tiles than the list has levels."""
    lens, Hq, Hkv, d = [17000, 1, 9], 16, 1, 16
    q, k, v, dout, cu = make(dev, "bf16", Hq, Hkv, d, lens, seed=9)
    for causal in (True, False):
        o, lse = A.fwd_varlen_gqa(q, k, v, cu, 17000, causal)
        status()
        e = torch.cat([torch.logsumexp((q[i:i + 500].double().transpose(0, 1) @ k[:17000, 0].double().t() / 4).masked_fill(
            torch.arange(17000, device=dev)[None] > torch.arange(i, min(i + 500, 17000), device=dev)[:, None] if causal else
            torch.zeros(1, 17000, dtype=torch.bool, device=dev), -INF), -1) for i in range(0, 17000, 500)], 1)
        assert (lse[:, :17000].double() - e).abs().max() <= P.sum_error(17000) + P.sum_error(16) * 30 + 2.0 ** -18
        check_fwd(o[17000:], lse[:, 17000:], q[17000:], k[17000:], v[17000:], lens[1:], causal, False)


def test_empty_sequences_and_tokens_behind_them(dev):
    for lens, behind in (([0, 0, 0], 5), ([0], 3), ([0, 7, 0], 0), ([0, 0, 1], 130)):
        q, k, v, dout, cu = make(dev, "bf16", 4, 2, 64, lens, seed=10, behind=behind)
        for bound in (max(max(lens), 1), 3000):
            o, lse = A.fwd_varlen_gqa(q, k, v, cu, bound, True)
            check_fwd(o, lse, q, k, v, lens, True, False)
            check_bwd(A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, bound, True), q, k, v, dout, lens, True, False)
            status()
    q = torch.empty(0, 4, 64, device=dev, dtype=torch.float16)
    k = torch.empty(0, 2, 64, device=dev, dtype=torch.float16)
    o, lse = A.fwd_varlen_gqa(q, k, k, torch.zeros(3, dtype=torch.int32, device=dev), 8, True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert [x.shape[0] for x in A.bwd_varlen_gqa(q, k, k, o, lse, o, torch.zeros(3, dtype=torch.int32, device=dev), 8, True)] == [0, 0, 0]
    status()


def test_elements_past_32_bits(dev):
    """1350 sequences of 100 tokens with 128 query heads: 2.2e9 elements of q, and the last sequences' rows."""
    n, L, Hq, Hkv, d = 1350, 100, 128, 2, 128
    T = n * L
    q, dout = (torch.zeros(T, Hq, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.zeros(T, Hkv, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    assert q.numel() > 2 ** 31
    g = torch.Generator(dev).manual_seed(11)
    picks = [0, 7, n // 2, n - 2, n - 1]
    for i in picks:
        for x in (q, k, v, dout):
            x[i * L:(i + 1) * L] = torch.randn(L, x.shape[1], d, generator=g, device=dev).to(x.dtype)
    cu = torch.arange(0, T + 1, L, device=dev, dtype=torch.int32)
    o, lse = A.fwd_varlen_gqa(q, k, v, cu, L, True)
    got = A.bwd_varlen_gqa(q, k, v, o, lse, dout, cu, L, True)
    status()
    for i in picks:
        t = slice(i * L, (i + 1) * L)
        check_fwd(o[t], lse[:, t], q[t], k[t], v[t], [L], True, False)
        check_bwd([x[t] for x in got], q[t], k[t], v[t], dout[t], [L], True, False)
    t = slice(3 * L, 4 * L)
    assert (o[t] == 0).all() and all((x[t] == 0).all() for x in got)


def test_refusals(dev):
    """What the library refuses comes back as an error before anything runs; shapes and types in the Python layer."""
    q, k, v, dout, cu = make(dev, "bf16", 4, 2, 64, [20, 9], seed=12, fused=False)
    for bad in (lambda: A.fwd_varlen_gqa(q.transpose(0, 1), k, v, cu, 20, True), lambda: A.fwd_varlen_gqa(q[..., :32], k, v, cu, 20, True),
                lambda: A.fwd_varlen_gqa(q, k[:-1], v[:-1], cu, 20, True), lambda: A.fwd_varlen_gqa(q, k, v[:, :1], cu, 20, True),
                lambda: A.fwd_varlen_gqa(q, k, v, cu[:1], 20, True), lambda: A.fwd_varlen_gqa(q, k, v, cu[None], 20, True),
                lambda: A.fwd_varlen_gqa(q, k, v, cu, -1, True), lambda: A.fwd_varlen_gqa(q[:, :3], k, v, cu, 20, True),
                lambda: A.fwd_varlen_gqa(q, k, v, cu, 2 ** 31, True), lambda: A.fwd_varlen_gqa(q, k, v, cu, 20, True, scale=-1.0),
                lambda: A.fwd_varlen_gqa(q, k.expand(29, 2, 64).transpose(1, 2), v, cu, 20, True)):
        with pytest.raises((ValueError, TypeError, _lib.AttnError)):
            bad()
    for bad in (lambda: A.fwd_varlen_gqa(q, k.half(), v, cu, 20, True), lambda: A.fwd_varlen_gqa(q, k, v, cu.long(), 20, True),
                lambda: A.fwd_varlen_gqa(q.double(), k.double(), v.double(), cu, 20, True), lambda: A.fwd_varlen_gqa([q], k, v, cu, 20, True)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(_lib.AttnError):  # a workspace that is too small
        A.fwd_varlen_gqa(q, k, v, cu, 20, True, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    x = torch.zeros(29, 4 * 64 + 4, device=dev, dtype=torch.bfloat16)
    with pytest.raises(_lib.AttnError):  # tokens 8 bytes off the 16 that a copy needs
        A.fwd_varlen_gqa(x[:, :256].view(29, 4, 64), k, v, cu, 20, True)
    o, lse = A.fwd_varlen_gqa(q, k, v, cu, 20, True)
    for bad in (lambda: A.bwd_varlen_gqa(q, k, v, o[:-1], lse, dout, cu, 20, True), lambda: A.bwd_varlen_gqa(q, k, v, o, lse.t(), dout, cu, 20, True),
                lambda: A.bwd_varlen_gqa(q, k, v, o, lse, dout[:, :2], cu, 20, True)):
        with pytest.raises(ValueError):
            bad()
    status()

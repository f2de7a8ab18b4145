"""GPU tests of attention over a KV cache in pages against 64 bits, with bounds from the roundings that the kernels make, and
of what a serving program does with it."""
import random

import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import pages_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    _lib.load()
    return torch.device("cuda:0")


def status(bad=False):
    torch.cuda.synchronize()
    assert A.get_device_status() == (_lib.ATTN_ERR_DEVICE_INPUT if bad else _lib.ATTN_OK)


def make(dev, dtype, Hq, Hkv, Nq, lens, page, d, seed=0, M=None, size=1.0):
    """A cache whose pages lie in no order; whatever no sequence holds is NaN."""
    g, rng = torch.Generator(dev).manual_seed(seed), random.Random(seed)
    owned = [P.pages_of(L, page) for L in lens]
    M = max(owned + [1]) if M is None else M
    order = list(range(sum(owned) + 3))
    rng.shuffle(order)
    k, v = (torch.full((len(order), Hkv, page, d), NAN, device=dev, dtype=DT[dtype]) for _ in range(2))
    table = torch.full((len(lens), M), -7, dtype=torch.int32)
    rows = []
    for b, L in enumerate(lens):
        x = torch.randn(2, Hkv, L, d, generator=g, device=dev) * torch.exp(0.5 * torch.randn(2, Hkv, 1, d, generator=g, device=dev))
        x[0] *= size
        rows.append(x.to(DT[dtype]))
        for i in range(owned[b]):
            at = order.pop()
            table[b, i] = at
            n = min(page, L - i * page)
            k[at, :, :n], v[at, :, :n] = rows[b][0][:, i * page:i * page + n], rows[b][1][:, i * page:i * page + n]
    q = torch.randn(len(lens), Hq, Nq, d, generator=g, device=dev).to(DT[dtype])
    return q, k, v, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), rows


def check(got, q, rows, causal, out_f32, scale=None):
    o, lse = got
    B, Hq, Nq, d = q.shape
    dt = q.dtype
    for b, kv in enumerate(rows):
        Hkv, L = kv.shape[1], kv.shape[2]
        G = Hq // Hkv
        few = G * Nq <= 16
        for h in range(Hkv):
            x = q[b, h * G:(h + 1) * G].double()
            k, v = kv[0, h].double(), kv[1, h].double()
            want, e, p, size = P.attend(x, k, v, L - Nq, causal, scale)
            # P in two 16-bit halves (few rows), rounded once (many), or in fp32
            rho = 2.0 ** -24 if dt == torch.float32 else P.HALF[dt] ** 2 * 2 if few else P.HALF[dt]
            half = 2.0 ** -24 if out_f32 else P.HALF[dt]
            bo, be = P.attend_bounds(v, p, size, want, d, rho, half)
            go, ge = o[b, h * G:(h + 1) * G].double(), lse[b, h * G:(h + 1) * G].double()
            none = e == -float("inf")
            assert torch.equal(ge == -float("inf"), none) and (go[none] == 0).all()
            assert ((go - want).abs() <= bo).all(), (b, h, float(((go - want).abs() - bo).max()))
            assert ((ge - e)[~none].abs() <= be[~none] + e[~none].abs() * 2.0 ** -22).all(), (b, h)


LENS = [0, 1, 15, 16, 17, 31, 33, 64, 100, 127, 128, 129, 257, 700]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,Hq,Hkv,Nq,d", [
    ("bf16", 8, 2, 1, 128), ("f16", 4, 4, 1, 64), ("bf16", 4, 1, 2, 80), ("f16", 3, 1, 3, 16), ("bf16", 16, 1, 1, 128), ("f16", 4, 2, 5, 48),
    ("bf16", 4, 2, 9, 64), ("f16", 17, 1, 1, 128), ("bf16", 8, 2, 40, 128), ("f16", 2, 2, 130, 64), ("bf16", 6, 2, 100, 112),
    ("f32", 4, 2, 1, 64), ("f32", 3, 1, 7, 128), ("f32", 2, 2, 40, 16)])
def test_against_64_bits(dev, dtype, Hq, Hkv, Nq, d, page, causal):
    q, k, v, table, lens, rows = make(dev, dtype, Hq, Hkv, Nq, LENS, page, d, seed=page + d)
    for out_f32 in (True, False):
        check(A.fwd_kvpages(q, k, v, table, lens, causal, out_f32=out_f32), q, rows, causal, out_f32 or dtype == "f32")
        status()


@pytest.mark.parametrize("dtype,Hq,Hkv,Nq,d,page,lens", [
    ("bf16", 8, 2, 1, 128, 64, [4001, 12000, 1, 0, 9000]), ("f16", 8, 8, 1, 64, 16, [3000, 8191]), ("bf16", 4, 1, 4, 128, 128, [20001]),
    ("f16", 32, 8, 1, 128, 32, [1001]), ("bf16", 32, 8, 2, 80, 16, [5000, 300]), ("bf16", 8, 1, 128, 128, 64, [6000, 200]),
    ("f32", 4, 4, 1, 64, 64, [2500, 1]), ("f16", 8, 1, 3, 64, 16, [7000, 33, 513, 0, 2049]), ("bf16", 8, 2, 20, 128, 32, [4100, 1, 1300]),
    ("bf16", 16, 2, 30, 80, 16, [1537, 2600])])
def test_long_caches(dev, dtype, Hq, Hkv, Nq, d, page, lens):
    """Runs that end inside a cache, clusters, key ranges that are joined."""
    q, k, v, table, n, rows = make(dev, dtype, Hq, Hkv, Nq, lens, page, d, seed=3)
    check(A.fwd_kvpages(q, k, v, table, n, True, out_f32=True), q, rows, True, True)
    status()


@pytest.mark.parametrize("Nq", [1, 3, 50])
def test_many_sequences(dev, Nq):
    """More sequences than CTAs, tables far wider than the sequences need, and a bound on the lengths."""
    rng = random.Random(4)
    lens = [rng.choice((0, 1, 5, 40, 130)) for _ in range(400)]
    q, k, v, table, n, rows = make(dev, "bf16", 4, 2, Nq, lens, 32, 64, seed=4, M=300)
    for bound in (None, 130, 9600):
        check(A.fwd_kvpages(q, k, v, table, n, True, max_seqlen=bound, out_f32=True), q, rows, True, True)
        status()


@pytest.mark.parametrize("dtype,Nq", [("bf16", 1), ("f16", 30), ("f32", 2)])
def test_large_scores(dev, dtype, Nq):
    """Scores far apart: the running maximum moves, most weights vanish."""
    q, k, v, table, lens, rows = make(dev, dtype, 8, 2, Nq, [900, 33, 1500], 16, 64, seed=5, size=8.0)
    check(A.fwd_kvpages(q, k, v, table, lens, False, scale=0.3, out_f32=True), q, rows, False, True, 0.3)
    status()


@pytest.mark.parametrize("dtype,Nq", [("bf16", 1), ("f16", 40), ("f32", 1)])
def test_bad_lengths_and_pages(dev, dtype, Nq):
    """A length out of range counts as none, a page outside the pool as zeros; the others are as they were."""
    lens = [200, 300, 90, 128]
    q, k, v, table, n, rows = make(dev, dtype, 4, 2, Nq, lens, 32, 64, seed=6)
    good = A.fwd_kvpages(q, k, v, table, n, True)
    status()
    bad = n.clone()
    bad[1] = 321
    o, lse = A.fwd_kvpages(q, k, v, table, bad, True)
    status(True)
    assert (o[1] == 0).all() and (lse[1] == -float("inf")).all()
    for i in (0, 2, 3):
        assert torch.equal(o[i], good[0][i]) and torch.equal(lse[i], good[1][i])
    for number in (-1, k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = number
        o, lse = A.fwd_kvpages(q, k, v, t, n, True)
        status(True)
        zeros = rows[0].clone()
        zeros[:, :, 64:96] = 0
        check((o[:1], lse[:1]), q[:1], [zeros], True, dtype == "f32")
        for i in (1, 2, 3):
            assert torch.equal(o[i], good[0][i]) and torch.equal(lse[i], good[1][i])
    o, lse = A.fwd_kvpages(q, k, v, table, n, True, max_seqlen=250)
    status(True)
    assert (lse[1] == -float("inf")).all() and torch.isfinite(lse[0, :, -1]).all()


def test_nothing_to_read(dev):
    q = torch.randn(2, 4, 3, 64, device=dev, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32, device=dev)
    for pages, M in ((0, 0), (0, 3), (4, 0)):
        pool = torch.zeros(pages, 2, 16, 64, device=dev, dtype=torch.bfloat16)
        o, lse = A.fwd_kvpages(q, pool, pool, torch.zeros(2, M, dtype=torch.int32, device=dev), n, True)
        status()
        assert (o == 0).all() and (lse == -float("inf")).all()
    pool = torch.zeros(3, 2, 16, 64, device=dev, dtype=torch.bfloat16)
    o, lse = A.fwd_kvpages(q[:, :, :0], pool, pool, torch.zeros(2, 2, dtype=torch.int32, device=dev), n, True)
    assert o.shape == (2, 4, 0, 64)
    o, lse = A.fwd_kvpages(q[:0], pool, pool, torch.zeros(0, 2, dtype=torch.int32, device=dev), n[:0], True)
    assert o.shape == (0, 4, 3, 64)
    status()


@pytest.mark.parametrize("Nq", [1, 2, 64])
def test_same_bits_each_time_and_in_a_graph(dev, Nq):
    """The same call again, on another stream, and captured: replayed after the lengths and the tables have changed."""
    lens = [3000, 17, 800, 0]
    q, k, v, table, n, rows = make(dev, "bf16", 8, 2, Nq, lens, 64, 128, seed=7)
    first = A.fwd_kvpages(q, k, v, table, n, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = A.fwd_kvpages(q, k, v, table, n, True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = A.fwd_kvpages(q, k, v, table, n, True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, out))
    table.copy_(table[torch.tensor([2, 1, 0, 3], device=dev)])
    n.copy_(torch.tensor([700, 16, 2999, 0], dtype=torch.int32))
    rows = [rows[2][:, :, :700], rows[1][:, :, :16], rows[0][:, :, :2999], rows[3]]
    graph.replay()
    status()
    check(out, q, rows, True, False)


def test_two_calls_at_once(dev):
    """Two streams, each with its own workspace, thirty times."""
    a = make(dev, "bf16", 8, 2, 1, [9000, 400, 3000], 64, 128, seed=8)
    b = make(dev, "f16", 8, 2, 60, [5000, 77], 32, 64, seed=9)
    wa, wb = A.fwd_kvpages(*a[:5], True), A.fwd_kvpages(*b[:5], True)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(30):
        with torch.cuda.stream(s):
            x = A.fwd_kvpages(*a[:5], True)
        with torch.cuda.stream(t):
            y = A.fwd_kvpages(*b[:5], True)
        got.append((x, y))
    status()
    for x, y in got:
        assert torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1]) and torch.equal(y[0], wb[0]) and torch.equal(y[1], wb[1])


def test_a_pool_past_32_bits(dev):
    """Pages whose elements lie past 2^32: 5 GB of keys."""
    page, Hkv, d, pages = 128, 8, 128, 20000
    k, v = (torch.zeros(pages, Hkv, page, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    assert k.numel() > 2 ** 31
    ids = [19999, 16500, 3, 18001]
    for i in ids:
        k[i].normal_()
        v[i].normal_()
    table = torch.tensor([ids, [18001, 19999, 0, 0]], dtype=torch.int32, device=dev)
    lens = torch.tensor([500, 200], dtype=torch.int32, device=dev)
    rows = [torch.stack([torch.cat([x[i] for i in t], 1)[:, :L] for x in (k, v)]) for t, L in ((ids, 500), ([18001, 19999], 200))]
    for Nq in (1, 33):
        q = torch.randn(2, 16, Nq, d, device=dev, dtype=torch.bfloat16)
        check(A.fwd_kvpages(q, k, v, table, lens, True, out_f32=True), q, rows, True, True)
    new = torch.randn(3, Hkv, d, device=dev, dtype=torch.bfloat16)
    A.kvpages_append(k, v, table, new, new, torch.tensor([0, 3, 3], dtype=torch.int32, device=dev), lens)
    assert torch.equal(k[18001, :, 500 - 384:503 - 384].transpose(0, 1), new)
    A.kvpages_copy(k, v, torch.tensor([[18001, 17777]], dtype=torch.int32, device=dev))
    assert torch.equal(k[17777], k[18001]) and torch.equal(v[17777], v[18001])
    status()


def test_the_whole_path(dev):
    """A batch of prompts through packed attention and into pages, then tokens by decode steps: the same as whole
    sequences attended to at once."""
    page, Hq, Hkv, d = 16, 8, 2, 64
    lens, steps = [37, 5, 120, 64], 5
    g = torch.Generator(dev).manual_seed(10)
    B, M = len(lens), 12
    rows = [torch.randn(L + steps, Hq + 2 * Hkv, d, generator=g, device=dev).to(torch.bfloat16) for L in lens]
    table = torch.full((B, M), -1, dtype=torch.int32, device=dev)
    n, refs = torch.zeros(B, dtype=torch.int32, device=dev), torch.zeros(60, dtype=torch.int32, device=dev)
    k, v = (torch.full((60, Hkv, page, d), NAN, device=dev, dtype=torch.bfloat16) for _ in range(2))
    x = torch.cat([r[:L] for r, L in zip(rows, lens)])
    q, kn, vn = x.split((Hq, Hkv, Hkv), 1)
    new = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = torch.cat((torch.zeros(1, device=dev, dtype=torch.int32), new.cumsum(0).to(torch.int32)))
    o, lse = A.fwd_varlen_gqa(q, kn, vn, cu, max(lens), True)
    table, refs = A.kvpages_reserve(table, n, refs, new, page)
    A.kvpages_append(k, v, table, kn, vn, cu, n)
    n = n + new
    outs = [[o[cu[b]:cu[b + 1]]] for b in range(B)]
    one = torch.ones(B, dtype=torch.int32, device=dev)
    cu1 = torch.arange(B + 1, device=dev, dtype=torch.int32)
    for i in range(steps):
        y = torch.stack([r[L + i] for r, L in zip(rows, lens)])
        q, kn, vn = y.split((Hq, Hkv, Hkv), 1)
        table, refs = A.kvpages_reserve(table, n, refs, one, page)
        A.kvpages_append(k, v, table, kn, vn, cu1, n)
        n = n + one
        o, _ = A.fwd_kvpages(q.reshape(B, Hq, 1, d).contiguous(), k, v, table, n, True)
        for b in range(B):
            outs[b].append(o[b, :, 0][None])
    status()
    for b, r in enumerate(rows):
        got = torch.cat(outs[b]).transpose(0, 1)
        for h in range(Hkv):
            G = Hq // Hkv
            qh = r[:, h * G:(h + 1) * G].double().transpose(0, 1)
            kh, vh = r[:, Hq + h].double(), r[:, Hq + Hkv + h].double()
            want, _, p, size = P.attend(qh, kh, vh, 0, True)
            bound, _ = P.attend_bounds(vh, p, size, want, d, P.HALF[torch.bfloat16], P.HALF[torch.bfloat16])
            assert ((got[h * G:(h + 1) * G].double() - want).abs() <= bound).all()


def test_refusals(dev):
    q, k, v, table, n, _ = make(dev, "bf16", 4, 2, 1, [20, 9], 16, 64)
    for bad in (lambda: A.fwd_kvpages(q[:1], k, v, table, n), lambda: A.fwd_kvpages(q, k, v[:-1], table, n), lambda: A.fwd_kvpages(q, k, v, table[0], n),
                lambda: A.fwd_kvpages(q, k, v, table, n[:1]), lambda: A.fwd_kvpages(q[..., :32], k, v, table, n), lambda: A.fwd_kvpages(q[:, :3], k, v, table, n),
                lambda: A.fwd_kvpages(q, k[:, :, :8], v[:, :, :8], table, n), lambda: A.fwd_kvpages(q, k[:, :, :8].contiguous(), v[:, :, :8].contiguous(), table, n),
                lambda: A.fwd_kvpages(q, k, v, table, n, max_seqlen=0), lambda: A.fwd_kvpages(q, k, v, table, n, scale=0.0),
                lambda: A.kvpages_append(k, v, table, q[:, :2, 0], q[:, :1, 0], torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)),
                lambda: A.kvpages_append(k, v, table, k[0], v[0], torch.tensor([0, 1], dtype=torch.int32, device=dev)),
                lambda: A.kvpages_copy(k, k, torch.zeros(1, 2, dtype=torch.int32, device=dev)),
                lambda: A.kvpages_copy(k, v, torch.zeros(2, dtype=torch.int32, device=dev))):
        with pytest.raises((ValueError, _lib.AttnError)):
            bad()
    for bad in (lambda: A.fwd_kvpages(q, k.half(), v.half(), table, n), lambda: A.fwd_kvpages(q, k, v, table.long(), n),
                lambda: A.fwd_kvpages(q, k, v, table, n.long()), lambda: A.fwd_kvpages(q, k, v, table, None), lambda: A.kvpages_copy(k, v, table.long())):
        with pytest.raises(TypeError):
            bad()
    refs, row = torch.zeros(9, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    for bad in (lambda: A.kvpages_free(table, n, refs, row[:1], 16), lambda: A.kvpages_free(table, n, refs, row, 17), lambda: A.kvpages_free(n, n, refs, row, 16),
                lambda: A.kvpages_fork(table, n, refs, row, row[:1], 16), lambda: A.kvpages_reserve(table, n, refs[None], row, 16),
                lambda: A.kvpages_free(table, n, refs, row, 16, out=(table, n)), lambda: A.kvpages_free(table, n, refs, row, 16, out=(table, refs, n)),
                lambda: A.kvpages_reserve(table, n, refs, row, 16, out=(table, refs[:4]))):
        with pytest.raises((ValueError, _lib.AttnError)):
            bad()
    with pytest.raises(_lib.AttnError):  # an output that lies over an input which it does not follow
        A.kvpages_free(table, n, refs, row, 16, out=(table, row, refs))
    with pytest.raises(TypeError):
        A.kvpages_reserve(table, n, refs.long(), row, 16)
    status()

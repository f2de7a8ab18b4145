"""GPU tests of a KV cache in pages: the books against a plain implementation, number by number, with everything that they
refuse; copies and appended tokens bit by bit; and what a serving program does with them (in place, graphs, streams)."""
import random

import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from exact_attention_50_gb300 import attention as A
from tests import pages_plain as P

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    _lib.load()
    return torch.device("cuda:0")


def status(bad):
    torch.cuda.synchronize()
    assert A.get_device_status() == (_lib.ATTN_ERR_DEVICE_INPUT if bad else _lib.ATTN_OK)


def ints(x, dev, shape=None):
    t = torch.tensor(x, dtype=torch.int32, device=dev)
    return t if shape is None else t.reshape(shape)


def state(rng, B, M, pages, page, shared=True):
    """A table that a program may have: some rows share their first full pages, some hold pages beyond their length, some
    are empty."""
    order = list(range(pages))
    rng.shuffle(order)
    table, lens, refs = [[-1] * M for _ in range(B)], [0] * B, [0] * pages
    for b in range(B):
        if rng.random() < 0.25:
            continue
        L = rng.choice((0, 1, page, page * M, rng.randint(0, page * M)))
        need = min(M, P.pages_of(L, page) + rng.choice((0, 0, 1)))
        row = []
        if shared and b and rng.random() < 0.4:
            row = [x for x in table[b - 1][:min(lens[b - 1], L) // page] if x >= 0]
        if need - len(row) > len(order):
            continue
        row += [order.pop() for _ in range(need - len(row))]
        table[b][:len(row)] = row
        lens[b] = L
        for x in row:
            refs[x] += 1
    return table, lens, refs


SIZES = [(1, 1, 1, 16), (1, 3, 2, 16), (5, 4, 21, 32), (9, 0, 4, 64), (3, 7, 0, 16), (40, 33, 700, 16), (64, 66, 5000, 64), (300, 9, 3001, 128),
         (70, 130, 20011, 16)]


def outs(given, in_place):
    return given if in_place else None


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,M,pages,page", SIZES)
def test_free(dev, B, M, pages, page, in_place):
    rng = random.Random(B * 7 + pages)
    table, lens, refs = state(rng, B, M, pages, page)
    keep = [rng.choice((0, 1, L, L + 3, rng.randint(0, L + 1), max(0, L - 9))) for L in lens]
    for spoil in (False, True):
        if spoil:
            keep[rng.randrange(B)] = -1
        want = P.free(table, lens, refs, keep, page)
        t, n, r = ints(table, dev, (B, M)), ints(lens, dev), ints(refs, dev)
        got = A.kvpages_free(t, n, r, ints(keep, dev), page, out=outs((t, n, r), in_place))
        status(want[3])
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,M,pages,page", SIZES)
def test_fork(dev, B, M, pages, page, in_place):
    rng = random.Random(B * 11 + pages)
    for spoil in range(3):
        table, lens, refs = state(rng, B, M, pages, page)
        empty = [b for b in range(B) if lens[b] == 0 and (M == 0 or table[b][0] < 0)]
        rng.shuffle(empty)
        src, dst = [rng.randrange(B) for _ in empty], empty
        if spoil == 1:  # twice the same dst, a dst that is not empty, numbers out of range, more forks than pages
            dst = dst + dst[:2] + [rng.randrange(B), B, -1, 0]
            src = src + [rng.randrange(B) for _ in dst[len(src):-2]] + [-1, B]
            src, dst = src[:len(dst)], dst[:len(src)]
        if spoil == 2:
            left = 2
            for i in range(pages):
                if refs[i] == 0:
                    left -= 1
                    refs[i] = 1 if left < 0 else 0
        want = P.fork(table, lens, refs, src, dst, page)
        t, n, r = ints(table, dev, (B, M)), ints(lens, dev), ints(refs, dev)
        got = A.kvpages_fork(t, n, r, ints(src, dev), ints(dst, dev), page, out=outs((t, n, r), in_place))
        status(want[4])
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
        assert got[3].tolist() == want[3]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,M,pages,page", SIZES)
def test_reserve(dev, B, M, pages, page, in_place):
    rng = random.Random(B * 13 + pages)
    for spoil in range(3):
        table, lens, refs = state(rng, B, M, pages, page)
        new = [rng.choice((0, 1, page - 1, page, rng.randint(0, max(0, M * page - L)))) for L in lens]
        if spoil < 2:
            new = [min(x, M * page - L) for x, L in zip(new, lens)]
        if spoil == 2:
            new[rng.randrange(B)] = -5
            lens[rng.randrange(B)] = -1
        if spoil == 1:  # the pages run out on the way
            left = max(1, pages // 20)
            for i in range(pages):
                if refs[i] == 0:
                    left -= 1
                    refs[i] = 1 if left < 0 else 0
        want = P.reserve(table, lens, refs, new, page)
        t, r = ints(table, dev, (B, M)), ints(refs, dev)
        got = A.kvpages_reserve(t, ints(lens, dev), r, ints(new, dev), page, out=outs((t, r), in_place))
        status(want[2])
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,M,pages,page", SIZES + [(200, 40, 100003, 16)])
def test_compact(dev, B, M, pages, page, in_place):
    rng = random.Random(B * 17 + pages)
    for spoil in (False, True):
        table, lens, refs = state(rng, B, M, pages, page)
        if spoil and M and pages:
            table[0][0] = pages + 3           # outside the pool
            spare = [i for i, r in enumerate(refs) if r == 0]
            if spare and spare[-1] >= sum(r > 0 for r in refs):
                table[B - 1][M - 1] = spare[-1]  # counted as free
        want = P.compact(table, refs)
        t, r = ints(table, dev, (B, M)), ints(refs, dev)
        got = A.kvpages_compact(t, r, out=outs((t, r), in_place))
        status(want[4])
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        assert got[2].tolist() == want[2] and got[3].tolist() == [want[3]]


def test_compact_entry_that_counts_as_free(dev):
    """A stale entry keeps its number and raises the status, before the used pages' end as behind it."""
    for entry in (1, 3, 6):  # U = 4: free places 1 and 3 are filled from 5 and 7, page 6 is free and stays so
        table, refs = [[0, 2, 5], [5, 7, entry]], [1, 0, 1, 0, 0, 2, 0, 1]
        want = P.compact(table, refs)
        assert want[4] and want[0][1] == [1, 3, entry]
        got = A.kvpages_compact(ints(table, dev), ints(refs, dev))
        status(True)
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2] and got[3].tolist() == [4]


def test_cut_inside_a_shared_page(dev):
    """A row cut inside a page that another shares gets it for itself by a fork: what is appended leaves the other as it was."""
    page, d, Hkv = 16, 64, 2
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(9, Hkv, page, d, generator=g).to(dev, torch.bfloat16) for _ in range(2))
    table, lens, refs = ints([[4, 7, 2], [4, 7, -1], [-1, -1, -1]], dev), ints([40, 32, 0], dev), ints([0, 0, 1, 0, 2, 0, 0, 2, 0], dev)
    before = k[[4, 7, 2]].clone(), v[[4, 7, 2]].clone()
    table, lens, refs = A.kvpages_free(table, lens, refs, ints([99, 21, 0], dev), page)
    assert lens.tolist() == [40, 21, 0] and refs.tolist() == [0, 0, 1, 0, 2, 0, 0, 2, 0]
    table, lens, refs, copies = A.kvpages_fork(table, lens, refs, ints([1], dev), ints([2], dev), page)
    A.kvpages_copy(k, v, copies)
    table, lens, refs = A.kvpages_free(table, lens, refs, ints([99, 0, 99], dev), page)
    assert table.tolist() == [[4, 7, 2], [-1, -1, -1], [4, 0, -1]] and refs.tolist() == [1, 0, 1, 0, 2, 0, 0, 1, 0]
    x = torch.randn(5, Hkv, d, generator=g).to(dev, torch.bfloat16)
    A.kvpages_append(k, v, table, x, -x, ints([0, 0, 0, 5], dev), lens)
    status(False)
    assert torch.equal(k[[4, 7, 2]], before[0]) and torch.equal(v[[4, 7, 2]], before[1])
    assert torch.equal(k[0, :, :5], before[0][1][:, :5]) and torch.equal(k[0, :, 5:10], x.transpose(0, 1)) and torch.equal(v[0, :, 5:10], -x.transpose(0, 1))


def test_books_of_every_row(dev):
    """65536 rows: the largest table."""
    B, page = 65536, 16
    table, lens, refs = torch.full((B, 2), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), torch.zeros(B + 9, dtype=torch.int32)
    half = B // 2
    table[:half, 0] = torch.arange(half, dtype=torch.int32) + 5
    lens[:half] = 1 + torch.arange(half, dtype=torch.int32) % 16
    refs[5:half + 5] = 1
    src, dst = torch.arange(half, dtype=torch.int32).flip(0), torch.arange(half, B, dtype=torch.int32)
    want = P.fork(table.tolist(), lens.tolist(), refs.tolist(), src.tolist(), dst.tolist(), page)
    got = A.kvpages_fork(*(x.to(dev) for x in (table, lens, refs, src, dst)), page)
    status(want[4])
    assert all(got[i].tolist() == want[i] for i in range(4))
    new = torch.ones(B, dtype=torch.int32)
    want = P.reserve(want[0], want[1], want[2], new.tolist(), page)
    got = A.kvpages_reserve(got[0], got[1], got[2], new.to(dev), page)
    status(want[2])
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1]


# ------------------------------------------------------------------------------------------ copies
@pytest.mark.parametrize("dtype,Hkv,page,d", [("bf16", 8, 64, 128), ("f16", 1, 16, 16), ("f32", 3, 32, 80), ("bf16", 16, 128, 128), ("f16", 2, 16, 48)])
def test_copy(dev, dtype, Hkv, page, d):
    n, g = 37, torch.Generator(dev).manual_seed(1)
    k, v = (torch.randn(n, Hkv, page, d, generator=g, device=dev).to(DT[dtype]) for _ in range(2))
    k[5, 0, 0, 0], v[6, 0, 1, 1] = float("nan"), float("inf")
    pairs = [[5, 30], [-1, -1], [6, 31], [5, 32], [7, 7], [-1, -1], [36, 0]] + [[-1, -1]] * 50
    wk, wv = k.clone(), v.clone()
    for a, b in pairs:
        if a >= 0:
            wk[b], wv[b] = k[a], v[a]
    A.kvpages_copy(k, v, ints(pairs, dev))
    status(False)
    same = lambda x, y: torch.equal(x.view(torch.int16 if x.element_size() == 2 else torch.int32), y.view(torch.int16 if y.element_size() == 2 else torch.int32))
    assert same(k, wk) and same(v, wv)
    A.kvpages_copy(k, v, ints([[3, n], [n, 3], [-1, 4], [4, -2]], dev))  # out of range: passed over
    status(True)
    assert same(k, wk) and same(v, wv)
    A.kvpages_copy(k, v, torch.empty((0, 2), dtype=torch.int32, device=dev))
    status(False)


# ------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,Hkv,page,d", [("bf16", 8, 64, 128), ("f16", 1, 16, 16), ("f32", 3, 32, 80), ("bf16", 5, 128, 64), ("f32", 8, 16, 128)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(dev, dtype, Hkv, page, d, fused):
    """Sequences that begin and end inside pages, that append nothing, one token, many; tokens behind the last; a projection's
    output cut into parts.  Everything else stays."""
    lens = [0, 1, page - 1, page, page + 5, 3 * page, 0, 7, 2]
    new = [3 * page + 1, 1, 2, 0, page, 2 * page - 3, 0, 1, 70]
    B, M = len(lens), 7
    owned = [P.pages_of(L + n, page) for L, n in zip(lens, new)]
    g, rng = torch.Generator(dev).manual_seed(2), random.Random(3)
    pages = sum(owned) + 4
    order = list(range(pages))
    rng.shuffle(order)
    table = [[-1] * M for _ in range(B)]
    for b, n in enumerate(owned):
        table[b][:n] = [order.pop() for _ in range(n)]
    T = sum(new) + 5
    x = torch.randn(T, 3 * Hkv, d, generator=g, device=dev).to(DT[dtype])
    kn, vn = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    if not fused:
        kn, vn = kn.contiguous(), vn.contiguous()
    k, v = (torch.randn(pages, Hkv, page, d, generator=g, device=dev).to(DT[dtype]) for _ in range(2))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    for held in (lens, None):
        wk, wv = k.clone(), v.clone()
        for b in range(B):
            for i in range(new[b]):
                pos = (held[b] if held else 0) + i
                wk[table[b][pos // page], :, pos % page] = kn[cu[b] + i]
                wv[table[b][pos // page], :, pos % page] = vn[cu[b] + i]
        A.kvpages_append(k, v, ints(table, dev), kn, vn, ints(cu, dev), None if held is None else ints(held, dev))
        status(False)
        assert torch.equal(k, wk) and torch.equal(v, wv)


def test_append_many_sequences(dev):
    """A token each of 3000 sequences and runs of empty ones: the search over cu_seqlens."""
    page, d, B = 16, 64, 3000
    new = [(b % 3 != 1) * (1 + (b % 700 == 0) * 30) for b in range(B)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    M = 3
    table = torch.arange(B * M, device=dev, dtype=torch.int32).reshape(B, M)
    k, v = (torch.zeros(B * M, 1, page, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    x = torch.randn(cu[-1], 1, d, device=dev, dtype=torch.bfloat16)
    lens = ints([b % 17 for b in range(B)], dev)
    A.kvpages_append(k, v, table, x, -x, ints(cu, dev), lens)
    status(False)
    seq = torch.repeat_interleave(torch.arange(B, device=dev), ints(new, dev).long())
    pos = lens.long()[seq] + torch.arange(cu[-1], device=dev) - ints(cu, dev).long()[seq]
    wk, wv = torch.zeros_like(k), torch.zeros_like(v)
    wk[table.long()[seq, pos // page], 0, pos % page] = x[:, 0]
    wv[table.long()[seq, pos // page], 0, pos % page] = -x[:, 0]
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_append_refuses_tokens_without_a_place(dev):
    page, d = 16, 64
    k, v = (torch.zeros(6, 2, page, d, device=dev, dtype=torch.float16) for _ in range(2))
    x = torch.ones(12, 2, d, device=dev, dtype=torch.float16)
    table = ints([[0, 1], [2, -1], [9, 3], [4, 5]], dev)
    # sequence 0 has no room for its tokens, 1's second page is not there, 2's first is outside the pool
    A.kvpages_append(k, v, table, x, x, ints([0, 2, 6, 9, 12], dev), ints([31, 14, 3, 16], dev))
    status(True)
    want = torch.zeros_like(k)
    want[2, :, 14:] = 1
    want[5, :, :3] = 1
    assert torch.equal(k, want) and torch.equal(v, want)
    for cu in ([1, 2, 6, 9, 12], [0, 2, 6, 9, 13], [0, 2, 6, 9, -1]):
        A.kvpages_append(k, v, table, x * 2, x, ints(cu, dev), ints([0, 0, 0, 0], dev))
        status(True)
        assert torch.equal(k, want)
    A.kvpages_append(k, v, table, x * 2, x * 2, ints([0, 5, 3, 9, 12], dev), ints([0, 0, 99, 99], dev))  # cu goes back: nothing out of bounds
    status(True)


# ------------------------------------------------------------------------------------------ together
def test_a_search_in_a_graph(dev):
    """A step of a search (cut, fork, copy, reserve, append) captured once, in place, and replayed with other numbers; the
    cache that the tables give is compared with one kept token by token."""
    page, Hkv, d, B, M, pages = 16, 2, 32, 12, 8, 90
    rng, g = random.Random(5), torch.Generator(dev).manual_seed(5)
    k, v = (torch.full((pages, Hkv, page, d), float("nan"), device=dev, dtype=torch.bfloat16) for _ in range(2))
    table, lens, refs = ints([[-1] * M] * B, dev), ints([0] * B, dev), ints([0] * pages, dev)
    keep, new, src, dst = (ints([0] * n, dev) for n in (B, B, 3, 3))
    cu = ints([0] * (B + 1), dev)
    kn, vn = (torch.zeros(60, Hkv, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    held = [[] for _ in range(B)]

    def step():
        A.kvpages_free(table, lens, refs, keep, page, out=(table, lens, refs))
        copies = A.kvpages_fork(table, lens, refs, src, dst, page, out=(table, lens, refs))[3]
        A.kvpages_copy(k, v, copies)
        A.kvpages_reserve(table, lens, refs, new, page, out=(table, refs))
        A.kvpages_append(k, v, table, kn, vn, cu, lens)
        lens.add_(new)

    stream = torch.cuda.Stream()
    graph = None
    for turn in range(14):
        ended = rng.sample(range(B), 4)
        keeps = [0 if b in ended[:3] else max(0, len(h) - rng.choice((0, 0, 2, 20))) for b, h in enumerate(held)]
        s = [rng.choice([b for b in range(B) if b not in ended[:3]]) for _ in range(3)]
        n = [rng.choice((0, 1, 1, 3, 9)) for _ in range(B)]
        n = [min(x, M * page - min(L, len(h))) for x, L, h in zip(n, keeps, held)]
        for i, b in enumerate(ended[:3]):
            n[b] = min(n[b], M * page - min(keeps[s[i]], len(held[s[i]])))
        x = torch.randn(60, Hkv, d, generator=g, device=dev).to(torch.bfloat16)
        c = [0]
        for y in n:
            c.append(c[-1] + y)
        assert c[-1] <= 60
        for to, y in ((keep, keeps), (new, n), (src, s), (dst, ended[:3]), (cu, c)):
            to.copy_(torch.tensor(y, dtype=torch.int32))
        kn.copy_(x)
        vn.copy_(-x)
        if turn == 3:
            torch.cuda.synchronize()
            saved = [t.clone() for t in (table, lens, refs, k, v)]
            with torch.cuda.stream(stream):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    step()
            for t, y in zip((table, lens, refs, k, v), saved):
                t.copy_(y)
        if graph is None:
            step()
        else:
            graph.replay()
        status(False)
        held = [h[:L] for h, L in zip(held, keeps)]
        for b, y in zip(ended[:3], s):
            held[b] = list(held[y])
        for b in range(B):
            held[b] = held[b] + [x[c[b] + i] for i in range(n[b])]
        assert lens.tolist() == [len(h) for h in held]
        t, owned = table.tolist(), [0] * pages
        for row in t:
            for y in row:
                if y >= 0:
                    owned[y] += 1
        assert refs.tolist() == owned
        for b, h in enumerate(held):
            for pos in (0, len(h) // 2, len(h) - 1):
                if h:
                    assert torch.equal(k[t[b][pos // page], :, pos % page], h[pos]) and torch.equal(v[t[b][pos // page], :, pos % page], -h[pos])
    # and the pool's pages in front
    t2, r2, copies, used = A.kvpages_compact(table, refs)
    A.kvpages_copy(k, v, copies)
    status(False)
    assert int(used) == sum(x > 0 for x in refs.tolist()) and all(x > 0 for x in r2.tolist()[:int(used)])
    t = t2.tolist()
    for b, h in enumerate(held):
        for pos in range(len(h)):
            assert torch.equal(k[t[b][pos // page], :, pos % page], h[pos])

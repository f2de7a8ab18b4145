"""A KV cache in pages, from the prompts that fill it to the tokens that follow, as measured cases.

The operators, in the order in which a program uses them:

  prompt    attention of whole prompts of different lengths, packed one behind the other, with fewer
            kv heads than query heads; "train" is the same with its gradients
  append    the tokens' keys and values written into the pages that a table gives each sequence
  paged     attention of one or a few new tokens, or of a chunk of a prompt, over such pages
  beams     sequences dropped or cut short, forked and given room: page tables and reference counts,
            and the copies of the pages that a fork may not share
  compact   the pages in use moved to the front of the pool

``run`` computes them in plain float32 torch operations, or, where ``own`` is set, calls the
package.  ``exact`` computes them once more from their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HEADS = ((32, 8), (32, 32), (8, 8), (16, 2), (12, 4), (4, 1))


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------------------- cases
def prompt(name, op, n, lo, hi, Hq, Hkv, d, dtype, causal, fused):
    """n sequences of lo to hi tokens; fused: q, k and v are parts of one projection's output."""
    return dict(name=name, op=op, n=n, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, causal=causal, fused=fused)


def paged(name, B, Hq, Hkv, Nq, lo, hi, page, d, dtype, causal):
    return dict(name=name, op="paged", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, lo=lo, hi=hi, page=page, d=d, dtype=dtype, causal=causal)


def append(name, B, Hkv, new_lo, new_hi, lo, hi, page, d, dtype):
    return dict(name=name, op="append", B=B, Hkv=Hkv, new_lo=new_lo, new_hi=new_hi, lo=lo, hi=hi, page=page, d=d, dtype=dtype)


def beams(name, B, forks, Hkv, lo, hi, page, d, dtype):
    return dict(name=name, op="beams", B=B, forks=forks, Hkv=Hkv, lo=lo, hi=hi, page=page, d=d, dtype=dtype)


def compact(name, B, Hkv, lo, hi, spare, page, d, dtype):
    """spare: the share of the pool's pages that are free, in percent."""
    return dict(name=name, op="compact", B=B, Hkv=Hkv, lo=lo, hi=hi, spare=spare, page=page, d=d, dtype=dtype)


def listed():
    return [
        # one short prompt: the time before its first token
        prompt("prompt one short", "prompt", 1, 201, 201, 32, 8, 128, "bf16", True, True),
        # prompts of a batch, of very different lengths
        prompt("prompt batch", "prompt", 16, 64, 2048, 32, 8, 128, "bf16", True, True),
        # a training step's forward and backward on packed sequences
        prompt("train batch", "train", 16, 64, 2048, 32, 8, 128, "bf16", True, False),
        # many short sequences, seen whole, 64 columns
        prompt("train short", "train", 200, 9, 150, 16, 2, 64, "f16", False, True),
        # one token of one conversation with a short history: the call's latency
        paged("paged one short", 1, 32, 8, 1, 1001, 1001, 64, 128, "bf16", True),
        # the benchmark's decode workload, its caches in pages
        paged("paged decode", 8, 32, 8, 1, 16384, 32768, 64, 128, "bf16", True),
        # a draft of five tokens checked at once, every head with its own keys, 64 columns, small pages
        paged("paged draft", 4, 32, 32, 5, 300, 4111, 16, 64, "f16", True),
        # a chunk of a long prompt against the pages of what came before it
        paged("paged chunk", 2, 32, 8, 2048, 16384, 16384, 128, 128, "bf16", True),
        # every decode step writes one token per sequence
        append("append one token", 8, 8, 1, 1, 16384, 32768, 64, 128, "bf16"),
        # whole prompts of different lengths go into empty sequences
        append("append prompts", 16, 8, 64, 4096, 0, 0, 16, 128, "bf16"),
        # a step of a search: some sequences end, some lose the last tokens, others are forked
        beams("pages beams", 64, 24, 8, 500, 4096, 64, 128, "bf16"),
        # a pool of which two fifths are free, after many sequences have come and gone
        compact("pages compact", 48, 8, 1000, 8192, 40, 64, 128, "bf16"),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("prompt", "train", "paged", "paged", "append", "beams", "compact"))
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice((64, 128, 128, 80))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    page = rng.choice((16, 32, 64, 128))
    if op in ("prompt", "train"):
        n = spread(rng, 1, 64)
        hi = spread(rng, 1, min(2048, int(8192 / math.sqrt(n))))  # scores of the plain form: no more than "prompt batch" has
        lo = rng.choice((hi, max(1, hi // 2), max(1, hi // 30)))
        c = prompt("", op, n, lo, hi, Hq, Hkv, d, dtype, rng.choice((True, True, False)), rng.choice((True, False)))
    elif op == "paged":
        B = rng.randint(1, 8)
        Nq = rng.choice((1, 1, rng.randint(2, 8), spread(rng, 9, 1024)))
        hi = spread(rng, 16, 8192 if Nq > 8 or B * Hkv > 64 else 32768)
        lo = rng.choice((hi, hi // 2, hi // 7))
        c = paged("", B, Hq, Hkv, Nq, lo, hi, page, d, dtype, rng.choice((True, True, False)))
    elif op == "append":
        hi = rng.choice((0, spread(rng, 1, 8192)))
        new = rng.choice((1, rng.randint(2, 8), spread(rng, 9, 4096)))
        c = append("", rng.randint(1, 16), Hkv, rng.choice((new, max(1, new // 20))), new, rng.choice((hi, hi // 2)), hi, page, d, dtype)
    elif op == "beams":
        B, hi = spread(rng, 8, 64), spread(rng, 16, 4096)
        c = beams("", B, rng.randint(1, B // 4), min(Hkv, 8), rng.choice((hi, hi // 2, hi // 7)), hi, page, d, dtype)
    else:
        hi = spread(rng, 16, 8192)
        c = compact("", spread(rng, 4, 48), min(Hkv, 8), rng.choice((hi // 2, hi // 7)), hi, rng.choice((20, 50, 75)), page, d, dtype)
    del c["name"]
    return c


def uneven(n, lo, hi, by=0.6180339887498949):
    """n whole numbers over [lo, hi], in no order, the first of them hi."""
    return [hi - int((hi - lo) * ((i * by) % 1.0)) for i in range(n)]


def ceil_div(a, b):
    return -(-a // b)


def visible(L, Nq, causal):
    """(query, key) pairs of one head."""
    return sum(min(L, max(0, L - Nq + i + 1)) for i in range(Nq)) if causal else Nq * L


# --------------------------------------------------------------------------------------- inputs
def normal(gen, shape, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)


def rows(gen, T, H, d, dev):
    """[T, H, d]: keys or values as a projection gives them, some columns and tokens far larger than others."""
    x = normal(gen, (T, H, d), dev)
    x *= torch.exp(0.5 * normal(gen, (1, H, d), dev) - 0.25)
    return x.mul_(torch.exp(0.3 * normal(gen, (T, H, 1), dev)))


def pool(gen, c, pages, dev):
    """[pages, Hkv, page, d] keys and values."""
    shape = (c["Hkv"], c["page"], c["d"])
    return tuple(rows(gen, pages * c["page"], c["Hkv"], c["d"], dev).to(DT[c["dtype"]])
                 .reshape(pages, c["page"], c["Hkv"], c["d"]).transpose(1, 2).contiguous().reshape((pages,) + shape) for _ in range(2))


def table_of(owned, M, order):
    """[B, M]: sequence b's owned[b] pages, taken from `order` one sequence after the other, then -1."""
    t = np.full((len(owned), M), -1, np.int32)
    at = 0
    for b, n in enumerate(owned):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def prepare(case, seed):
    c, dev = case, device()
    gen = torch.Generator(dev).manual_seed(int(seed) * 1000003 + 29)
    some = np.random.RandomState((int(seed) * 7919 + 13) % (2 ** 31))
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)  # noqa: E731
    dt, Hkv, d = DT[c["dtype"]], c["Hkv"], c["d"]
    st = {"case": c}
    if c["op"] in ("prompt", "train"):
        lens = uneven(c["n"], c["lo"], c["hi"])
        T, Hq = sum(lens), c["Hq"]
        st["cu"], st["longest"] = i32(np.concatenate(([0], np.cumsum(lens)))), c["hi"]
        x = torch.cat((normal(gen, (T, Hq, d), dev), rows(gen, T, Hkv, d, dev), rows(gen, T, Hkv, d, dev)), 1).to(dt)
        st["q"], st["k"], st["v"] = x.split((Hq, Hkv, Hkv), 1)
        if not c["fused"]:
            st["q"], st["k"], st["v"] = (y.contiguous() for y in (st["q"], st["k"], st["v"]))
        if c["op"] == "train":
            st["dout"] = normal(gen, (T, Hq, d), dev).to(dt)
        return st
    page, B = c["page"], c["B"]
    lens = uneven(B, c["lo"], c["hi"])
    st["lens"] = i32(lens)
    if c["op"] == "paged":
        owned = [ceil_div(L, page) for L in lens]
        M = ceil_div(c["hi"], page)
        pages = sum(owned) + 3
        st["k"], st["v"] = pool(gen, c, pages, dev)
        st["table"] = i32(table_of(owned, M, some.permutation(pages)))
        st["q"] = normal(gen, (B, c["Hq"], c["Nq"], d), dev).to(dt)
    elif c["op"] == "append":
        new = uneven(B, c["new_lo"], c["new_hi"], 0.7548776662466927)
        owned = [ceil_div(L + n, page) for L, n in zip(lens, new)]
        pages = sum(owned) + 3
        st["k"], st["v"] = pool(gen, c, pages, dev)
        st["table"] = i32(table_of(owned, max(owned), some.permutation(pages)))
        st["cu"] = i32(np.concatenate(([0], np.cumsum(new))))
        st["k_new"], st["v_new"] = (rows(gen, sum(new), Hkv, d, dev).to(dt) for _ in range(2))
    else:
        if c["op"] == "beams":  # the last rows of the table are empty: room for the forks
            lens = [L if b < B - c["forks"] else 0 for b, L in enumerate(lens)]
            st["lens"] = i32(lens)
        owned = [ceil_div(L, page) for L in lens]
        M = ceil_div(c["hi"], page) + 1
        if c["op"] == "beams":
            pages = sum(owned) + B + c["forks"] + 3
            at = some.permutation(pages)
        else:
            pages = max(1, sum(owned) * 100 // (100 - c["spare"]))
            at = some.permutation(pages)
        table = table_of(owned, M, at)
        half = B // 2 if c["op"] == "beams" else 0
        for b in range(1, half, 3):  # beams that share their first pages with the one before
            n = min(owned[b - 1], owned[b]) // 2
            table[b, :n] = table[b - 1, :n]
        refs = np.bincount(table[table >= 0].astype(np.int64), minlength=pages)
        st["table"], st["refs"] = i32(table), i32(refs)
        st["k"], st["v"] = pool(gen, c, pages, dev)
        if c["op"] == "beams":
            n, f = B - c["forks"], c["forks"]
            keep = np.array(lens)
            keep[2:n:7] = 0                                     # these have ended
            keep[3:n:5] = np.maximum(keep[3:n:5] - 9, 0)        # these lose the tokens of a rejected draft
            st["keep"] = i32(keep)
            st["src"], st["dst"] = i32(some.randint(0, n, f)), i32(n + some.permutation(f))
            st["new"] = i32(some.randint(0, 6, B))
    return st


# ---------------------------------------------------------------------------------- plain forms
def padded(x, cu, n, N):
    """[T, H, d] -> float32 [n, H, N, d], zeros behind each sequence; and which of its rows are tokens."""
    j = torch.arange(N, device=x.device)[None]
    start = cu[:-1, None].long()
    held = j < (cu[1:, None] - start)
    at = torch.where(held, start + j, torch.zeros_like(j))
    return (x[at].float() * held[:, :, None, None]).transpose(1, 2), held


def plain_prompt(st):
    """Scores of the padded batch, [n, Hkv, G, N, N]; the gradients by their formulas."""
    c = st["case"]
    n, N, G, Hkv, d = c["n"], c["hi"], c["Hq"] // c["Hkv"], c["Hkv"], c["d"]
    scale = 1.0 / math.sqrt(d)
    q, held = padded(st["q"], st["cu"], n, N)
    k, v = (padded(st[x], st["cu"], n, N)[0] for x in ("k", "v"))
    q = q.reshape(n, Hkv, G * N, d)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).reshape(n, Hkv, G, N, N)
    seen = held[:, None, :] & held[:, :, None]
    if c["causal"]:
        j = torch.arange(N, device=s.device)
        seen = seen & (j[None, :] <= j[:, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + m)[..., 0].reshape(n, c["Hq"], N).transpose(1, 2)[held].t()
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total)).reshape(n, Hkv, G * N, N)
    o = torch.matmul(p, v)

    def packed(x, H):
        return x.reshape(n, H, N, d).transpose(1, 2)[held].to(st["q"].dtype)

    out = {"o": packed(o, c["Hq"]), "lse": lse.contiguous()}
    if c["op"] == "train":
        g = padded(st["dout"], st["cu"], n, N)[0].reshape(n, Hkv, G * N, d)
        out["dv"] = packed(torch.matmul(p.transpose(-1, -2), g), Hkv)
        ds = torch.matmul(g, v.transpose(-1, -2)).sub_((g * o).sum(-1, keepdim=True)).mul_(p)
        out["dq"] = packed(torch.matmul(ds, k).mul_(scale), c["Hq"])
        out["dk"] = packed(torch.matmul(ds.transpose(-1, -2), q).mul_(scale), Hkv)
    return out


def plain_paged(st):
    c = st["case"]
    B, Hq, Nq, d = st["q"].shape
    Hkv, G = c["Hkv"], Hq // c["Hkv"]
    at = st["table"].clamp(min=0).long()
    N = at.shape[1] * c["page"]
    k, v = (x[at].transpose(1, 2).reshape(B, Hkv, N, d).float() for x in (st["k"], st["v"]))
    s = torch.matmul(st["q"].float().reshape(B, Hkv, G * Nq, d), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    L = st["lens"].long()[:, None, None]
    last = L - 1
    if c["causal"]:
        last = torch.minimum(last, L - Nq + torch.arange(Nq, device=s.device)[None, :, None])
    seen = (torch.arange(N, device=s.device)[None, None, :] <= last).expand(B, Nq, N)
    s = s.reshape(B, Hkv, G, Nq, N).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + m)[..., 0].reshape(B, Hq, Nq)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p.reshape(B, Hkv, G * Nq, N), v).reshape(B, Hq, Nq, d)
    return {"o": o.to(st["q"].dtype), "lse": lse}


def plain_append(st):
    c = st["case"]
    t = torch.arange(st["k_new"].shape[0], device=st["cu"].device, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:], t, right=True)
    pos = (st["lens"][b] + t - st["cu"][b]).long()
    at = st["table"][b, pos // c["page"]].long()
    st["k"][at, :, pos % c["page"]] = st["k_new"]
    st["v"][at, :, pos % c["page"]] = st["v_new"]
    return {"k": st["k"], "v": st["v"]}


def free_pages(refs):
    """The free pages' numbers, ascending, then the others."""
    return torch.sort((refs != 0).to(torch.int32), stable=True).indices.to(torch.int32)


def plain_free(table, lens, refs, keep, page):
    kept = torch.minimum(keep, lens)
    drop = (table >= 0) & (torch.arange(table.shape[1], device=table.device)[None] >= ((kept + page - 1) // page)[:, None])
    gone = torch.zeros_like(refs).scatter_add_(0, table.clamp(min=0).reshape(-1).long(), drop.to(torch.int32).reshape(-1))
    return torch.where(drop, torch.full_like(table, -1), table), kept, refs - gone


def plain_fork(table, lens, refs, src, dst, page):
    M = table.shape[1]
    L = lens[src.long()]
    full, tail = L // page, L % page > 0
    order = free_pages(refs)
    fresh = order[(torch.cumsum(tail, 0) - 1).clamp(min=0)]
    i = torch.arange(M, device=table.device)[None]
    shared = i < full[:, None]
    row = torch.where(shared, table[src.long()], torch.full_like(table[:1], -1))
    row = torch.where((i == full[:, None]) & tail[:, None], fresh[:, None], row)
    old = torch.gather(table[src.long()], 1, full[:, None].long().clamp(max=M - 1))[:, 0]
    copies = torch.where(tail[:, None], torch.stack((old, fresh), 1), torch.full_like(old, -1)[:, None])
    refs = refs.scatter_add(0, row.clamp(min=0).reshape(-1).long(), (row >= 0).to(torch.int32).reshape(-1))
    return table.index_copy(0, dst.long(), row), lens.index_copy(0, dst.long(), L), refs, copies


def plain_reserve(table, lens, refs, new, page):
    have = (table >= 0).sum(1).to(torch.int32)
    need = ((lens + new + page - 1) // page - have).clamp(min=0)
    first = torch.cumsum(need, 0).to(torch.int32) - need
    i = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)[None] - have[:, None]
    fresh = (i >= 0) & (i < need[:, None])
    order = free_pages(refs)
    row = order[(first[:, None] + i).clamp(0, order.numel() - 1).long()]
    refs = refs.scatter_add(0, torch.where(fresh, row, torch.zeros_like(row)).reshape(-1).long(), fresh.to(torch.int32).reshape(-1))
    return torch.where(fresh, row, table), refs


def plain_copy(k, v, copies):
    pairs = copies[copies[:, 0] >= 0].long()
    k[pairs[:, 1]] = k[pairs[:, 0]]
    v[pairs[:, 1]] = v[pairs[:, 0]]


def plain_beams(st):
    page = st["case"]["page"]
    table, lens, refs = plain_free(st["table"], st["lens"], st["refs"], st["keep"], page)
    table, lens, refs, copies = plain_fork(table, lens, refs, st["src"], st["dst"], page)
    plain_copy(st["k"], st["v"], copies)
    table, refs = plain_reserve(table, lens, refs, st["new"], page)
    return {"table": table, "lens": lens, "refs": refs, "copies": copies, "k": st["k"], "v": st["v"]}


def plain_compact(st):
    table, refs = st["table"], st["refs"]
    P = refs.numel()
    j = torch.arange(P, device=refs.device)
    used = refs > 0
    U = used.sum()
    holes = torch.sort((used | (j >= U)).to(torch.int32), stable=True).indices
    movers = torch.sort((~used | (j < U)).to(torch.int32), stable=True).indices
    moves = (used & (j >= U)).sum()
    n = P // 2
    real = j[:n] < moves
    src, dst = (torch.where(real, x[:n], torch.full_like(x[:n], -1)) for x in (movers, holes))
    copies = torch.stack((src, dst), 1).to(torch.int32)
    to = j.clone()
    to[src[real]] = dst[real]
    out = torch.zeros_like(refs)
    out[to[used]] = refs[used]
    plain_copy(st["k"], st["v"], copies)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table)
    return {"table": table, "refs": out, "copies": copies, "used": U.to(torch.int32).reshape(1), "k": st["k"], "v": st["v"]}


# ------------------------------------------------------------------------- the package's kernels
def own_prompt(st):
    import exact_attention_50_gb300 as A
    c = st["case"]
    o, lse = A.fwd_varlen_gqa(st["q"], st["k"], st["v"], st["cu"], st["longest"], c["causal"])
    out = {"o": o, "lse": lse}
    if c["op"] == "train":
        out["dq"], out["dk"], out["dv"] = A.bwd_varlen_gqa(st["q"], st["k"], st["v"], o, lse, st["dout"], st["cu"], st["longest"], c["causal"])
    return out


def own_paged(st):
    import exact_attention_50_gb300 as A
    o, lse = A.fwd_kvpages(st["q"], st["k"], st["v"], st["table"], st["lens"], causal=st["case"]["causal"])
    return {"o": o, "lse": lse}


def own_append(st):
    import exact_attention_50_gb300 as A
    A.kvpages_append(st["k"], st["v"], st["table"], st["k_new"], st["v_new"], st["cu"], st["lens"])
    return {"k": st["k"], "v": st["v"]}


def own_beams(st):
    import exact_attention_50_gb300 as A
    page = st["case"]["page"]
    table, lens, refs = A.kvpages_free(st["table"], st["lens"], st["refs"], st["keep"], page)
    table, lens, refs, copies = A.kvpages_fork(table, lens, refs, st["src"], st["dst"], page)
    A.kvpages_copy(st["k"], st["v"], copies)
    table, refs = A.kvpages_reserve(table, lens, refs, st["new"], page)
    return {"table": table, "lens": lens, "refs": refs, "copies": copies, "k": st["k"], "v": st["v"]}


def own_compact(st):
    import exact_attention_50_gb300 as A
    table, refs, copies, used = A.kvpages_compact(st["table"], st["refs"])
    A.kvpages_copy(st["k"], st["v"], copies)
    return {"table": table, "refs": refs, "copies": copies, "used": used, "k": st["k"], "v": st["v"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": own_prompt, "train": own_prompt, "paged": own_paged, "append": own_append, "beams": own_beams, "compact": own_compact}[op](state)
    return {"prompt": plain_prompt, "train": plain_prompt, "paged": plain_paged, "append": plain_append, "beams": plain_beams, "compact": plain_compact}[op](state)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    es, d, Hkv = 4 if c["dtype"] == "f32" else 2, c["d"], c["Hkv"]
    if c["op"] in ("prompt", "train"):
        lens = uneven(c["n"], c["lo"], c["hi"])
        T, Hq = sum(lens), c["Hq"]
        pairs = sum(visible(L, L, c["causal"]) for L in lens) * Hq
        size = T * d * es
        if c["op"] == "prompt":
            return {"bytes": float(size * (2 * Hq + 2 * Hkv) + 4 * T * Hq), "flops": 4.0 * d * pairs}
        return {"bytes": float(size * (4 * Hq + 4 * Hkv) + 4 * T * Hq), "flops": 14.0 * d * pairs}
    lens, page = uneven(c["B"], c["lo"], c["hi"]), c["page"]
    if c["op"] == "paged":
        pairs = sum(visible(L, c["Nq"], c["causal"]) for L in lens) * c["Hq"]
        held = sum(lens) * Hkv * d * es * 2 + 4 * sum(ceil_div(L, page) for L in lens)
        return {"bytes": float(held + c["B"] * c["Hq"] * c["Nq"] * (2 * d * es + 4)), "flops": 4.0 * d * pairs}
    one = Hkv * page * d * es * 2  # a page of keys and one of values
    if c["op"] == "append":
        T = sum(uneven(c["B"], c["new_lo"], c["new_hi"], 0.7548776662466927))
        return {"bytes": float(T * Hkv * d * es * 4 + 12 * T), "flops": 0.0}
    M = ceil_div(c["hi"], page) + 1
    if c["op"] == "beams":
        owned = sum(ceil_div(L, page) for L in lens[:c["B"] - c["forks"]])
        return {"bytes": float(2 * one * c["forks"] + 8 * c["B"] * M + 8 * owned), "flops": 0.0}
    owned = sum(ceil_div(L, page) for L in lens)
    pages = max(1, owned * 100 // (100 - c["spare"]))
    moved = owned * (pages - owned) / pages  # of pages in no order
    return {"bytes": float(2 * one * moved + 8 * c["B"] * M + 8 * pages), "flops": 0.0}


# ----------------------------------------------------------------------------------------- exact
def exact_head(q, k, first, causal):
    """Scores [G, Nq, L] of q [G, Nq, d] and k [L, d], query i seeing the keys up to first + i; and their log-sum-exp."""
    s = torch.einsum("gid,jd->gij", q, k) / math.sqrt(q.shape[-1])
    if causal:
        i, j = torch.arange(q.shape[1], device=q.device), torch.arange(k.shape[0], device=q.device)
        s = torch.where(j[None, :] > first + i[:, None], torch.full((), -math.inf, dtype=s.dtype, device=s.device), s)
    if k.shape[0] == 0:
        return s, torch.full(s.shape[:2], -math.inf, dtype=s.dtype, device=s.device)
    return s, torch.logsumexp(s, -1)


def weights_of(s, lse):
    return torch.where(s == -math.inf, torch.zeros_like(s), torch.exp(s - lse[..., None]))


def exact_prompt(c, st):
    G, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros((c["Hq"], o.shape[0]), dtype=torch.float64, device=o.device)
    dq = torch.zeros_like(o)
    dk, dv = (torch.zeros(st["k"].shape, dtype=torch.float64, device=o.device) for _ in range(2))
    at = 0
    for L in uneven(c["n"], c["lo"], c["hi"]):
        t = slice(at, at + L)
        at += L
        for h in range(c["Hkv"]):
            g = slice(h * G, (h + 1) * G)
            q, k, v = st["q"][t, g].double().transpose(0, 1), st["k"][t, h].double(), st["v"][t, h].double()
            s, e = exact_head(q, k, 0, c["causal"])
            p = weights_of(s, e)
            y = p @ v
            o[t, g], lse[g, t] = y.transpose(0, 1), e
            if c["op"] == "train":
                do = st["dout"][t, g].double().transpose(0, 1)
                dv[t, h] = torch.einsum("gij,gid->jd", p, do)
                ds = p * (do @ v.t() - (do * y).sum(-1, keepdim=True))
                dq[t, g] = (ds @ k * scale).transpose(0, 1)
                dk[t, h] = torch.einsum("gij,gid->jd", ds, q) * scale
    out = {"o": o, "lse": lse}
    if c["op"] == "train":
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def exact_paged(c, st):
    B, Hq, Nq, d = st["q"].shape
    G = Hq // c["Hkv"]
    q = st["q"].double().reshape(B, c["Hkv"], G, Nq, d)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
    for b, L in enumerate(uneven(c["B"], c["lo"], c["hi"])):
        at = st["table"][b, :ceil_div(L, c["page"])].long()
        for h in range(c["Hkv"]):
            k, v = (x[at, h].reshape(-1, d)[:L].double() for x in (st["k"], st["v"]))
            s, lse[b, h] = exact_head(q[b, h], k, L - Nq, c["causal"])
            o[b, h] = weights_of(s, lse[b, h]) @ v
    return {"o": o.reshape(B, Hq, Nq, d), "lse": lse.reshape(B, Hq, Nq)}


def exact_pages(c, st):
    """The tables by hand, sequence by sequence and page by page."""
    page = c["page"]
    table, refs, lens = ([list(r) for r in st["table"].tolist()], st["refs"].tolist(), st["lens"].tolist())
    k, v = st["k"], st["v"]
    if c["op"] == "beams":
        for b, keep in enumerate(st["keep"].tolist()):
            lens[b] = min(lens[b], keep)
            for i in range(ceil_div(lens[b], page), len(table[b])):
                if table[b][i] >= 0:
                    refs[table[b][i]] -= 1
                    table[b][i] = -1
        free = [i for i, r in enumerate(refs) if r == 0]
        copies = []
        for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
            full = lens[s] // page
            table[t] = table[s][:full] + [-1] * (len(table[s]) - full)
            for x in table[t][:full]:
                refs[x] += 1
            copies.append([-1, -1])
            if lens[s] % page:
                copies[-1] = [table[s][full], free.pop(0)]
                table[t][full] = copies[-1][1]
                refs[copies[-1][1]] = 1
            lens[t] = lens[s]
        free = [i for i, r in enumerate(refs) if r == 0]
        for b, n in enumerate(st["new"].tolist()):
            for i in range(sum(x >= 0 for x in table[b]), ceil_div(lens[b] + n, page)):
                table[b][i] = free.pop(0)
                refs[table[b][i]] = 1
        out = {"lens": torch.tensor(lens, dtype=torch.int32)}
    else:
        used = [i for i, r in enumerate(refs) if r > 0]
        U = len(used)
        copies = [[a, b] for a, b in zip([i for i in used if i >= U], [i for i in range(U) if refs[i] == 0])]
        to = dict((a, b) for a, b in copies)
        table = [[to.get(x, x) for x in r] for r in table]
        for a, b in copies:
            refs[b], refs[a] = refs[a], 0
        copies += [[-1, -1]] * (len(refs) // 2 - len(copies))
        out = {"used": torch.tensor([U], dtype=torch.int32)}
    pairs = torch.tensor([x for x in copies if x[0] >= 0], dtype=torch.int64).reshape(-1, 2).to(k.device)
    out["k"], out["v"] = k.double(), v.double()
    for x, y in ((out["k"], k), (out["v"], v)):
        x[pairs[:, 1]] = y[pairs[:, 0]].double()
    for name, x in (("table", table), ("refs", refs), ("copies", copies)):
        out[name] = torch.tensor(x, dtype=torch.int32)
    out["copies"] = out["copies"].reshape(-1, 2)
    return out


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] in ("prompt", "train"):
        return exact_prompt(c, st)
    if c["op"] == "paged":
        return exact_paged(c, st)
    if c["op"] in ("beams", "compact"):
        return exact_pages(c, st)
    out = {"k": st["k"].double(), "v": st["v"].double()}
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        pos = torch.arange(L, L + n, device=st["k"].device)
        at = st["table"][b].long()[pos // c["page"]]
        out["k"][at, :, pos % c["page"]] = st["k_new"][cu[b]:cu[b + 1]].double()
        out["v"][at, :, pos % c["page"]] = st["v_new"][cu[b]:cu[b + 1]].double()
    return out

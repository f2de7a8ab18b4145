"""The operators around a KV cache that is too long to keep whole, as measured cases.

Four operators, in the order in which a serving program uses them:

  weights   the attention weight that each cached key has received, added up over queries and
            the heads of its group: w_j += sum_i exp(scale q_i.k_j - LSE_i)
  evict     the cache cut down to the keys of the largest added-up weight and the last ones
  append8   new tokens written into a cache of 8 bits, with one scale per block of tokens and head
  attend8   attention of queries over such a cache

``run`` computes them in plain float32 torch operations, or, where ``own`` is set, calls the
package.  ``exact`` computes them once more from their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
C8 = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}  # the largest code of each 8-bit type
TINY = 2.0 ** -126                  # a scale below the smallest normal number counts as zero
HEADS = ((32, 8), (32, 32), (8, 8), (16, 2), (12, 4), (4, 1))


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---------------------------------------------------------------------------------------- cases
def attend8(name, B, Hq, Hkv, Nq, Nk, lo, d, block, dtype, cache, causal):
    return dict(name=name, op="attend8", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, lo=lo, d=d, block=block, dtype=dtype,
                cache=cache, causal=causal)


def append8(name, B, Hkv, Nn, Nk, lo, d, block, dtype, cache):
    return dict(name=name, op="append8", B=B, Hkv=Hkv, Nn=Nn, Nk=Nk, lo=lo, d=d, block=block, dtype=dtype, cache=cache)


def weights(name, B, Hq, Hkv, Nq, Nk, lo, d, dtype, causal):
    return dict(name=name, op="weights", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, lo=lo, d=d, dtype=dtype, causal=causal)


def evict(name, B, Hkv, Nk, lo, d, keep, recent, dtype):
    return dict(name=name, op="evict", B=B, Hkv=Hkv, Nk=Nk, lo=lo, d=d, keep=keep, recent=recent, dtype=dtype)


def listed():
    return [
        # one token of one conversation with a short history: the call's latency
        attend8("attend8 one short", 1, 32, 8, 1, 1001, 1001, 128, 64, "bf16", "i8", True),
        # the decode workload of the benchmark, its caches held in 8 bits
        attend8("attend8 decode", 8, 32, 8, 1, 32768, 16384, 128, 64, "bf16", "i8", True),
        # a draft of five tokens checked at once, every head with its own keys, 64 columns, small blocks
        attend8("attend8 draft e4m3", 4, 32, 32, 5, 4111, 300, 64, 32, "f16", "e4m3", True),
        # a chunk of a long prompt against the cache of what came before it
        attend8("attend8 chunk", 2, 32, 8, 2048, 16384, 16384, 128, 128, "bf16", "i8", True),
        # every decode step writes one token per sequence
        append8("append8 one token", 8, 8, 1, 32768, 16384, 128, 64, "bf16", "i8"),
        # whole prompts of different lengths go into an empty cache
        append8("append8 prompts", 4, 8, 16384, 16500, 0, 128, 64, "bf16", "e4m3"),
        # each decode step's weights over long caches
        weights("weights decode", 8, 32, 8, 1, 32768, 16384, 128, "bf16", True),
        # the last 48 queries of each prompt judge its keys; odd lengths
        weights("weights window", 4, 32, 8, 48, 8191, 4001, 128, "bf16", True),
        # all queries of the benchmark's training shape
        weights("weights prompt", 4, 32, 8, 2048, 2048, 2048, 128, "bf16", True),
        # one conversation, cut to a small cache
        evict("evict one", 1, 8, 2048, 2048, 128, 256, 64, "bf16"),
        # long caches of a batch, cut to an eighth
        evict("evict batch", 8, 8, 32768, 16384, 128, 3968, 128, "bf16"),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("attend8", "attend8", "append8", "weights", "weights", "evict"))
    Hq, Hkv = rng.choice(HEADS)
    B, d = rng.randint(1, 8), rng.choice((64, 128, 128, 80))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    cache, block = rng.choice(("i8", "e4m3")), rng.choice((16, 32, 64, 128))
    Nk = spread(rng, 16, 32768 if B * Hkv <= 64 else 8192)
    lo = rng.choice((Nk, Nk // 2, Nk // 7))
    if op in ("attend8", "weights"):
        Nq = rng.choice((1, 1, rng.randint(2, 8), spread(rng, 9, 1024)))
        if Nq > 8:  # scores of the plain form: no more than the largest listed case has
            Nk = min(Nk, 8192)
            lo = min(lo, Nk)
        causal = rng.choice((True, True, False))
        if op == "attend8":
            return {k: v for k, v in attend8("", B, Hq, Hkv, Nq, Nk, lo, d, block, dtype, cache, causal).items() if k != "name"}
        return {k: v for k, v in weights("", B, Hq, Hkv, Nq, Nk, lo, d, dtype, causal).items() if k != "name"}
    if op == "append8":
        Nn = min(rng.choice((1, rng.randint(2, 8), spread(rng, 9, 16384))), Nk)
        lo = min(lo, Nk - Nn)
        return {k: v for k, v in append8("", B, Hkv, Nn, Nk, lo, d, block, dtype, cache).items() if k != "name"}
    keep = spread(rng, 1, max(1, Nk // 2))
    return {k: v for k, v in evict("", B, Hkv, Nk, lo, d, keep, rng.randint(0, min(256, Nk)), dtype).items() if k != "name"}


def lengths(c):
    """Each sequence's cached tokens: over [lo, hi], in no order.  An append leaves room for Nn."""
    hi = c["Nk"] - c.get("Nn", 0)
    lo = min(c["lo"], hi)
    return [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(c["B"])]


def new_lengths(c):
    """The tokens that each sequence appends: one each, or prompts of Nn/2 to Nn."""
    n = c["Nn"]
    return [n - int(n / 2 * ((b * 0.6180339887498949) % 1.0)) for b in range(c["B"])]


def visible(L, Nq, causal):
    """(query, key) pairs of one head."""
    return sum(min(L, max(0, L - Nq + i + 1)) for i in range(Nq)) if causal else Nq * L


# --------------------------------------------------------------------------------------- inputs
def normal(gen, shape, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)


def keys(gen, shape, dtype, dev):
    """Keys or values as a projection gives them: some columns and some tokens far larger than others."""
    x = normal(gen, shape, dev)
    x *= torch.exp(0.5 * normal(gen, (shape[0], shape[1], 1, shape[3]), dev) - 0.25)
    x *= torch.exp(0.3 * normal(gen, (shape[0], shape[1], shape[2], 1), dev))
    return x.to(dtype)


def in_blocks(x, block, fill=0.0):
    """[..., N, d] or [..., N] padded to whole blocks along the tokens: [..., n, block(, d)]."""
    n = x.shape[2]
    short = -n % block
    if short:
        tail = list(x.shape)
        tail[2] = short
        x = torch.cat((x, torch.full(tail, fill, dtype=x.dtype, device=x.device)), 2)
    return x.reshape(x.shape[:2] + (x.shape[2] // block, block) + x.shape[3:])


def coded(x, cache):
    """Float32 values in steps of their scale, rounded to the codes of the 8-bit type."""
    if cache == "i8":
        return torch.round(x).clamp(-127.0, 127.0).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def scale_of(amax, cache):
    s = amax * (1.0 / TOP[cache])
    return torch.where(s < TINY, torch.zeros_like(s), s)


def inverse(s):
    return torch.where(s == 0, torch.zeros_like(s), torch.reciprocal(s))


def quantised(x, block, cache):
    """A cache of 8 bits as it stands after its tokens were written block by block."""
    n = x.shape[2]
    xb = in_blocks(x.float(), block)
    s = scale_of(xb.abs().amax((-1, -2)), cache)
    q = coded(xb * inverse(s)[..., None, None], cache)
    return q.reshape(q.shape[:2] + (-1, q.shape[-1]))[:, :, :n].contiguous(), s.contiguous()


def prepare(case, seed):
    c, dev = case, device()
    gen = torch.Generator(dev).manual_seed(int(seed) * 1000003 + 17)
    B, Hkv, Nk, d, dt = c["B"], c["Hkv"], c["Nk"], c["d"], DT[c["dtype"]]
    st = {"case": c, "lens": torch.tensor(lengths(c), dtype=torch.int32, device=dev)}
    if c["op"] == "append8":
        st["k8"], st["ks"] = quantised(keys(gen, (B, Hkv, Nk, d), dt, dev), c["block"], c["cache"])
        st["v8"], st["vs"] = quantised(keys(gen, (B, Hkv, Nk, d), dt, dev), c["block"], c["cache"])
        st["k"], st["v"] = (keys(gen, (B, Hkv, c["Nn"], d), dt, dev) for _ in range(2))
        st["new"] = torch.tensor(new_lengths(c), dtype=torch.int32, device=dev)
    elif c["op"] == "attend8":
        st["q"] = normal(gen, (B, c["Hq"], c["Nq"], d), dev).to(dt)
        st["k8"], st["ks"] = quantised(keys(gen, (B, Hkv, Nk, d), dt, dev), c["block"], c["cache"])
        st["v8"], st["vs"] = quantised(keys(gen, (B, Hkv, Nk, d), dt, dev), c["block"], c["cache"])
    elif c["op"] == "weights":
        st["q"] = normal(gen, (B, c["Hq"], c["Nq"], d), dev).to(dt)
        st["k"] = keys(gen, (B, Hkv, Nk, d), dt, dev)
        st["w"] = normal(gen, (B, Hkv, Nk), dev).exp()  # what earlier queries left
        st["lse"] = plain_scores(st["q"], st["k"].float(), st["lens"], c["causal"])[1]
    else:
        st["k"], st["v"] = (keys(gen, (B, Hkv, Nk, d), dt, dev) for _ in range(2))
        w = torch.exp(1.5 * normal(gen, (B, Hkv, Nk), dev))
        st["w"] = torch.where(w < 1.0, torch.floor(w * 64.0) / 64.0, w)  # light keys have equal weights
        cap = c["keep"] + c["recent"] + 64  # room for the tokens that follow
        st["k_out"], st["v_out"] = (torch.zeros((B, Hkv, cap, d), dtype=dt, device=dev) for _ in range(2))
    return st


# ---------------------------------------------------------------------------------- plain forms
def plain_scores(q, k, lens, causal):
    """Scaled scores of the group's rows in float32, -inf where a query does not see a key, and
    each row's log-sum-exp as [B, Hq, Nq]."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    s = torch.matmul(q.float().reshape(B, Hkv, -1, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    j = torch.arange(Nk, device=q.device)
    L = lens.long()[:, None, None]
    last = L - 1
    if causal:
        last = torch.minimum(last, L - Nq + torch.arange(Nq, device=q.device)[None, :, None])
    seen = (j[None, None, :] <= last).expand(B, Nq, Nk)
    s = s.reshape(B, Hkv, Hq // Hkv, Nq, Nk).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    lse = torch.log(torch.exp(s - m).sum(-1)) + m[..., 0]
    return s.reshape(B, Hkv, -1, Nk), lse.reshape(B, Hq, Nq)


def plain_attend8(st):
    c, block = st["case"], st["case"]["block"]
    k, v = (x.float() * s.repeat_interleave(block, 2)[:, :, :x.shape[2], None] for x, s in ((st["k8"], st["ks"]), (st["v8"], st["vs"])))
    s, lse = plain_scores(st["q"], k, st["lens"], c["causal"])
    rows = lse.reshape(s.shape[:3])[..., None]
    p = torch.exp(s - torch.where(rows == -math.inf, torch.zeros_like(rows), rows))
    seen = torch.arange(c["Nk"], device=v.device)[None] < st["lens"][:, None]
    o = torch.matmul(p, v * seen[:, None, :, None])
    return {"o": o.reshape(st["q"].shape).to(st["q"].dtype), "lse": lse}


def plain_append8_one(x8, scales, x_new, lens, new, block, cache):
    """In place, over a window of tokens that holds each sequence's touched blocks."""
    B, Hkv, Nk, d = x8.shape
    Nn, blocks = x_new.shape[2], scales.shape[2]
    L, n = lens.long()[:, None], new.long()[:, None]
    W = min(Nk, -(-(Nn + block - 1) // block) * block)
    tok = torch.clamp(L // block * block, max=Nk - W) + torch.arange(W, device=x8.device)
    wb = min(blocks, (W - 1) // block + 2)
    blk = torch.clamp(tok[:, :1] // block, max=blocks - wb) + torch.arange(wb, device=x8.device)
    at = (tok // block - blk[:, :1])[:, None].expand(B, Hkv, W)
    rows = tok[:, None, :, None].expand(B, Hkv, W, d)
    is_old, is_new = tok < L, (tok >= L) & (tok < L + n)
    take = (tok - L).clamp(0, Nn - 1)
    x = torch.gather(x_new, 2, take[:, None, :, None].expand(B, Hkv, W, d)).float()
    largest = torch.where(is_new[:, None], x.abs().amax(-1), torch.zeros((), device=x.device))
    amax = torch.zeros((B, Hkv, wb), device=x.device).scatter_reduce(2, at, largest, "amax")
    old = (blk * block < L)[:, None]
    touched = ((blk * block < L + n) & ((blk + 1) * block > L) & (n > 0))[:, None]
    which = blk[:, None].expand(B, Hkv, wb)
    s_old = torch.gather(scales, 2, which)
    s = scale_of(amax, cache)
    s = torch.where(old & (s_old > s), s_old, s)
    s = torch.where(touched, s, s_old)
    grown = touched & old & (s > s_old)
    inv = inverse(s)
    f = torch.where(grown, s_old * inv, torch.ones_like(s))

    def per_token(y):
        return torch.gather(y, 2, at)[..., None]

    held = torch.gather(x8.view(torch.uint8), 2, rows)
    q = torch.where(is_new[:, None, :, None], coded(x * per_token(inv), cache).view(torch.uint8), held)
    moved = coded(held.view(x8.dtype).float() * per_token(f), cache).view(torch.uint8)
    q = torch.where(is_old[:, None, :, None] & per_token(grown), moved, q)
    x8.view(torch.uint8).scatter_(2, rows, q)
    scales.scatter_(2, which, s)


def plain_append8(st):
    c = st["case"]
    plain_append8_one(st["k8"], st["ks"], st["k"], st["lens"], st["new"], c["block"], c["cache"])
    plain_append8_one(st["v8"], st["vs"], st["v"], st["lens"], st["new"], c["block"], c["cache"])
    return {"k8": st["k8"], "v8": st["v8"], "ks": st["ks"], "vs": st["vs"]}


def plain_weights(st):
    s, _ = plain_scores(st["q"], st["k"].float(), st["lens"], st["case"]["causal"])
    rows = st["lse"].reshape(s.shape[:3])[..., None]
    p = torch.exp(s - torch.where(rows == -math.inf, torch.zeros_like(rows), rows))
    return {"w": st["w"] + p.sum(2)}


def plain_evict(st):
    c = st["case"]
    B, Hkv, Nk, M = c["B"], c["Hkv"], c["Nk"], c["keep"] + c["recent"]
    j = torch.arange(Nk, device=st["w"].device)[None]
    L = st["lens"].long()[:, None]
    w = torch.where((j >= L - c["recent"])[:, None], torch.full_like(st["w"], math.inf), st["w"])
    w = torch.where((j >= L)[:, None], torch.full_like(w, -math.inf), w)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :M]
    left = torch.minimum(L, torch.full_like(L, M))
    n = order.shape[2]
    slot = torch.arange(n, device=w.device)[None]
    order = torch.where((slot < left)[:, None], order, torch.full_like(order, Nk)).sort(2).values
    at = order.clamp(max=Nk - 1)
    held = (order < Nk)
    index = torch.full((B, Hkv, M), -1, dtype=torch.int32, device=w.device)
    index[:, :, :n] = torch.where(held, order, torch.full_like(order, -1)).to(torch.int32)
    out = {"index": index, "lens": left[:, 0].to(torch.int32)}
    out["w"] = torch.zeros((B, Hkv, st["k_out"].shape[2]), device=w.device)
    out["w"][:, :, :n] = torch.where(held, torch.gather(st["w"], 2, at), torch.zeros((), device=w.device))
    for name, x, y in (("k", st["k"], st["k_out"]), ("v", st["v"], st["v_out"])):
        rows = torch.gather(x, 2, at[..., None].expand(B, Hkv, n, c["d"]))
        out[name] = y.clone()
        out[name][:, :, :n] = torch.where(held[..., None], rows, y[:, :, :n])
    return out


# ------------------------------------------------------------------------- the package's kernels
def own_attend8(st):
    import exact_attention_50_gb300 as A
    c = st["case"]
    o, lse = A.fwd_kvcache8(st["q"], st["k8"], st["v8"], st["ks"], st["vs"], st["lens"], causal=c["causal"], block=c["block"])
    return {"o": o, "lse": lse}


def own_append8(st):
    import exact_attention_50_gb300 as A
    A.kvcache8_append(st["k8"], st["v8"], st["ks"], st["vs"], st["k"], st["v"], st["lens"], st["new"], block=st["case"]["block"])
    return {"k8": st["k8"], "v8": st["v8"], "ks": st["ks"], "vs": st["vs"]}


def own_weights(st):
    import exact_attention_50_gb300 as A
    return {"w": A.kvcache_weights(st["q"], st["k"], st["lse"], st["lens"], causal=st["case"]["causal"], weights=st["w"])}


def own_evict(st):
    import exact_attention_50_gb300 as A
    c = st["case"]
    k, v, w, index, lens = A.kvcache_evict(st["k"], st["v"], st["w"], c["keep"], c["recent"], st["lens"], out=(st["k_out"], st["v_out"]))
    return {"k": k, "v": v, "w": w, "index": index, "lens": lens}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend8": own_attend8, "append8": own_append8, "weights": own_weights, "evict": own_evict}[op](state)
    return {"attend8": plain_attend8, "append8": plain_append8, "weights": plain_weights, "evict": plain_evict}[op](state)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c, lens = case, lengths(case)
    es = 4 if c["dtype"] == "f32" else 2
    H, d = c["Hkv"], c["d"]
    if c["op"] == "append8":
        n = sum(new_lengths(c)) * H
        return {"bytes": 2.0 * n * d * (es + 1), "flops": 2.0 * n * d * 2}
    if c["op"] == "evict":
        left = sum(min(L, c["keep"] + c["recent"]) for L in lens) * H
        return {"bytes": float(sum(lens) * H * 4 + left * (2 * 2 * d * es + 8)), "flops": float(sum(lens) * H)}
    rows = c["B"] * c["Hq"] * c["Nq"]
    pairs = sum(visible(L, c["Nq"], c["causal"]) for L in lens) * c["Hq"]
    if c["op"] == "weights":
        return {"bytes": float(rows * (d * es + 4) + sum(lens) * H * d * es + 8 * c["B"] * H * c["Nk"]), "flops": 2.0 * d * pairs}
    blocks = sum(-(-L // c["block"]) for L in lens) * H
    return {"bytes": float(rows * (2 * d * es + 4) + 2 * sum(lens) * H * d + 8 * blocks), "flops": 4.0 * d * pairs}


# ----------------------------------------------------------------------------------------- exact
def exact_head(q, k, L, causal):
    """One (sequence, key head): scores [G, Nq, L] and log-sum-exp [G, Nq] of q [G, Nq, d] and k [L, d]."""
    G, Nq, d = q.shape
    s = torch.einsum("gid,jd->gij", q.double(), k.double()) / math.sqrt(d)
    if causal:
        i, j = torch.arange(Nq, device=q.device), torch.arange(L, device=q.device)
        s = torch.where(j[None, :] - i[:, None] > L - Nq, torch.full((), -math.inf, dtype=s.dtype, device=s.device), s)
    if L == 0:
        return s, torch.full((G, Nq), -math.inf, dtype=torch.float64, device=q.device)
    return s, torch.logsumexp(s, -1)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    lens = lengths(c)
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] in ("attend8", "weights"):
        G = c["Hq"] // Hkv
        q = st["q"].reshape(B, Hkv, G, c["Nq"], c["d"])
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device)
        if c["op"] == "weights":
            w = st["w"].double()
            given = st["lse"].double().reshape(lse.shape)
        for b, L in enumerate(lens):
            for h in range(Hkv):
                if c["op"] == "weights":
                    s, _ = exact_head(q[b, h], st["k"][b, h, :L], L, c["causal"])
                    p = torch.exp(s - given[b, h][..., None])
                    w[b, h, :L] += torch.where(s == -math.inf, torch.zeros_like(p), p).sum((0, 1))
                    continue
                at = torch.arange(L, device=q.device) // c["block"]
                k = st["k8"][b, h, :L].float().double() * st["ks"][b, h].double()[at][:, None]
                v = st["v8"][b, h, :L].float().double() * st["vs"][b, h].double()[at][:, None]
                s, lse[b, h] = exact_head(q[b, h], k, L, c["causal"])
                p = torch.exp(s - lse[b, h][..., None])
                o[b, h] = torch.where(s == -math.inf, torch.zeros_like(p), p) @ v
        if c["op"] == "weights":
            return {"w": w}
        return {"o": o.reshape(st["q"].shape), "lse": lse.reshape(B, c["Hq"], c["Nq"])}
    if c["op"] == "append8":
        out, top = {}, TOP[c["cache"]]
        for name, x8, s, x in (("k", st["k8"], st["ks"], st["k"]), ("v", st["v8"], st["vs"], st["v"])):
            s64, held = s.double().clone(), x8.float().double()
            for b, (L, n) in enumerate(zip(lens, new_lengths(c))):
                first = L // c["block"] * c["block"]
                for a in range(first, L + n, c["block"]):
                    e, i = min(a + c["block"], L + n), a // c["block"]
                    fresh = x[b, :, max(a, L) - L:e - L].double()
                    step = fresh.abs().amax((1, 2)) / top
                    if a < L:
                        step = torch.maximum(step, s64[b, :, i])
                        back = s64[b, :, i] / step
                        held[b, :, a:L] = torch.where((back < 1)[:, None, None], rounded(held[b, :, a:L] * back[:, None, None], c["cache"]), held[b, :, a:L])
                    held[b, :, max(a, L):e] = rounded(fresh / step.clamp(min=TINY)[:, None, None], c["cache"])
                    s64[b, :, i] = step
            out[name + "8"], out[name + "s"] = (held if c["cache"] == "e4m3" else held.to(torch.int8)), s64
        return out
    w = st["w"].cpu().numpy()
    M, cap = c["keep"] + c["recent"], st["k_out"].shape[2]
    out = {"k": st["k_out"].double(), "v": st["v_out"].double(), "w": torch.zeros(B, Hkv, cap, dtype=torch.float64),
           "index": torch.full((B, Hkv, M), -1, dtype=torch.int32), "lens": torch.tensor([min(L, M) for L in lens], dtype=torch.int32)}
    for b, L in enumerate(lens):
        for h in range(Hkv):
            old = max(0, L - c["recent"])
            best = np.lexsort((np.arange(old), -w[b, h, :old]))[:M - (L - old)]
            kept = np.sort(np.concatenate((best, np.arange(old, L))))
            at = torch.from_numpy(kept)
            out["index"][b, h, :len(kept)] = at.int()
            out["w"][b, h, :len(kept)] = torch.from_numpy(w[b, h, kept]).double()
            out["k"][b, h, :len(kept)] = st["k"][b, h, at.to(st["k"].device)].double()
            out["v"][b, h, :len(kept)] = st["v"][b, h, at.to(st["v"].device)].double()
    return out


def rounded(x, cache):
    """To the nearest code of the 8-bit type, ties to even: whole numbers, or three binary places
    behind the leading one down to steps of 2^-9."""
    if cache == "i8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)

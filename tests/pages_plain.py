"""Plain implementations for the tests of packed attention with grouped heads and of caches in pages: attention and its
gradients in 64 bits with the error bounds that the kernels' roundings allow, and the books sequence by sequence."""
import math

import torch

# half a step of rounding, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def sum_error(n):
    """A sum of n products in fp32: an MMA adds 16 at a time, the parts of tiles and ranges follow; a fp32 loop takes one
    after the other.  Steps of 2^-23 (the tensor cores may cut off instead of rounding), half of them one way."""
    return (n / 8 + 64) * 2.0 ** -23


def attend(q, k, v, first, causal, scale=None):
    """One kv head: q [G, Nq, d], k and v [L, d] in 64 bits, query i seeing keys up to first + i.  Returns o, lse, p, and the
    sum of |q k| behind each score."""
    G, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    s = torch.einsum("gid,jd->gij", q, k) * scale
    size = torch.einsum("gid,jd->gij", q.abs(), k.abs()) * scale
    if causal:
        i, j = torch.arange(Nq, device=q.device), torch.arange(k.shape[0], device=q.device)
        s = s.masked_fill(j[None, :] > first + i[:, None], -math.inf)
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((G, Nq), -math.inf, dtype=q.dtype, device=q.device), s, size
    lse = torch.logsumexp(s, -1)
    p = torch.where(s == -math.inf, torch.zeros_like(s), torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]))
    return p @ v, lse, p, size


def attend_bounds(v, p, size, o, d, rho, half):
    """What o and lse may be off: rho is the rounding of P, half that of the output."""
    n = p.shape[-1]
    if n == 0:
        return torch.zeros_like(o), torch.zeros(o.shape[:2], dtype=o.dtype, device=o.device)
    e_s = size * sum_error(d)                        # of a score, and so of its exponential, relative
    e_p = e_s + 2.0 ** -20                           # ex2.approx, the row's maximum and scale: a few 2^-22
    each = (p * (rho + 2 * e_p)) @ v.abs()           # numerator, and the sum that divides it
    shared = (p * e_p).sum(-1, keepdim=True) * (p @ v.abs())
    tiny = n * 2.0 ** -24 * v.abs().amax(0)          # fp16 weights below 2^-14 of the largest
    bound = each + shared + sum_error(n) * 2 * (p @ v.abs()) + tiny + half * o.abs() * 1.01
    return bound, (p * e_p).sum(-1) + sum_error(n) + 2.0 ** -20


def spread(x, dim):
    """The sum over `dim` of independent errors of up to |x| each: no more than their sum, and beyond six times the root of the
    sum of squares (a rounding's standard deviation is 0.58 of its largest value, so that is ten deviations) not to be met."""
    return torch.minimum(x.abs().sum(dim), 6 * x.square().sum(dim).sqrt())


def grads(q, k, v, dout, first, causal, half_in, half_out, rho, scale=None, few=0):
    """One kv head in 64 bits: (dq, dk, dv) and their bounds.  The kernels take D = dO . O with O as the forward gave it, its P
    and itself rounded (half_in each; the first `few` queries: D summed over the keys), hold P and dS with an error of rho, relative, and round the results (half_out)."""
    G, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, _, p, size = attend(q, k, v, first, causal, scale)
    n, rows = p.shape[-1], sum_error(G * Nq)
    e_p = 2 * size * sum_error(d) + sum_error(n) + 2.0 ** -19  # p from the forward's LSE: both errors
    dv = torch.einsum("gij,gid->jd", p, dout)
    dp = dout @ v.t()
    ds = p * (dp - (dout * o).sum(-1, keepdim=True))
    dq, dk = ds @ k * scale, torch.einsum("gij,gid->jd", ds, q) * scale
    e_dp = (dout.abs() @ v.abs().t()) * sum_error(d)
    # D's error, one number for a row: the roundings of O's columns, of the weights behind them, and the sums
    other = (p * 2 * e_p) @ v.abs() + 2 * sum_error(n) * (p @ v.abs()) + n * 2.0 ** -24 * v.abs().amax(0) + sum_error(d) * o.abs()
    rounded = spread(half_in * dout * o, -1) + spread(half_in * p * dp, -1)
    if few:  # these rows' D is a sum over their keys
        rounded[:, :few] = ((p * e_dp + sum_error(n) * (p * dp).abs()).sum(-1))[:, :few]
    e_d = (rounded + (dout.abs() * other).sum(-1))[..., None]
    e_ds = ds.abs() * (e_p + rho) + p * e_dp  # per (query, key), beside D's
    tiny = 2.0 ** -24 * (1 + ds.abs().amax())  # fp16 parts of dS below its normal numbers
    b_dv = torch.einsum("gij,gid->jd", p * (e_p + rho + rows), dout.abs()) + half_out * dv.abs() * 1.01 + G * Nq * 2.0 ** -24 * dout.abs().amax((0, 1))
    b_dq = ((e_ds + sum_error(n) * ds.abs()) @ k.abs() + e_d * (p @ k).abs()) * scale + half_out * dq.abs() * 1.01 + n * tiny * scale * k.abs().amax()
    pe = p * e_d
    by_d = torch.minimum(torch.einsum("gij,gid->jd", pe, q.abs()), 6 * torch.einsum("gij,gid->jd", pe.square(), q.square()).sqrt())
    b_dk = (torch.einsum("gij,gid->jd", e_ds + rows * ds.abs(), q.abs()) + by_d) * scale + half_out * dk.abs() * 1.01 + G * Nq * tiny * scale * q.abs().amax()
    return (dq, dk, dv), (b_dq, b_dk, b_dv)


# ------------------------------------------------------------------------------------------ books
def pages_of(tokens, page):
    return -(-tokens // page)


def free(table, lens, refs, keep, page):
    table, lens, refs, bad = [list(r) for r in table], list(lens), list(refs), False
    for b, row in enumerate(table):
        if lens[b] < 0 or keep[b] < 0:
            bad = True
            continue
        lens[b] = min(lens[b], keep[b])
        for i in range(pages_of(lens[b], page), len(row)):
            if row[i] >= 0:
                if row[i] < len(refs):
                    refs[row[i]] -= 1
                else:
                    bad = True
                row[i] = -1
    return table, lens, refs, bad


def fork(table, lens, refs, src, dst, page):
    old, old_lens = [list(r) for r in table], list(lens)
    table, lens, out, bad = [list(r) for r in table], list(lens), list(refs), False
    spare = [i for i, r in enumerate(refs) if r <= 0]
    copies, seen, M = [], set(), len(table[0]) if table else 0
    for s, t in zip(src, dst):
        copies.append([-1, -1])
        first = t not in seen
        seen.add(t)
        ok = 0 <= s < len(old) and 0 <= t < len(old) and first
        if ok:
            L = old_lens[s]
            ok = old_lens[t] == 0 and (M == 0 or old[t][0] < 0) and L >= 0 and pages_of(L, page) <= M
            ok = ok and (L == 0 or 0 <= old[s][(L - 1) // page] < len(refs))
        if ok and L % page:
            ok = bool(spare)
            fresh = spare.pop(0) if spare else None
        if not ok:
            bad = True
            continue
        full = L // page
        table[t] = old[s][:full] + [-1] * (M - full)
        for x in table[t][:full]:
            out[x] += 1
        if L % page:
            copies[-1] = [old[s][full], fresh]
            table[t][full] = fresh
            out[fresh] = 1
        lens[t] = L
    return table, lens, out, copies, bad


def reserve(table, lens, refs, new, page):
    table, out, bad = [list(r) for r in table], list(refs), False
    spare = [i for i, r in enumerate(refs) if r <= 0]
    taken = 0
    for b, row in enumerate(table):
        have = next((i for i, x in enumerate(row) if x < 0), len(row))
        want = pages_of(lens[b] + new[b], page)
        if lens[b] < 0 or new[b] < 0 or want > len(row):
            bad = True
            continue
        need = max(0, want - have)
        if need and taken + need > len(spare):
            bad = True
            taken += need
            continue
        for i in range(need):
            row[have + i] = spare[taken + i]
            out[spare[taken + i]] = 1
        taken += need
    return table, out, bad


def compact(table, refs):
    used = [i for i, r in enumerate(refs) if r > 0]
    U = len(used)
    moves = list(zip([i for i in used if i >= U], [i for i in range(U) if refs[i] <= 0]))
    to, bad = dict(moves), False
    table = [list(r) for r in table]
    for row in table:
        for i, x in enumerate(row):
            if x in to:
                row[i] = to[x]
            elif x >= U or (x >= 0 and refs[x] <= 0):
                bad = True
    out = [r if r > 0 else 0 for r in refs[:U]] + [0] * (len(refs) - U)
    for a, b in moves:
        out[b] = refs[a]
    return table, out, [list(m) for m in moves] + [[-1, -1]] * (len(refs) // 2 - len(moves)), U, bad

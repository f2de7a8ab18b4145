"""Plain implementations of the cache operators for the tests: definitions in 64 bits (or, where
codes are compared bit by bit, single IEEE float32 operations in numpy), with no tiling, and the
error bounds that the kernels' roundings allow."""
import math

import numpy as np
import torch

TOP = {"i8": 127.0, "e4m3": 448.0}
C8 = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
# half a step of rounding, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


# ------------------------------------------------------------------ codes, in float32 like the definition
def round_code(x, cache):
    """float32 array -> the values of the nearest codes (ties to even), within the type's range."""
    x = np.asarray(x, np.float32)
    if cache == "i8":
        return np.clip(np.rint(x), -127, 127).astype(np.float32)
    y = x.astype(np.float64)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.clip(np.rint(y / step) * step, -448, 448).astype(np.float32)


def block_scale(x, cache):
    """max |x| times the float32 reciprocal of the largest code; below the smallest normal number: 0."""
    amax = np.max(np.abs(x), initial=np.float32(0))
    s = np.float32(amax) * np.float32(1.0 / TOP[cache])
    return np.float32(0) if s < np.float32(2.0 ** -126) else np.float32(s)


def append(codes, scale, x_new, L, n, block, cache):
    """One head: codes [Nk, d] (values), scale [blocks]; x_new [Nn, d]; all float32.  In place."""
    for a in range(L // block * block, L + n, block):
        lo, hi, i = max(a, L), min(a + block, L + n), a // block
        if lo >= hi:
            continue
        new = x_new[lo - L:hi - L].astype(np.float32)
        s = block_scale(new, cache)
        old = np.float32(scale[i])
        if lo > a and old > s:
            s = old
        inv = np.float32(0) if s == 0 else np.float32(1) / s
        codes[lo:hi] = round_code(new * inv, cache)
        if lo > a and s > old:
            codes[a:lo] = round_code(codes[a:lo] * (old * inv), cache)
        scale[i] = s


def quantise(x, block, cache):
    """A whole cache [B,H,N,d] of floats -> (codes tensor, scales) on x's device."""
    x = x.float()
    B, H, N, d = x.shape
    nb = -(-N // block)
    xp = torch.zeros(B, H, nb * block, d, device=x.device)
    xp[:, :, :N] = x
    xb = xp.reshape(B, H, nb, block, d)
    s = xb.abs().amax((-1, -2)) / TOP[cache]
    q = xb / torch.where(s == 0, torch.ones_like(s), s)[..., None, None]
    q = torch.round(q).clamp(-127, 127).to(torch.int8) if cache == "i8" else q.clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(B, H, -1, d)[:, :, :N].contiguous(), s.contiguous()


def dequantise(x8, scale, block):
    N = x8.shape[2]
    return x8.float().double() * scale.double().repeat_interleave(block, 2)[:, :, :N, None]


# ----------------------------------------------------------------------------------- attention
def seen_keys(Nq, Nk, L, causal, device):
    """[Nq, Nk] bool: query i sees key j < L and, causal, j <= L - Nq + i."""
    j = torch.arange(Nk, device=device)[None]
    i = torch.arange(Nq, device=device)[:, None]
    m = (j < L).expand(Nq, Nk)
    return m & (j <= L - Nq + i) if causal else m


def attend(q, k, v, lens, causal, scale=None):
    """q [B,Hq,Nq,d]; k, v [B,Hkv,Nk,d] float64.  Returns o, lse, A = P |V| (what an error
    of the weights is multiplied by), and E [B,Hq,Nq], a bound of a float32 sum's error in a row's
    scores: d + 16 roundings of 2^-24 of the largest sum of |q k|.  Keys that a batch does not see are
    left out before anything is computed, so they may hold anything."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, A = (torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=q.device)
    E = torch.zeros_like(lse)
    for b in range(B):
        L = Nk if lens is None else int(lens[b])
        if L == 0:
            continue
        m = seen_keys(Nq, L, L, causal, q.device)
        for h in range(Hq):
            kk, vv, qq = k[b, h // G, :L], v[b, h // G, :L], q[b, h].double()
            s = (qq @ kk.T * scale).masked_fill(~m, -math.inf)
            row = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(row == -math.inf, torch.zeros_like(row), row)[:, None])
            o[b, h], A[b, h], lse[b, h] = p @ vv, p @ vv.abs(), row
            E[b, h] = (qq.abs() @ kk.abs().T * scale).amax(-1) * (d + 16) * 2.0 ** -24
    return o, lse, A, E


def weights(q, k, lse, lens, causal, w_in, scale=None):
    """Returns the added-up weights and a bound of their error: a score's error E as in attend, the
    exponential's 2^-18, and the sum's roundings."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, Hkv, Nk, dtype=torch.float64, device=q.device) if w_in is None else w_in.double().clone()
    err = out.abs() * 2.0 ** -23
    for b in range(B):
        L = Nk if lens is None else int(lens[b])
        if L == 0:
            continue
        m = seen_keys(Nq, L, L, causal, q.device)
        for h in range(Hq):
            kk, qq = k[b, h // G, :L].double(), q[b, h].double()
            s = qq @ kk.T * scale
            p = torch.exp(s - lse[b, h].double()[:, None]).masked_fill(~m, 0.0)
            E = (qq.abs() @ kk.abs().T * scale) * (d + 16) * 2.0 ** -24 + lse[b, h].double().abs().nan_to_num(0, 0, 0)[:, None] * 2.0 ** -22
            out[b, h // G, :L] += p.sum(0)
            # adding one by one: at most R roundings of the running sum
            err[b, h // G, :L] += (p * (2 * E + 2.0 ** -18)).sum(0)
    err += out.abs() * min(2.0 ** -10, (G * Nq + 4) * 2.0 ** -24)
    return out, err


def evict(k, v, w, L, keep, recent):
    """One head: the kept positions, in order."""
    if L <= keep + recent:
        return np.arange(L)
    old = np.asarray(w[:L - recent], np.float64)
    key = np.where(np.isnan(old), np.inf, old)
    # NaN above infinity: a second key
    best = np.lexsort((np.arange(len(old)), -key, ~np.isnan(old)))[:keep]
    return np.sort(np.concatenate((best, np.arange(L - recent, L))))


def attend8(q, k8, v8, ks, vs, block, lens, causal, scale=None):
    """Attention over an 8-bit cache in 64 bits, with the errors that it may have before its output is
    rounded.  Returns o, lse, a bound [B,Hq,Nq,d] of each element's error, one [B,Hq,Nq] of the length of
    a row's error vector where rounding errors of different keys are independent, and E of attend.

    The kernels round P vs of a key to fp16 (u = 2^-11 of it; a term below 2^-14 of the unit, 2^-25 of the
    unit), the unit at most the largest P vs among the keys that the row sees, and multiply by
    the codes exactly.  A score's error E enters numerator and denominator, the exponential's is
    2^-18.  For the length: (u + E)^2 per key in squares, and 2^-17 of sum P|V| for what the fp32 sums
    and the exponential may have in common."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k8.shape[1:3]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    new = lambda *s: torch.zeros(B, Hq, Nq, *s, dtype=torch.float64, device=q.device)
    o, bound, length, E, lse = new(d), new(d), new(), new(), new() - math.inf
    at = torch.arange(Nk, device=q.device) // block
    u = 2.0 ** -11
    for b in range(B):
        L = Nk if lens is None else int(lens[b])
        if L == 0:
            continue
        m = seen_keys(Nq, L, L, causal, q.device)
        for h in range(Hq):
            g = h // G
            sv, code = vs[b, g].double()[at[:L]], v8[b, g, :L].float().double()
            kk = k8[b, g, :L].float().double() * ks[b, g].double()[at[:L]][:, None]
            vv, qq = code * sv[:, None], q[b, h].double()
            s = (qq @ kk.T * scale).masked_fill(~m, -math.inf)
            row = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(row == -math.inf, torch.zeros_like(row), row)[:, None])
            e = (qq.abs() @ kk.abs().T * scale).amax(-1) * (d + 16) * 2.0 ** -24
            t = p * sv
            top = t.amax(-1, keepdim=True)
            small = (t < 2.0 ** -14 * top).double()
            pv = p @ vv.abs()
            low = 2.0 ** -25 * top
            o[b, h], lse[b, h], E[b, h] = p @ vv, row, e
            bound[b, h] = pv * (u + 2 * e[:, None] + 2.0 ** -18) + low * (small @ code.abs())
            squares = (u + e)[:, None] ** 2 * ((p * p) @ (vv * vv)) + low ** 2 * (small @ (code * code))
            length[b, h] = (squares + (2.0 ** -17 * pv) ** 2).sum(-1).sqrt()
    return o, lse, bound, length, E


def check_attend8(o32, o, lse, q, k8, v8, ks, vs, block, lens, causal, scale=None):
    """o32: the fp32 outputs, o: those in q's type (or None).  Every element, every row's length (where weights are
    even, a tile of wrong values hides within the elements' bound on a long cache, not within this one), the LSE."""
    ro, rl, bound, length, E = attend8(q, k8, v8, ks, vs, block, lens, causal, scale)
    assert bool(torch.isfinite(o32).all())
    err = (o32.double() - ro).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())
    got = err.norm(dim=-1)
    assert bool((got <= length).all()), float((got / length.clamp(min=1e-300)).max())
    if o is not None:
        u = HALF[q.dtype]
        tiny = 2.0 ** -25 if q.dtype == torch.float16 else 2.0 ** -134  # half the smallest step of the type
        assert bool(((o.double() - ro).abs() <= bound + u * (ro.abs() + bound) + tiny).all())
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((o32[empty] == 0).all())
    off = (lse.double() - rl).abs().masked_fill(empty, 0)
    assert bool((off <= E + 2.0 ** -18 + rl.abs().masked_fill(empty, 0) * 2.0 ** -22).all()), float(off.max())

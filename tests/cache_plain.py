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

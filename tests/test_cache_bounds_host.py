"""The bounds that the GPU tests of the 8-bit attention use, tried on the CPU: outputs with the roundings that
the kernels make pass, outputs of a cache with one tile's values wrong do not.  And the attention's workspace."""
import pytest
import torch

from exact_attention_50_gb300 import _lib, build
from tests import cache_plain as P

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def case(L, d, dtype, cache, block, Nq=1, G=1, power=0):
    g = torch.Generator().manual_seed(L + d)
    rows = lambda: torch.randn(1, 1, L, d, generator=g) * torch.exp(0.5 * torch.randn(1, 1, L, 1, generator=g))
    k8, ks = P.quantise(rows(), block, cache)
    v8, vs = P.quantise(rows(), block, cache)
    if power:
        vs = vs * torch.exp2(-(torch.arange(vs.shape[2]) * 5 % power).float())
    return (0.25 * torch.randn(1, G, Nq, d, generator=g)).to(DT[dtype]), k8, v8, ks, vs  # weights of one size: every key counts


def rounded(q, k8, v8, ks, vs, block, causal):
    """P vs in fp16, in units of a power of two just below the row's largest."""
    Nq, L, d = q.shape[2], k8.shape[2], q.shape[3]
    at = torch.arange(L) // block
    o = torch.zeros(q.shape, dtype=torch.float64)
    for h in range(q.shape[1]):
        kk = k8[0, 0].float().double() * ks[0, 0].double()[at][:, None]
        s = (q[0, h].double() @ kk.T / d ** 0.5).masked_fill(~P.seen_keys(Nq, L, L, causal, q.device), -float("inf"))
        p = torch.softmax(s, -1)
        t = p * vs[0, 0].double()[at]
        unit = torch.exp2(torch.floor(torch.log2(t.amax(-1, keepdim=True))))
        o[0, h] = (t / unit).half().double() * unit @ v8[0, 0].float().double()
    return o


CASES = [(30011, 64, "bf16", "i8", 64), (30011, 48, "f16", "e4m3", 16), (12321, 128, "bf16", "i8", 64), (12321, 64, "f16", "e4m3", 64),
         (40001, 64, "f16", "e4m3", 32), (100001, 16, "bf16", "i8", 16), (9000, 112, "f16", "i8", 16), (700, 80, "f16", "i8", 16)]


@pytest.mark.parametrize("L,d,dtype,cache,block", CASES)
def test_one_wrong_tile_is_found(L, d, dtype, cache, block):
    q, k8, v8, ks, vs = case(L, d, dtype, cache, block, G=4)
    ro, rl = P.attend8(q, k8, v8, ks, vs, block, None, False)[:2]
    good = rounded(q, k8, v8, ks, vs, block, False)
    P.check_attend8(good.float(), good.to(q.dtype), rl.float(), q, k8, v8, ks, vs, block, None, False)
    n = 32
    for first in (0, L // 3 // n * n, (L - 1) // n * n - n):
        for what in ("zeros", "the tile before", "a scale"):
            bad8, bads = v8.clone(), vs.clone()
            at = slice(first, first + n)
            if what == "zeros":
                bad8.view(torch.uint8)[0, 0, at] = 0
            elif what == "the tile before":
                bad8.view(torch.uint8)[0, 0, at] = v8.view(torch.uint8)[0, 0, (first - n) % L:][:n]
            else:
                bads[0, 0, first // block] *= 1.25
            wrong = P.attend8(q, k8, bad8, ks, bads, block, None, False)[0]
            if torch.equal(wrong, ro):
                continue
            with pytest.raises(AssertionError):
                P.check_attend8(wrong.float(), None, rl.float(), q, k8, v8, ks, vs, block, None, False)


@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_small_scales_are_held_to_their_own_size(block, dtype):
    """Rows that see a block of 2^-28 only: zeros, or twice its values, are found; so is one small block among others."""
    L, Nq = block + 20, 30
    q, k8, v8, ks, vs = case(L, 64, dtype, "i8", block, Nq)
    vs[:, :, 0] *= 2.0 ** -28
    ro, rl = P.attend8(q, k8, v8, ks, vs, block, None, True)[:2]
    good = rounded(q, k8, v8, ks, vs, block, True)
    P.check_attend8(good.float(), good.to(q.dtype), rl.float(), q, k8, v8, ks, vs, block, None, True)
    for f in (0.0, 2.0, 1.01):
        s = vs.clone()
        s[:, :, 0] *= f
        wrong = P.attend8(q, k8, v8, ks, s, block, None, True)[0]
        with pytest.raises(AssertionError):
            P.check_attend8(wrong.float(), None, rl.float(), q, k8, v8, ks, vs, block, None, True)


def test_scales_over_forty_powers_pass_with_one_rounding():
    for L in (700, 9000):
        q, k8, v8, ks, vs = case(L, 64, "bf16", "i8", 16, Nq=5, G=2, power=41)
        vs[:, :, 3] = 0
        for causal in (True, False):
            rl = P.attend8(q, k8, v8, ks, vs, 16, None, causal)[1]
            good = rounded(q, k8, v8, ks, vs, 16, causal)
            P.check_attend8(good.float(), good.to(q.dtype), rl.float(), q, k8, v8, ks, vs, 16, None, causal)


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,d", [(8, 32, 8, 17, 32768, 128), (64, 32, 8, 32, 32768, 128), (500, 8, 8, 100, 9001, 80), (1, 32, 8, 64, 2 ** 20, 128),
                                              (1, 1, 1, 65, 2 ** 23, 128), (3, 128, 128, 300, 70000, 64)])
def test_workspace_of_many_rows_does_not_grow_with_the_batch(B, Hq, Hkv, Nq, Nk, d):
    """The keys and values of one time in 16 bits (1 GB, or one kv head's), a float per 16 keys of those, and the parts
    of at most 128 ranges of those rows."""
    build.build()
    _lib.load()
    size = _lib.attn_fwd_kvcache8_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)
    pair, rows = 4 * Nk * d, Hq // Hkv * Nq
    held = max(2 ** 30, pair)
    pairs = min(B * Hkv, max(1, 2 ** 30 // pair))
    assert min(pairs * pair // 2, held) <= size <= held * (1 + 1 / (16 * d)) + pairs * 4 + 128 * pairs * rows * (d + 1) * 4 + 2048

"""64-bit references and inputs of the packed-query attention tests."""
import math

import torch

BS = 16
# Bound of one output element against 64 bits.  The weights p are rounded once
# to bf16 (relative 2^-8) and the result once more; scores, exponentials and
# sums are fp32: a score sums D <= 128 exact products, off by at most
# 128 * 2^-24 * sum |q k| * scale < 2^-12 for the inputs here (sum |q k| *
# scale < 32), which is the relative error it gives p, and ex2.approx adds 2^-22.  With
# A = sum p |v| / sum p:  |err| <= 2^-8 |out| + (1 + 2^-8) (2^-8 + 2 * 2^-12) A
# (the 2 * 2^-12: numerator and normaliser).
ROUND = 2.0 ** -8
FP32 = 2.0 ** -12


def out_bound(ref, spread):
    return ROUND * ref.abs() + (1 + ROUND) * (ROUND + 2 * FP32) * spread + 1e-30


# lse = log of the same sum: its absolute error is the scores' (2^-12), the
# logarithm's 2^-22 and one fp32 rounding of the result
def lse_bound(ref):
    return FP32 + 2.0 ** -21 + 2.0 ** -23 * ref.abs()


def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def make_pool(pages, hkv, d, g, device, extra=3):
    """K/V pools of NaN (so that a read of an unowned slot shows), page ids shuffled."""
    n = sum(pages) + extra
    ids = torch.randperm(n, generator=g, device=device).to(torch.int32)
    pool = torch.full((2, n, hkv, BS, d), float("nan"), dtype=torch.bfloat16, device=device)
    return ids, pool


def attend(q, k, v, visible, scale):
    """q [R, D], k, v [T, D] in 64 bits, visible [R, T] -> out, lse, A."""
    s = (q @ k.T) * scale
    s = s.masked_fill(~visible, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, p @ v.abs()


def reference(q, kpool, vpool, table, firsts, counts, lens, limits, hkv, scale, extra=None):
    """Rows [first, first + count) of every sequence over its first `lens`
    tokens; limits[b][i]: positions below it are visible to token i; extra[b]:
    [count, lens] more visible ones, or None."""
    t, hq, d = q.shape
    g = hq // hkv
    dev = q.device
    out = torch.zeros((t, hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((t, hq), dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    for b, (first, count, total) in enumerate(zip(firsts, counts, lens)):
        if count == 0:
            continue
        ids = table[b, :(total + BS - 1) // BS].long()
        pos = torch.arange(total, device=dev)
        vis = pos[None] < torch.as_tensor(limits[b], device=dev)[:, None]
        if extra is not None:
            vis = vis | extra[b]
        vis = vis.repeat_interleave(g, 0)
        for h in range(hkv):
            k = kpool[ids, h].reshape(-1, d)[:total].double()
            v = vpool[ids, h].reshape(-1, d)[:total].double()
            mine = q[first:first + count, h * g:(h + 1) * g].reshape(-1, d).double()
            o, l, a = attend(mine, k, v, vis, scale)
            sl = (slice(first, first + count), slice(h * g, (h + 1) * g))
            out[sl], lse[sl], spread[sl] = o.view(count, g, d), l.view(count, g), a.view(count, g, d)
    return out, lse, spread


def check(got, lse, ref, what=""):
    out_ref, lse_ref, spread = ref
    err = (got.double() - out_ref).abs()
    bound = out_bound(out_ref, spread)
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    if lse is not None:
        worst = ((lse.double() - lse_ref).abs() / lse_bound(lse_ref)).max().item()
        assert worst <= 1.0, f"{what}: lse {worst:.3f} of the bound"

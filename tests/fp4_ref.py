"""64-bit definitions of 4-bit rows, norms, rotation and attention over 4-bit
pages, for the tests (any device)."""
import math

import torch

BS = 16
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.tensor([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127], dtype=torch.float64)  # bytes 0..0x7e


def f32(x):
    return x.float().double()


def nearest(x, table):
    """Index of the table's value nearest to x >= 0; a tie goes to the even index."""
    t = table.to(x.device)
    hi = torch.searchsorted(t, x.contiguous()).clamp(1, len(t) - 1)
    lo = hi - 1
    a, b = x - t[lo], t[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def encode(rows, factor):
    """bf16 rows [..., H, D] -> (codes 0..15 [..., H, D], scale bytes [..., H, D / 16])."""
    x = rows.double().unflatten(-1, (-1, 16))
    f = factor.double()[:, None]
    t = f32(x.abs().amax(-1) / f32(6.0 * f))
    byte = nearest(t.clamp(max=448.0), E4M3)
    step = f32(E4M3.to(x.device)[byte] * f)[..., None]
    q = torch.where(step > 0, f32(x / torch.where(step > 0, step, 1.0)), 0.0)
    code = nearest(q.abs().clamp(max=6.0), LEVELS) + 8 * (torch.signbit(q) & (step > 0)).long()
    return code.flatten(-2), byte


def values(code, byte, factor):
    v = LEVELS.to(code.device)[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    s = E4M3.to(code.device)[byte]
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * factor.double()[:, None]


def pack(code, byte):
    """Rows [..., 9 D / 16] of codes, two a byte, and scales."""
    return torch.cat([(code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8), byte.to(torch.uint8)], -1)


def to_pool(rows):
    """Rows [P, 16, H, 9 D / 16] as a pool [P, H, 9 D]."""
    d = rows.shape[-1] * 16 // 9
    x = rows.transpose(1, 2)
    return torch.cat([x[..., :d // 2].flatten(2), x[..., d // 2:].flatten(2)], -1).contiguous()


def from_pool(pool):
    """(codes, scale bytes) [P, 16, H, D], [P, 16, H, D / 16] of a pool."""
    d = pool.shape[-1] // 9
    raw = pool[..., :8 * d].unflatten(-1, (16, d // 2)).transpose(1, 2).long()
    code = torch.stack([raw & 15, raw >> 4], -1).flatten(-2)
    return code.contiguous(), pool[..., 8 * d:].unflatten(-1, (16, d // 16)).transpose(1, 2).long().contiguous()


def pool_values(pool, factor):
    """Values [P, 16, H, D] of a pool in 64 bits (any value where a scale byte is none)."""
    code, byte = from_pool(pool)
    return values(code, byte.clamp(max=0x7e), factor)


def rotate(x, weight, positions, cos_sin, eps, interleaved):
    """Normed (with a weight) and rotated heads x [T, H, D], and the bound of
    their fp32 form's error before its rounding to bf16: a sum of D <= 256
    squares (2^-16 relative, half of it in the root), the root's 2 ulp and four
    products' roundings, each relative to the terms of the pair: below 2^-15
    (|a| + |b|)."""
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    bound = 2.0 ** -15 * y.abs()
    if cos_sin is not None:
        r = cos_sin.shape[1]
        cs = cos_sin.double()[positions.long()][:, None]
        c, s = cs[..., :r // 2], cs[..., r // 2:]
        sl = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        a, b = y[..., sl[0]], y[..., sl[1]]
        out = y.clone()
        out[..., sl[0]], out[..., sl[1]] = a * c - b * s, b * c + a * s
        for k in sl:
            bound[..., k] = 2.0 ** -15 * (a.abs() + b.abs())
        y = out
    return y, bound


def attention(q, k, v, table, lens, ancestors, scale):
    """q [B, n, Hq, D] over decoded pools k, v [P, 16, H, D] (64 bits); ancestors:
    n masks or None.  Returns out, lse and their error bounds.

    Scores: D products summed in fp32, each sum off by at most 2^-23 of the
    terms' magnitudes (the products are exact), so err = D 2^-23 sum|q k| scale,
    and as much again relative in a weight and in the normaliser.  Weights: 2^-11
    in f16, or 2^-25 of the row's largest weight where they are subnormal; the
    exponential 2^-22.  The result is rounded to bf16 once (2^-8)."""
    b, n, hq, d = q.shape
    hkv = k.shape[2]
    g = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    for i, length in enumerate(lens):
        pos = torch.arange(length + n, device=q.device)
        page = table[i].long()[pos // BS]
        vis = torch.ones((n, length + n), dtype=torch.bool, device=q.device)
        for j in range(n):
            for s in range(n):
                vis[j, length + s] = bool(ancestors[j] >> s & 1) if ancestors is not None else s <= j
        vis = vis.repeat_interleave(g, 0)
        for h in range(hkv):
            kk, vv = k[page, pos % BS, h], v[page, pos % BS, h]
            mine = q[i, :, h * g:(h + 1) * g].reshape(n * g, d).double()
            x = (mine @ kk.T * scale).masked_fill(~vis, -math.inf)
            norm = torch.logsumexp(x, 1)
            p = torch.exp(x - norm[:, None])
            err = d * 2.0 ** -23 * ((mine.abs() @ kk.abs().T) * scale).masked_fill(~vis, 0.0).amax(1)
            o = p @ vv
            rel = 2.0 ** -11 + 2.0 ** -21 + 2 * err
            tiny = 2.0 ** -25 * p.amax(1, keepdim=True) * (vis.double() @ vv.abs())
            bound = 2.0 ** -8 * o.abs() + 1.01 * (rel[:, None] * (p @ vv.abs()) + tiny) + 1e-30
            sl = (i, slice(None), slice(h * g, (h + 1) * g))
            out[sl], lse[sl] = o.view(n, g, d), norm.view(n, g)
            ob[sl], lb[sl] = bound.view(n, g, d), (err + 2.0 ** -20 + 2.0 ** -22 * norm.abs()).view(n, g)
    return out, lse, ob, lb

"""GPU tests of the softmax in svpa_paged_verify_attn_fp4: many small weights
behind a dominant one, and scores that outgrow the reference maxima, in every
number of columns that the kernel is built for."""
import math

import pytest
import torch

import fp4_ref as F
from speculative_verify_paged_attn_gb300 import svpa
from test_gpu_fp4_attn import BF, BS, DEV, Case, gen

pytestmark = pytest.mark.gpu
# (queries, query heads, kv heads): 1, 16, 32, 48, 64, 65, 116 and 128 rows of a kv head
ROWS = [(1, 1, 1), (2, 16, 2), (4, 8, 1), (6, 16, 2), (8, 8, 1), (5, 13, 1), (29, 8, 2), (16, 8, 1)]


def put(c, pool, factor, seq, pos, rows):
    """bf16 rows [len(pos), Hkv, D] at positions of a sequence."""
    code, byte = F.from_pool(pool)
    pos = torch.as_tensor(pos, device=DEV)
    page = c.table[seq].long()[pos // BS]
    code[page, pos % BS], byte[page, pos % BS] = F.encode(rows.to(BF), factor)
    pool.copy_(F.to_pool(F.pack(code, byte)))


@pytest.mark.parametrize("level", [10.0, 14.3, 18.0, 20.6, 22.6, 24.2, 26.0])
@pytest.mark.parametrize("n,hq,hkv", ROWS)
@pytest.mark.parametrize("d,at", [(64, 0), (128, 0), (128, 1490)])
def test_small_weights_behind_a_dominant_one(n, hq, hkv, d, at, level):
    """A token with V = 0, the first one or one that raises the references later,
    takes nearly all of the weight; the others, 2^-level of it each, make the output.

    The bound of a row, with p the normalised weights: a weight is rounded to 11
    bits (2^-11 relative).  The row's largest weight is held as 2^5 at least, so one
    below 2^-19 of it is below f16's smallest normal value, 2^-14, and is rounded to a
    multiple of 2^-24: by at most 2^-25, which is 2^-30 of the largest.  Exponential
    2^-21, scores as in fp4_ref.attention (twice), one rounding to bf16 (2^-8)."""
    ctx, scale = [3000, 4100, 61], 1 / math.sqrt(d)
    c = Case(ctx, n, hq, hkv, d, seed=1, factor=False)
    g = gen(2)
    one = torch.ones((1, hkv, d), device=DEV)
    for i, length in enumerate(ctx):
        every = torch.arange(length + n, device=DEV)
        put(c, c.kp, c.f1, i, every, torch.zeros((length + n, hkv, d), device=DEV))
        first = min(at, length - 1)
        put(c, c.kp, c.f1, i, [first], 0.75 * one)  # 6 * 2^-3: held exactly
        put(c, c.vp, c.f1, i, every, 0.5 + torch.rand((length + n, hkv, d), generator=g, device=DEV))
        put(c, c.vp, c.f1, i, [first], 0.0 * one)
    # the rows' levels lie a little apart
    rows = torch.linspace(0.98, 1.02, n * hq, device=DEV).view(1, n, hq, 1)
    c.q.copy_((level * math.log(2) / (0.75 * d * scale) * rows).expand_as(c.q))
    c.call()
    assert svpa.check_error(c.err) == 0
    k, v = F.pool_values(c.kp, c.f1), F.pool_values(c.vp, c.f1)
    out, lse, _, lb = F.attention(c.q, k, v, c.table, ctx, None, scale)
    assert ((c.lse.double() - lse).abs() <= lb).all()
    gq = hq // hkv
    for i, length in enumerate(ctx):
        pos = torch.arange(length + n, device=DEV)
        page = c.table[i].long()[pos // BS]
        for h in range(hkv):
            kk, vv = k[page, pos % BS, h], v[page, pos % BS, h]
            q = c.q[i, :, h * gq:(h + 1) * gq].reshape(n * gq, d).double()
            x = q @ kk.T * scale
            seen = pos[None] <= length + torch.arange(n, device=DEV).repeat_interleave(gq)[:, None]
            p = torch.softmax(x.masked_fill(~seen, -math.inf), 1)
            err = d * 2.0 ** -23 * (q.abs() @ kk.abs().T * scale).amax(1, keepdim=True)
            want = p @ vv  # (V >= 0: the sum of the terms' magnitudes)
            bound = (2.0 ** -8 + 1.01 * (2.0 ** -11 + 2.0 ** -21 + 2 * err)) * want
            bound = bound + 1.01 * 2.0 ** -30 * p.amax(1, keepdim=True) * (seen.double() @ vv)
            got = c.out[i, :, h * gq:(h + 1) * gq].reshape(n * gq, d).double()
            worst = ((got - want).abs() / bound).max().item()
            assert worst <= 1.0, f"sequence {i}, head {h}: {worst:.2f} of the bound"


@pytest.mark.parametrize("jump", [5.0, 7.9, 8.3, 14.0, 16.0, 31.0, 100.0, 119.0, 125.0, 131.0, 300.0])
@pytest.mark.parametrize("n,hq,hkv", ROWS)
def test_scores_that_jump_between_blocks(n, hq, hkv, jump):
    """Tokens of blocks 1, 2, 3 and on exceed all before them by `jump` log2 units
    each, in the rows of some heads alone: of the first, of the last, of every third."""
    for d, heads in ((128, [0]), (128, [hq - 1]), (64, list(range(0, hq, 3))), (128, list(range(hq)))):
        scale, low = 1 / math.sqrt(d), d // 2
        c = Case([1500, 140, 700], n, hq, hkv, d, seed=n + hq, factor=False)
        # random keys in the lower dimensions, steps in the upper ones: a query of equal
        # upper elements scores i jumps with a row of 2^-4 i, which is held exactly
        code, byte = F.from_pool(c.kp)
        code[..., low:] = 0
        c.kp.copy_(F.to_pool(F.pack(code, byte)))
        c.q[:, :, heads, :low] = 0
        c.q[:, :, heads, low:] = torch.tensor(jump * math.log(2) / (2.0 ** -4 * low * scale), device=DEV).to(BF)
        for i, at in enumerate((130, 260, 400, 513, 640, 900, 1023, 1300)):
            row = torch.zeros((1, hkv, d), device=DEV)
            row[..., low:] = 2.0 ** -4 * (i + 1)
            for s, length in enumerate(c.ctx):
                if at < length:
                    put(c, c.kp, c.f1, s, [at], row)
        c.call()
        c.check()


@pytest.mark.parametrize("n,hq,hkv", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_wide_scores(n, hq, hkv, d):
    """Random scores of some ten and some hundred log2 units: many raises, in any column and block."""
    for spread, seed in ((6.0, 1), (60.0, 2)):
        c = Case([2000, 129, 900, 5], n, hq, hkv, d, tree=n > 2, seed=seed, spread=spread)
        c.call()
        c.check()


def test_wide_scores_of_pairs_cut_between_ctas():
    """One long sequence: nearly every CTA has a part with references of its own."""
    for n, hq, hkv, d in ((1, 8, 8, 128), (6, 8, 1, 128), (16, 8, 1, 64)):
        c = Case([30000], n, hq, hkv, d, seed=n, spread=8.0)
        c.call()
        c.check()

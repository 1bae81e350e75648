"""GPU tests of svpa_paged_verify_attn_fp4 against 64 bits."""
import math
import random

import pytest
import torch

import fp4_ref as F
from speculative_verify_paged_attn_gb300 import svpa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BS = 16
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def tree_masks(n, seed):
    rng = random.Random(seed)
    masks = [1]
    for j in range(1, n):
        masks.append(masks[rng.randrange(j)] | 1 << j)
    return masks


class Case:
    def __init__(self, ctx, n, hq, hkv, d, tree=False, seed=0, scale=None, factor=True, spread=1.0, width=0):
        g = gen(seed)
        b = len(ctx)
        self.ctx, self.n, self.scale = ctx, n, scale or 1 / math.sqrt(d)
        pages = [-(-(c + n) // BS) for c in ctx]
        total = sum(pages) + 3
        ids = torch.randperm(total, generator=g, device=DEV).tolist()
        self.w = max(pages) + width
        self.table = ints([[ids.pop() for _ in range(p)] + [2 ** 31 - 1] * (self.w - p) for p in pages])
        self.kf = 0.5 + torch.rand(hkv, generator=g, device=DEV) if factor else None
        self.vf = 0.5 + torch.rand(hkv, generator=g, device=DEV) if factor else None
        self.f1 = torch.ones(hkv, device=DEV)
        # what no sequence owns: scale bytes that are not numbers
        self.kp, self.vp = [torch.full((total, hkv, 9 * d), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]
        for pool, f in ((self.kp, self.kf), (self.vp, self.vf)):
            code, byte = F.from_pool(pool)
            for i, c in enumerate(ctx):
                pos = torch.arange(c + n, device=DEV)
                x = (torch.randn((c + n, hkv, d), generator=g, device=DEV) * spread).to(BF)
                page = self.table[i].long()[pos // BS]
                code[page, pos % BS], byte[page, pos % BS] = F.encode(x, self.f1 if f is None else f)
            pool.copy_(F.to_pool(F.pack(code, byte)))
        self.q = torch.randn((b, n, hq, d), generator=g, device=DEV).to(BF)
        self.masks = tree_masks(n, seed) if tree else None
        self.p = svpa.attn_params(b, n, hq, hkv, d, self.w, total, kv_fp4=True, sm_scale=self.scale)
        self.ws = torch.zeros(svpa.paged_verify_attn_fp4_workspace_size(self.p), dtype=torch.uint8, device=DEV)
        self.cl = ints(ctx)
        self.err = ints([0])
        self.out = torch.full_like(self.q, float("nan"))
        self.lse = torch.full((b, n, hq), float("nan"), device=DEV)

    def call(self, lse=True, stream=None, ws=None):
        svpa.paged_verify_attn_fp4(self.p, self.q, self.kp, self.vp, self.table, self.cl, self.out,
                                   workspace=self.ws if ws is None else ws, error_flag=self.err, k_factor=self.kf,
                                   v_factor=self.vf, ancestor_mask=self.masks, lse=self.lse if lse else None,
                                   stream=stream)

    def reference(self):
        k, v = [F.pool_values(p, self.f1 if f is None else f) for p, f in ((self.kp, self.kf), (self.vp, self.vf))]
        return F.attention(self.q, k, v, self.table, self.ctx, self.masks, self.scale)

    def check(self, lse=True):
        assert svpa.check_error(self.err) == 0
        out, norm, ob, lb = self.reference()
        assert torch.isfinite(self.out).all()
        worst = ((self.out.double() - out).abs() / ob).max().item()
        assert worst <= 1.0, f"{worst:.3f} of the bound"
        if lse:
            worst = ((self.lse.double() - norm).abs() / lb).max().item()
            assert worst <= 1.0, f"lse: {worst:.3f} of the bound"
        # counters and tickets are left at zero
        assert int(self.ws[:256 + (64 << 10)].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("ctx,n,hq,hkv,d,tree", [
    ([0], 1, 1, 1, 128, False), ([1], 1, 8, 1, 64, False), ([15], 1, 8, 8, 128, False), ([127, 128, 129], 1, 8, 2, 128, False),
    ([5, 0, 300], 3, 4, 4, 64, False), ([112, 125, 126, 127, 128, 130], 6, 16, 2, 128, False),
    ([1000, 3, 517], 6, 64, 8, 128, False), ([260, 31, 700, 16, 2], 5, 32, 32, 128, False), ([400, 90], 16, 8, 1, 128, False),
    ([123, 513], 29, 8, 2, 128, True), ([0, 64, 1023], 29, 8, 2, 64, True), ([900], 64, 2, 1, 128, True),
    ([60, 50], 64, 4, 2, 64, True), ([7], 18, 7, 1, 128, True), ([2047, 2048, 2049], 2, 14, 2, 64, False),
    ([4000], 1, 16, 1, 128, False), ([9000, 40], 6, 8, 1, 128, False), ([300] * 40, 1, 4, 4, 128, False),
    ([130 + 5 * i for i in range(50)], 3, 6, 2, 128, False), ([10] * 300, 2, 4, 2, 64, False),
])
def test_against_64_bits(ctx, n, hq, hkv, d, tree):
    c = Case(ctx, n, hq, hkv, d, tree, seed=len(ctx) + n)
    c.call()
    c.check()


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = random.Random(seed)
    hkv, g = rng.choice([(1, 1), (2, 4), (3, 7), (8, 8), (5, 1), (1, 16), (2, 3)])
    n = rng.randrange(1, min(64, 128 // g) + 1)
    ctx = [rng.randrange(0, rng.choice([20, 300, 2500])) for _ in range(rng.randrange(1, 9))]
    c = Case(ctx, n, hkv * g, hkv, rng.choice([64, 128]), rng.random() < 0.5, seed=100 + seed, factor=rng.random() < 0.7,
             width=rng.randrange(3))
    c.call()
    c.check()


def test_without_lse_and_factors():
    c = Case([200, 33], 4, 8, 2, 128, factor=False)
    c.call(lse=False)
    c.check(lse=False)
    assert torch.isnan(c.lse).all()


def test_scores_that_grow_along_the_history():
    """Later blocks exceed every reference maximum before them."""
    c = Case([1500], 4, 8, 1, 128, seed=3)
    pos = torch.arange(1504, device=DEV)
    code, byte = F.from_pool(c.kp)
    x = (c.q[0, 0, 0].float() * (pos[:, None] / 250.0)).to(BF)[:, None]
    page = c.table[0].long()[pos // BS]
    code[page, pos % BS], byte[page, pos % BS] = F.encode(x, c.kf)
    c.kp.copy_(F.to_pool(F.pack(code, byte)))
    c.call()
    c.check()


@pytest.mark.parametrize("size", [1e-30, 1e-6, 300.0, 1e5])
def test_query_sizes(size):
    """Rows of very different sizes in one sequence; large ones against a small scale."""
    c = Case([333], 5, 8, 2, 128, seed=5, scale=min(0.09, 0.5 / size))
    c.q[0, :, 0] = (c.q[0, :, 0].float() * size).to(BF)
    c.q[0, 2, 5] = 0
    c.call()
    c.check()


@pytest.mark.parametrize("kf,vf", [(2.0 ** -50, 2.0 ** 50), (2.0 ** 50, 2.0 ** -50)])
def test_factors_of_any_size(kf, vf):
    c = Case([200, 17], 3, 8, 2, 64, seed=6, factor=False)
    c.kf, c.vf = torch.full((2,), kf, device=DEV), torch.full((2,), vf, device=DEV)
    c.p.sm_scale = c.scale = 0.125 / kf
    c.call()
    c.check()


def test_masked_slots_do_not_matter():
    """Speculative slots that no row but their own sees, of the largest values there are."""
    c = Case([100], 6, 8, 2, 128, seed=8)
    c.masks = [1 << j | 1 for j in range(6)]
    c.call()
    c.check()
    first = c.out.clone()
    code, byte = F.from_pool(c.kp)
    page = c.table[0].long()[105 // BS]
    code[page, 105 % BS], byte[page, 105 % BS] = 7, 0x7e
    c.kp.copy_(F.to_pool(F.pack(code, byte)))
    c.call()
    c.check()
    assert torch.equal(first[:, :5], c.out[:, :5])


@pytest.mark.parametrize("what,status", [
    ("block", "SVPA_ERR_BAD_BLOCK"), ("negative block", "SVPA_ERR_BAD_BLOCK"), ("length", "SVPA_ERR_INVALID_ARG"),
    ("negative length", "SVPA_ERR_INVALID_ARG"), ("largest length", "SVPA_ERR_INVALID_ARG"),
    ("factor", "SVPA_ERR_INVALID_ARG"), ("query", "SVPA_ERR_INVALID_ARG"),
])
def test_reported_on_the_device(what, status):
    c = Case([300, 40, 77], 3, 8, 2, 128)
    c.call()
    c.check()
    good = c.out.clone()
    c.table, c.cl, saved = c.table.clone(), c.cl.clone(), (c.table, c.cl, c.q.clone(), c.vf.clone())
    if what == "block":
        c.table[1, 1] = c.p.num_blocks
    elif what == "negative block":
        c.table[1, 0] = -1
    elif what == "length":
        c.cl[1] = c.w * BS - 2
    elif what == "negative length":
        c.cl[1] = -1
    elif what == "largest length":
        c.cl[1] = 2 ** 31 - 1
    elif what == "factor":
        c.vf[1] = float("nan")
    else:
        c.q[1, 1, 3, 77] = float("inf")
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == status
    if "length" in what or "block" in what:  # the other sequences' rows are right
        assert torch.equal(c.out[0], good[0]) and torch.equal(c.out[2], good[2])
    # the next call is right
    c.err.zero_()
    c.table, c.cl, c.q, c.vf = saved
    c.out.fill_(float("nan"))
    c.call()
    c.check()


def test_same_bits_every_time_and_in_a_graph():
    c = Case([700, 30, 2000], 6, 16, 2, 128, seed=9)
    c.call()
    c.check()
    first = c.out.clone(), c.lse.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    for _ in range(3):
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)
    # new lengths in the captured buffers
    c.ctx = [650, 29, 5]
    c.cl.copy_(ints(c.ctx))
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_two_calls_at_once_with_their_own_workspaces():
    a, b = Case([3000, 200], 6, 64, 8, 128, seed=1), Case([2500] * 3, 5, 8, 8, 128, seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(stream=sa)
        b.call(stream=sb)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_one_workspace_for_calls_in_turn():
    cases = [Case([700, 90], 6, 64, 8, 128, seed=1), Case([50] * 9, 1, 4, 4, 64, seed=2),
             Case([1500], 29, 8, 2, 128, True, seed=3)]
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device=DEV)
    q = torch.randn((2, 5, 8, 128), device=DEV).to(BF)
    pool = torch.randn((40, 2, 16, 128), device=DEV).to(BF)
    p = svpa.attn_params(2, 5, 8, 2, 128, 20, 40)
    big = torch.zeros(max(ws.numel(), svpa.attn_workspace_size(p)), dtype=torch.uint8, device=DEV)
    t, cl, err = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20), ints([300, 200]), ints([0])
    alone, out = torch.empty_like(q), torch.empty_like(q)
    svpa.paged_verify_attn(p, q, pool, pool, t, cl, alone, workspace=torch.zeros_like(big), error_flag=err)
    for c in cases + cases[::-1]:
        c.call(ws=big)
        svpa.paged_verify_attn(p, q, pool, pool, t, cl, out, workspace=big, error_flag=err)
        c.check()
        assert torch.equal(alone, out)
    assert svpa.check_error(err) == 0


def test_more_pairs_than_tickets():
    """20000 (sequence, kv head) pairs: their tickets lie where other calls keep partial results."""
    c = Case([40] * 2500, 1, 8, 8, 64, seed=4)
    c.ws = torch.cat([c.ws[:256], c.ws[256:].fill_(0xff)])
    c.call()
    assert svpa.check_error(c.err) == 0
    got = c.out.clone()
    # the same sequences, a few at a time
    for first in (0, 1200, 2400):
        p = svpa.attn_params(100, 1, 8, 8, 64, c.w, c.p.num_blocks, kv_fp4=True, sm_scale=c.scale)
        ws = torch.zeros(svpa.paged_verify_attn_fp4_workspace_size(p), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(c.q[:100])
        svpa.paged_verify_attn_fp4(p, c.q[first:first + 100].contiguous(), c.kp, c.vp,
                                   c.table[first:first + 100].contiguous(), c.cl[first:first + 100].contiguous(), out,
                                   workspace=ws, error_flag=c.err, k_factor=c.kf, v_factor=c.vf)
        assert svpa.check_error(c.err) == 0
        ref = out.double()
        # (parts may be joined elsewhere: two roundings to bf16 and to f16 apart)
        assert ((got[first:first + 100].double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -10).all()


def test_empty_batch():
    c = Case([5], 1, 2, 1, 64)
    c.p.batch = 0
    c.call()
    assert svpa.check_error(c.err) == 0 and torch.isnan(c.out).all()


def test_pages_far_in_the_pool():
    """Pools of more than 2^32 bytes: the same sequences in pages at their ends."""
    c = Case([200, 33], 3, 8, 2, 64, seed=11)
    c.call()
    c.check()
    near, lse = c.out.clone(), c.lse.clone()
    blocks = 3_800_000  # 4.4 GB each
    shift = blocks - c.p.num_blocks
    far = [torch.zeros((blocks, 2, 9 * 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for big, small in zip(far, (c.kp, c.vp)):
        big[shift:] = small
    p = svpa.attn_params(2, 3, 8, 2, 64, c.w, blocks, kv_fp4=True, sm_scale=c.scale)
    table = torch.where(c.table < c.p.num_blocks, c.table + shift, c.table)
    c.out.fill_(float("nan"))
    svpa.paged_verify_attn_fp4(p, c.q, *far, table, c.cl, c.out, workspace=c.ws, error_flag=c.err, k_factor=c.kf,
                               v_factor=c.vf, lse=c.lse)
    assert svpa.check_error(c.err) == 0 and torch.equal(c.out, near) and torch.equal(c.lse, lse)


def test_captured_graphs_of_one_workspace_in_turn():
    a, b = Case([900, 40], 5, 16, 2, 128, seed=12), Case([300] * 7, 1, 8, 8, 64, seed=13)
    ws = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device=DEV)
    graphs, side = [], torch.cuda.Stream()
    for c in (a, b):
        c.call(ws=ws)
        c.check()
        c.first = c.out.clone(), c.lse.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.call(ws=ws)
        graphs.append(g)
    for _ in range(3):
        for c, g in zip((a, b), graphs):
            c.out.fill_(float("nan"))
            g.replay()
    torch.cuda.synchronize()
    for c in (a, b):
        assert svpa.check_error(c.err) == 0
        assert torch.equal(c.first[0], c.out) and torch.equal(c.first[1], c.lse)

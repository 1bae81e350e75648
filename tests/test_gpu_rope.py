"""GPU tests of svpa_qk_norm_rope, svpa_rope_kv_write, svpa_kv_read and
svpa_kv_append_fp4, and of the tree commit on 4-bit pages."""
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


def table(rows, r):
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (
        -torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Rows:
    """Queries, keys and values of t tokens, contiguous or slices of one projection."""

    def __init__(self, t, hq, hkv, d, r, norm=True, fused=False, seed=0, far=5000):
        g = gen(seed)
        x = (torch.randn((t, hq + 2 * hkv, d), generator=g, device=DEV) * 3).to(BF)
        parts = x.split([hq, hkv, hkv], 1)
        self.q, self.k, self.v = parts if fused else [p.contiguous() for p in parts]
        self.pos = torch.randint(0, far, (t,), generator=g, device=DEV).to(torch.int32)
        self.table = table(far, r) if r else None
        self.qw = (1 + torch.randn(d, generator=g, device=DEV) / 4).to(BF) if norm else None
        self.kw = (1 + torch.randn(d, generator=g, device=DEV) / 4).to(BF) if norm else None
        self.err = ints([0])
        self.t, self.hq, self.hkv, self.d = t, hq, hkv, d

    def call(self, q_out, k_out, **kw):
        svpa.qk_norm_rope(self.q, self.k, self.pos, self.table, q_out, k_out, error_flag=self.err, q_weight=self.qw,
                          k_weight=self.kw, eps=1e-5, **kw)

    def rotated(self, interleaved=False):
        q = torch.full((self.t, self.hq, self.d), float("nan"), dtype=BF, device=DEV)
        k = torch.full((self.t, self.hkv, self.d), float("nan"), dtype=BF, device=DEV)
        self.call(q, k, interleaved=interleaved)
        assert svpa.check_error(self.err) == 0
        return q, k


def close(got, ref, bound):
    err = (got.double() - ref).abs()
    # one rounding to bf16 of a value that is off by the bound
    limit = 2.0 ** -8 * ref.abs() + 1.01 * bound + 1e-38
    assert torch.isfinite(got).all()
    assert (err <= limit).all(), (err / limit).max().item()


@pytest.mark.parametrize("t,hq,hkv,d,r,norm,interleaved,fused", [
    (1, 8, 1, 128, 128, True, False, False), (5, 64, 8, 128, 128, True, False, True), (33, 7, 7, 64, 64, False, True, True),
    (17, 14, 2, 128, 64, True, False, False), (9, 3, 1, 256, 256, True, True, True), (6, 5, 3, 256, 48, True, False, True),
    (40, 32, 32, 128, 96, False, False, False), (3, 9, 4, 64, 16, True, True, False), (700, 4, 2, 128, 128, True, False, True),
    (4, 2, 1, 128, 0, True, False, False), (4, 17, 9, 64, 32, True, False, False),
])
def test_norm_and_rotation(t, hq, hkv, d, r, norm, interleaved, fused):
    x = Rows(t, hq, hkv, d, r, norm, fused)
    q, k = x.rotated(interleaved)
    close(q, *F.rotate(x.q, x.qw, x.pos, x.table, 1e-5, interleaved))
    close(k, *F.rotate(x.k, x.kw, x.pos, x.table, 1e-5, interleaved))


@pytest.mark.parametrize("r", [128, 0])
def test_in_place_and_one_side_only(r):
    x = Rows(21, 6, 2, 128, r, fused=True)
    q, k = x.rotated()
    keep = x.v.clone()
    x.call(x.q, x.k)  # within the projection
    assert torch.equal(x.q, q) and torch.equal(x.k, k) and torch.equal(x.v, keep)
    y = Rows(21, 6, 2, 128, r, fused=True)
    ko = torch.empty_like(k)
    svpa.qk_norm_rope(None, y.k, y.pos, y.table, None, ko, error_flag=y.err, k_weight=y.kw, eps=1e-5)
    assert torch.equal(ko, k)
    # a weight for the queries alone: the keys turn unnormed
    svpa.qk_norm_rope(y.q, y.k, y.pos, y.table, torch.empty_like(q), ko, error_flag=y.err, q_weight=y.qw, eps=1e-5)
    close(ko, *F.rotate(y.k, None, y.pos, y.table, 1e-5, False))
    assert svpa.check_error(y.err) == 0


def test_small_and_large_rows():
    x = Rows(4, 2, 1, 64, 64)
    x.q[0], x.q[1], x.q[2] = 0, 1e-20, 1e15
    q, _ = x.rotated()
    close(q, *F.rotate(x.q, x.qw, x.pos, x.table, 1e-5, False))
    assert (q[0] == 0).all()


def test_bad_positions_are_reported():
    for bad in (-1, 5000, 2 ** 31 - 1):
        x = Rows(9, 4, 2, 64, 64)
        x.pos[4] = bad
        q, k = torch.zeros_like(x.q), torch.zeros_like(x.k)
        x.call(q, k)
        assert svpa.STATUS[svpa.check_error(x.err)] == "SVPA_ERR_INVALID_ARG"
        assert (q[4] == 0).all() and (k[4] == 0).all()


# ---------------------------------------------------------------- pages
def empty_pool(kind, blocks, hkv, d):
    if kind == "bf16":
        return torch.full((blocks, hkv, BS, d), 7.0, dtype=BF, device=DEV), None
    if kind == "fp8":
        return (torch.full((blocks, hkv, BS, d), 0x21, dtype=torch.uint8, device=DEV),
                torch.full((blocks, hkv, BS, d // 64), 3.0, device=DEV))
    return torch.full((blocks, hkv, 9 * d), 0x21, dtype=torch.uint8, device=DEV), None


def some_slots(t, blocks, seed, holes=0):
    rng = random.Random(seed)
    s = rng.sample(range(blocks * BS), t)
    for i in rng.sample(range(t), holes):
        s[i] = -1 - rng.randrange(3)
    return ints(s)


def factors(hkv, seed, lo=0.3, hi=2.0):
    return lo + (hi - lo) * torch.rand(hkv, generator=gen(seed), device=DEV)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("t,hq,hkv,d,r,fused,holes", [
    (1, 8, 1, 128, 128, False, 0), (37, 14, 2, 64, 64, True, 4), (60, 4, 9, 128, 64, True, 9), (150, 0, 3, 256, 256, False, 0),
    (20, 8, 33, 64, 0, True, 1),
])
def test_write_is_rotation_then_write(kind, t, hq, hkv, d, r, fused, holes):
    blocks = -(-t // BS) + 3
    x = Rows(t, hq, hkv, d, r, True, fused, seed=t)
    slots = some_slots(t, blocks, t, holes)
    live = slots >= 0
    if r:
        x.pos[~live] = -5  # a padding row's position is not read
    kp, ks = empty_pool(kind, blocks, hkv, d)
    vp, vs = empty_pool(kind, blocks, hkv, d)
    start = kp.clone()
    kf, vf = (factors(hkv, 1), factors(hkv, 2)) if kind == "fp4" else (None, None)
    q_out = torch.full((t, hq, d), 9.0, dtype=BF, device=DEV) if hq else None
    svpa.rope_kv_write(x.k, x.v, x.pos, slots, x.table, kp, vp, error_flag=x.err, q=x.q if hq else None, q_out=q_out,
                       q_weight=x.qw if hq else None, k_weight=x.kw, eps=1e-5, k_scale=ks, v_scale=vs,
                       scale_tile=64 if kind == "fp8" else 0, fp4=kind == "fp4", k_factor=kf, v_factor=vf)
    assert svpa.check_error(x.err) == 0
    x.pos[~live] = 0
    if hq:
        q, k = x.rotated()
        q[~live] = 9.0
        assert torch.equal(q_out, q)
    else:
        k = torch.empty_like(x.k)
        svpa.qk_norm_rope(None, x.k, x.pos, x.table, None, k, error_flag=x.err, k_weight=x.kw, eps=1e-5)
    if kind != "fp4":
        kp2, ks2 = empty_pool(kind, blocks, hkv, d)
        vp2, vs2 = empty_pool(kind, blocks, hkv, d)
        svpa.kv_write(k, x.v.contiguous(), slots, kp2, vp2, error_flag=x.err, k_scale=ks2, v_scale=vs2,
                      scale_tile=64 if kind == "fp8" else 0)
        assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
        if kind == "fp8":
            assert torch.equal(ks, ks2) and torch.equal(vs, vs2)
    else:
        for pool, rows, f in ((kp, k, kf), (vp, x.v, vf)):
            code, byte = F.from_pool(start)
            c, s = F.encode(rows[live], f)
            code.flatten(0, 1)[slots[live].long()] = c
            byte.flatten(0, 1)[slots[live].long()] = s
            assert torch.equal(pool, F.to_pool(F.pack(code, byte)))
    # and read back, padding rows left as they were
    ko = torch.full((t, hkv, d), 5.0, dtype=BF, device=DEV)
    vo = torch.full((t, 2 * hkv, d), 5.0, dtype=BF, device=DEV)[:, hkv:]  # out of a wider buffer
    svpa.kv_read(slots, kp, vp, ko, vo, error_flag=x.err, k_scale=ks, v_scale=vs, scale_tile=64 if kind == "fp8" else 0,
                 fp4=kind == "fp4", k_factor=kf, v_factor=vf)
    assert svpa.check_error(x.err) == 0
    for got, pool, sc, f in ((ko, kp, ks, kf), (vo, vp, vs, vf)):
        if kind == "bf16":
            want = pool.transpose(1, 2).flatten(0, 1)
        elif kind == "fp8":
            want = (pool.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 64)) * sc[..., None]).flatten(-2)
            want = want.transpose(1, 2).flatten(0, 1).to(BF)
        else:
            code, byte = F.from_pool(pool)
            want = F.values(code, byte, torch.ones_like(f)).float() * f[:, None]  # a product exact, then one rounding
            want = want.to(BF).flatten(0, 1)
        want = want[slots.long().clamp(min=0)]
        want[~live] = 5.0
        assert torch.equal(got, want)


@pytest.mark.parametrize("seed", range(4))
def test_codes_of_all_magnitudes(seed):
    """Every finite bf16 value meets scales and factors of many sizes, borders and ties among them."""
    bits = torch.arange(0, 0x10000, dtype=torch.int32, device=DEV)
    x = bits[(bits & 0x7fff) < 0x7f80].to(torch.int16).view(BF)
    g = gen(seed)
    if seed < 3:  # neighbours in magnitude share a group
        x = x[torch.argsort(x.abs().float(), stable=True)]
    else:
        x = x[torch.randperm(x.numel(), generator=g, device=DEV)]
    n = x.numel() // 128 * 128
    k = x[:n].view(-1, 1, 128).contiguous()
    f = torch.tensor([[1.0], [1.1], [2.0 ** -60], [1.5 * 2.0 ** 59]][seed], device=DEV)
    blocks = -(-k.shape[0] // BS)
    kp, vp = empty_pool("fp4", blocks, 1, 128)[0], empty_pool("fp4", blocks, 1, 128)[0]
    start = kp.clone()
    slots = torch.arange(k.shape[0], dtype=torch.int32, device=DEV)
    err = ints([0])
    svpa.rope_kv_write(k, k, slots, slots, None, kp, vp, error_flag=err, fp4=True, k_factor=f, v_factor=None)
    assert svpa.check_error(err) == 0
    for pool, fac in ((kp, f), (vp, torch.ones(1, device=DEV))):
        code, byte = F.from_pool(start)
        code.flatten(0, 1)[:k.shape[0]], byte.flatten(0, 1)[:k.shape[0]] = F.encode(k, fac)
        assert torch.equal(pool, F.to_pool(F.pack(code, byte)))


def test_what_cannot_be_held_is_reported():
    def run(k=None, f=None, slot=None, v=None):
        x = Rows(5, 1, 2, 64, 0)
        if k is not None:
            x.k[3, 1, 17] = k
        if v is not None:
            x.v[2, 0, 63] = v
        slots = ints([0, 1, 2, 3, 4 if slot is None else slot])
        kp, vp = empty_pool("fp4", 2, 2, 64)[0], empty_pool("fp4", 2, 2, 64)[0]
        fac = None if f is None else torch.tensor([1.0, f], device=DEV)
        svpa.rope_kv_write(x.k, x.v, slots, slots, None, kp, vp, error_flag=x.err, fp4=True, k_factor=fac)
        return svpa.STATUS[svpa.check_error(x.err)]
    assert run() == "SVPA_OK"
    for bad in (float("nan"), float("inf"), float("-inf")):
        assert run(k=bad) == "SVPA_ERR_INVALID_ARG" and run(v=bad) == "SVPA_ERR_INVALID_ARG"
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -61, 2.0 ** 61):
        assert run(f=bad) == "SVPA_ERR_INVALID_ARG"
    assert run(slot=32) == "SVPA_ERR_BAD_BLOCK" and run(slot=2 ** 31 - 1) == "SVPA_ERR_BAD_BLOCK"
    err, kp = ints([0]), empty_pool("fp4", 2, 2, 64)[0]
    rows = torch.empty((2, 2, 64), dtype=BF, device=DEV)
    svpa.kv_read(ints([3, 32]), kp, kp, rows, rows.clone(), error_flag=err, fp4=True)
    assert svpa.STATUS[svpa.check_error(err)] == "SVPA_ERR_BAD_BLOCK"


# ---------------------------------------------------------------- a step's append
class Append:
    def __init__(self, ctx, n_new, hkv, d, shared=0, seed=0, free=None):
        """Sequences of ctx[b] tokens, the first `shared` tokens (whole pages and a
        part of one) in pages that all of them hold."""
        g = gen(seed)
        self.ctx, self.n, self.hkv, self.d, b = ctx, n_new, hkv, d, len(ctx)
        held = [-(-c // BS) for c in ctx]
        self.width = max(-(-(c + n_new) // BS) for c in ctx) + 1
        sp = -(-shared // BS)
        need = sum(-(-(c + n_new) // BS) for c in ctx) + sp + 2
        ids = torch.randperm(need, generator=g, device=DEV).tolist()
        common = [ids.pop() for _ in range(sp)]
        self.blocks = need
        rows, count = [], [0] * need
        for h in held:
            mine = common[:min(h, sp)] + [ids.pop() for _ in range(max(0, h - sp))]
            for x in mine:
                count[x] += 1
            rows.append(mine + [-1] * (self.width - h))
        self.table, self.count = ints(rows), ints(count)
        self.free = ints(ids + [-1] * (need - len(ids)))
        self.top = ints([len(ids) if free is None else free])
        self.cl = ints(ctx)
        self.kf, self.vf = factors(hkv, seed + 1), factors(hkv, seed + 2)
        self.kp, self.vp = [torch.randint(0, 0x7f, (need, hkv, 9 * d), generator=g, device=DEV).to(torch.uint8)
                            for _ in range(2)]
        self.k, self.v = [torch.randn((b, n_new, hkv, d), generator=g, device=DEV).to(BF) for _ in range(2)]
        self.err = ints([0])

    def gathered(self, pool, table, length):
        code, byte = F.from_pool(pool)
        pos = torch.arange(length, device=DEV)
        page = table.long()[pos // BS]
        return code[page, pos % BS], byte[page, pos % BS]

    def run(self):
        before = [[self.gathered(p, t, c) for t, c in zip(self.table.clone(), self.ctx)] for p in (self.kp, self.vp)]
        top = int(self.top)
        svpa.kv_append_fp4(self.k, self.v, self.table, self.cl, self.count, self.free, self.top, self.kp, self.vp,
                           error_flag=self.err, k_factor=self.kf, v_factor=self.vf)
        assert svpa.check_error(self.err) == 0
        for pool, old, new, f in ((self.kp, before[0], self.k, self.kf), (self.vp, before[1], self.v, self.vf)):
            for b, c in enumerate(self.ctx):
                code, byte = self.gathered(pool, self.table[b], c + self.n)
                wc, ws = F.encode(new[b], f)
                assert torch.equal(code[:c], old[b][0]) and torch.equal(byte[:c], old[b][1])
                assert torch.equal(code[c:], wc) and torch.equal(byte[c:], ws)
        held = torch.bincount(self.table[self.table >= 0].long(), minlength=self.blocks)
        assert torch.equal(held.int(), self.count)
        assert top - int(self.top) == int((self.count > 0).sum()) - (self.blocks - top)


@pytest.mark.parametrize("ctx,n_new,hkv,d,shared", [
    ([0], 1, 1, 64, 0), ([3, 15, 16, 31, 100], 5, 8, 128, 0), ([0, 1, 40], 40, 3, 64, 0), ([29] * 7, 4, 2, 128, 29),
    ([16 + i for i in range(33)], 17, 2, 64, 16), ([200, 7], 3, 33, 64, 0), ([5, 21], 6, 1, 16, 0), ([9], 2, 2, 1024, 0),
])
def test_append(ctx, n_new, hkv, d, shared):
    Append(ctx, n_new, hkv, d, shared).run()


def test_append_without_free_blocks():
    a = Append([15, 15], 5, 2, 64, free=1)
    kp = a.kp.clone()
    svpa.kv_append_fp4(a.k, a.v, a.table, a.cl, a.count, a.free, a.top, a.kp, a.vp, error_flag=a.err)
    assert svpa.STATUS[svpa.check_error(a.err)] == "SVPA_ERR_OUT_OF_BLOCKS" and torch.equal(kp, a.kp)


@pytest.mark.parametrize("d", [64, 128])
def test_tree_commit_moves_4_bit_rows(d):
    n, ctx = 9, [14, 30, 3]
    a = Append(ctx, n, 3, d, seed=4)
    a.run()
    path = ints([[0, 2, 5, 8, -1], [0, 1, -1, -1, -1], [0, 4, 7, -1, -1]])
    taken = [3, 0, 2]
    before = [[a.gathered(p, a.table[b], c + n) for b, c in enumerate(ctx)] for p in (a.kp, a.vp)]
    svpa.block_table_commit(n, a.table, a.cl, ints(taken), a.count, a.free, a.top, error_flag=a.err, path_nodes=path,
                            k_pool=a.kp, v_pool=a.vp, num_kv_heads=3, head_dim=d, kv_fp4=True)
    assert svpa.check_error(a.err) == 0 and a.cl.tolist() == [c + k + 1 for c, k in zip(ctx, taken)]
    for pool, old in ((a.kp, before[0]), (a.vp, before[1])):
        for b, (c, k) in enumerate(zip(ctx, taken)):
            keep = list(range(c + 1)) + [c + int(x) for x in path[b, 1:k + 1]]
            code, byte = a.gathered(pool, a.table[b], c + k + 1)
            assert torch.equal(code, old[b][0][keep]) and torch.equal(byte, old[b][1][keep])


def test_far_slots():
    """Pools of more than 2^32 bytes."""
    blocks, hkv, d = 3_800_000, 2, 64  # 4.4 GB each
    pool = torch.zeros((blocks, hkv, 9 * d), dtype=torch.uint8, device=DEV)
    x = Rows(4, 1, hkv, d, 0)
    slots = ints([blocks * BS - 1, 3, blocks * BS - 17, (blocks - 5) * BS])
    svpa.rope_kv_write(x.k, x.k, slots, slots, None, pool, pool, error_flag=x.err, fp4=True)
    ko = torch.empty_like(x.k)
    svpa.kv_read(slots, pool, pool, ko, torch.empty_like(ko), error_flag=x.err, fp4=True)
    assert svpa.check_error(x.err) == 0
    want = F.values(*F.encode(x.k, torch.ones(hkv, device=DEV)), torch.ones(hkv, device=DEV))
    assert torch.equal(ko.double(), want)
    assert int((pool != 0).flatten(1).any(1).sum()) == 4


@pytest.mark.parametrize("t,hkv,d", [(1, 1, 64), (300, 32, 128), (3000, 8, 128), (9000, 3, 128), (5000, 40, 128),
                                     (4999, 33, 128)])
def test_reads_of_any_length(t, hkv, d):
    """Few rows, many, and many of long rows: every slot of a pool in an order of its own, two pages never named."""
    g = gen(t)
    blocks = -(-t // BS) + 2
    pool = [torch.randint(0, 256, (blocks, hkv, 9 * d), generator=g, device=DEV).to(torch.uint8) for _ in range(2)]
    for p in pool:  # scales that the writes store
        p[..., 8 * d:] &= 0x7f
        p[..., 8 * d:].clamp_(max=0x7e)
    slots = torch.randperm((blocks - 2) * BS, generator=g, device=DEV)[:t].to(torch.int32)
    out = torch.full((2, t, hkv + 1, d), float("nan"), dtype=BF, device=DEV)
    kf, vf = factors(hkv, t), factors(hkv, t + 1)
    err = ints([0])
    svpa.kv_read(slots, *pool, out[0, :, :hkv], out[1, :, :hkv], error_flag=err, fp4=True, k_factor=kf, v_factor=vf)
    assert svpa.check_error(err) == 0
    for got, p, f in zip(out, pool, (kf, vf)):
        want = F.pool_values(p, f)[slots.long() // BS, slots.long() % BS]
        # code times scale is exact; one product in fp32, one rounding to bf16
        assert torch.equal(got[:, :hkv], want.float().to(BF)) and torch.isnan(got[:, hkv:]).all()


@pytest.mark.parametrize("t", [1, 60, 61, 200, 300, 620, 1300, 2600])
def test_a_token_does_not_depend_on_the_others(t):
    """The same tokens alone and among many: each number of words a lane and of warps a token."""
    x = Rows(2600, 64, 8, 128, 128, fused=True, seed=7)
    q, k = x.rotated()
    y = Rows(2600, 64, 8, 128, 128, fused=True, seed=7)
    y.t, y.q, y.k, y.v, y.pos = t, y.q[:t], y.k[:t], y.v[:t], y.pos[:t]
    got = y.rotated()
    assert torch.equal(got[0], q[:t]) and torch.equal(got[1], k[:t])

"""GPU tests of svpa_block_table_build, svpa_kv_write and svpa_logits_process."""
import random

import pytest
import torch

from speculative_verify_paged_attn_gb300 import svpa
from speculative_verify_paged_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BS = 16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- block tables
class Build:
    def __init__(self, lens, prefix=0, width=None, spare=0, free=None, seed=0):
        rng = random.Random(seed)
        self.lens, self.prefix = list(lens), prefix
        self.pages = [-(-n // BS) for n in lens]
        need = sum(p - prefix // BS for n, p in zip(lens, self.pages) if n > 0)
        total = need + prefix // BS + 7
        ids = list(range(total))
        rng.shuffle(ids)
        self.blocks, stack = ids[:prefix // BS], ids[prefix // BS:]
        self.top = len(stack) if free is None else free
        self.width = width or max(max(self.pages), prefix // BS, 1)
        self.new = sum(max(n - prefix, 0) for n in lens)
        self.count = [0] * total
        for i in self.blocks:
            self.count[i] = 1 + rng.randrange(3)
        self.stack = stack + [-5] * (total - len(stack))
        self.d = dict(lens=ints(self.lens), table=ints([[-99] * self.width] * len(lens)),
                      cu=ints([-99] * (len(lens) + 1)), slots=ints([-99] * (self.new + spare)), count=ints(self.count),
                      stack=ints(self.stack), top=ints([self.top]))
        self.prefix_blocks = ints(self.blocks) if prefix else None
        self.ws = torch.zeros(svpa.block_table_build_workspace_size(len(lens)), dtype=torch.uint8, device=DEV)
        self.err = ints([0])

    def call(self, stream=None):
        d = self.d
        svpa.block_table_build(d["lens"], d["table"], d["cu"], d["slots"], d["count"], d["stack"], d["top"],
                               workspace=self.ws, error_flag=self.err, prefix_blocks=self.prefix_blocks, stream=stream)

    def expected(self):
        top, count = self.top, list(self.count)
        table, cu, slots = [], [0], []
        for n, pages in zip(self.lens, self.pages):
            row = []
            if n > 0:
                row = list(self.blocks)
                for b in row:
                    count[b] += 1
                while len(row) < pages:
                    top -= 1
                    row.append(self.stack[top])
                    count[row[-1]] = 1
                slots += [row[p // BS] * BS + p % BS for p in range(self.prefix, n)]
            table.append(row + [-1] * (self.width - len(row)))
            cu.append(len(slots))
        slots += [-1] * (self.d["slots"].numel() - len(slots))
        return dict(lens=self.lens, table=table, cu=cu, slots=slots, count=count, stack=self.stack, top=[top])

    def check(self):
        assert svpa.check_error(self.err) == 0
        assert int(self.ws.view(torch.int32).abs().sum()) == 0
        want = self.expected()
        for name, t in self.d.items():
            assert t.tolist() == want[name], name


@pytest.mark.parametrize("lens,prefix,kw", [
    ([1], 0, {}), ([16], 0, dict(width=9)), ([17, 0, 15, 16, 1], 0, dict(spare=3)), ([0, 0, 0], 0, {}),
    ([48, 33, 32], 32, dict(spare=1)), ([0, 100, 0], 96, dict(width=31)), ([800, 800], 800, dict(spare=5)),
    ([5000, 1, 333, 4096], 0, dict(width=400)), (list(range(1, 600)), 0, {}), ([40] * 1000, 16, dict(width=3)),
    ([20000, 7, 20000], 0, dict(width=1251, spare=50)), ([3] * 8192, 0, dict(width=1)),
    ([20 + i % 3 for i in range(8192)], 16, dict(width=5, spare=3)),
])
def test_tables_and_slots(lens, prefix, kw):
    c = Build(lens, prefix, **kw)
    c.call()
    c.check()


def test_random_tables():
    for seed in range(25):
        rng = random.Random(seed)
        prefix = BS * rng.choice([0, 0, 1, 5])
        lens = [rng.choice([0, prefix + rng.randrange(1, 700)]) for _ in range(rng.randrange(1, 70))]
        c = Build(lens, prefix, spare=rng.randrange(4), seed=seed)
        c.call()
        c.check()


@pytest.mark.parametrize("what,status", [
    ("negative", "SVPA_ERR_INVALID_ARG"), ("below prefix", "SVPA_ERR_INVALID_ARG"),
    ("past the table", "SVPA_ERR_INVALID_ARG"), ("slots", "SVPA_ERR_INVALID_ARG"), ("top", "SVPA_ERR_INVALID_ARG"),
    ("dead prefix", "SVPA_ERR_INVALID_ARG"), ("blocks", "SVPA_ERR_OUT_OF_BLOCKS"), ("prefix", "SVPA_ERR_BAD_BLOCK"),
])
def test_refused_on_the_device_and_nothing_changed(what, status):
    c = Build([40 + i for i in range(300)], 32)
    if what == "negative":
        c.d["lens"][7] = -1
    elif what == "below prefix":
        c.d["lens"][7] = 31
    elif what == "past the table":
        c.d["lens"][7] = c.width * BS + 1
    elif what == "slots":
        c.d["slots"] = c.d["slots"][:-1].clone()
    elif what == "top":
        c.d["top"].fill_(c.d["count"].numel() + 1)
    elif what == "dead prefix":
        c.d["count"][c.blocks[1]] = 0
    elif what == "blocks":
        c.d["top"].fill_(sum(c.pages) - 2 * 300 - 1)
    else:
        c.prefix_blocks[1] = c.d["count"].numel()
    before = {k: v.clone() for k, v in c.d.items()}
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == status
    for k, v in c.d.items():
        assert torch.equal(v, before[k]), k
    assert int(c.ws.view(torch.int32).abs().sum()) == 0


def test_a_bad_stack_entry_is_reported_and_skipped():
    c = Build([40, 50], 0)
    c.d["stack"][c.top - 3] = 1 << 29
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_BAD_BLOCK"
    assert int(c.d["table"][0, 2]) == -1 and c.d["slots"][32:40].tolist() == [-1] * 8


def test_tables_captured():
    c = Build([100, 33, 0, 250], 32, spare=4)
    start = {k: v.clone() for k, v in c.d.items()}
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    for _ in range(2):
        for k, v in start.items():
            c.d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        c.check()


# ---------------------------------------------------------------- K/V scatter
def write_case(t, hkv, d, fp8, fused, seed=0, holes=()):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    nb = -(-t // BS) + 3
    wide = hkv * (4 if fused else 1)
    x = (torch.randn((2, t, wide, d), generator=g, device=DEV) * 3).to(torch.bfloat16)
    k, v = (x[0][:, hkv:2 * hkv], x[0][:, 2 * hkv:3 * hkv]) if fused else (x[0], x[1])
    slots = torch.randperm(nb * BS, generator=g, device=DEV)[:t].to(torch.int32)
    for i in holes:
        slots[i] = -1 - i
    kind = torch.uint8 if fp8 else torch.int16
    pools = [torch.randint(0, 100, (nb, hkv, BS, d), generator=g, device=DEV).to(kind) for _ in range(2)]
    scales = [torch.full((nb, hkv, BS, d // 64), 7.0, device=DEV) for _ in range(2)] if fp8 else [None, None]
    return k, v, slots, pools, scales


def write_expected(x, slots, pool, scale, fp8):
    pool = pool.clone()
    live = slots >= 0
    at = slots[live].long()
    rows = x[live]
    if not fp8:
        pool[at // BS, :, at % BS] = rows.contiguous().view(torch.int16)
        return pool, None
    scale = scale.clone()
    tiles = rows.double().reshape(*rows.shape[:2], -1, 64)
    amax = tiles.abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, 1.0).float()  # correctly rounded: 53 >= 2 * 24 + 2 bits
    codes = (tiles / sc.double()[..., None]).float().to(torch.float8_e4m3fn)
    pool[at // BS, :, at % BS] = codes.reshape(rows.shape).view(torch.uint8)
    scale[at // BS, :, at % BS] = sc
    return pool, scale


@pytest.mark.parametrize("t,hkv,d,fp8,fused,holes", [
    (1, 1, 8, False, False, ()), (1, 4, 64, True, True, ()), (5, 2, 128, False, True, (0, 3)),
    (57, 8, 128, True, False, (1, 2, 56)), (130, 3, 72, False, False, ()), (33, 5, 64, True, True, (7,)),
    (700, 8, 128, False, True, ()), (19, 1, 1024, False, False, ()), (40, 20, 128, True, False, ()),
    (3, 2, 64, False, False, (0, 1, 2)), (2000, 2, 192, True, True, (5,)),
])
def test_rows_land_in_their_slots(t, hkv, d, fp8, fused, holes):
    k, v, slots, pools, scales = write_case(t, hkv, d, fp8, fused, holes=holes)
    if fp8:  # a tile of zeros, one of a single large value, one of tiny ones
        k[0, 0, :64] = 0
        v[0, 0, :64] = 0
        v[0, 0, 5] = 3.0e38
        k[-1, -1, -64:] = 1.0e-38
    want = [write_expected(x, slots, p, s, fp8) for x, p, s in zip((k, v), pools, scales)]
    err = ints([0])
    views = [p if fp8 else p.view(torch.bfloat16) for p in pools]
    svpa.kv_write(k, v, slots, *views, error_flag=err, k_scale=scales[0], v_scale=scales[1],
                  scale_tile=64 if fp8 else 0)
    assert svpa.check_error(err) == 0
    for (p, s), got, sg in zip(want, pools, scales):
        assert torch.equal(got, p)
        assert s is None or torch.equal(sg, s)


def test_every_bf16_value_gets_the_code_of_its_quotient():
    """All bf16 magnitudes against tiles of many scales: codes at and near the
    ties of E4M3 included."""
    vals = torch.arange(0, 0x7F80, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for top in (1.0, 1.75, 448.0, 3.0e38, 2.0 ** -100, 1.0e-37, 2.0 ** -126):
        small = vals[vals <= torch.tensor(top, device=DEV).to(torch.bfloat16).float()]
        # the values a tile of this maximum tells apart, sampled over their whole range
        pick = small[(torch.rand(64 * 63 * 2, generator=g, device=DEV) ** 0.25 * small.numel()).long().clamp(max=small.numel() - 1)]
        x = torch.cat([pick.view(-1, 63), torch.full((128, 1), top, device=DEV)], 1).to(torch.bfloat16)
        x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.5, x, -x).view(64, 2, 64)
        slots = torch.arange(64, dtype=torch.int32, device=DEV)
        pools = [torch.zeros((4, 2, BS, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros((4, 2, BS, 1), device=DEV) for _ in range(2)]
        want = write_expected(x, slots, pools[0], scales[0], True)
        err = ints([0])
        svpa.kv_write(x, x, slots, *pools, error_flag=err, k_scale=scales[0], v_scale=scales[1], scale_tile=64)
        assert svpa.check_error(err) == 0
        for p, s in zip(pools, scales):
            assert torch.equal(p, want[0]) and torch.equal(s, want[1]), top


def test_the_scatter_matches_the_append():
    """The same rows written by kv_append (fresh pages) and through a slot map, FP8 tile scales."""
    wl = W.WORKLOADS["fp8_t64"].scaled(num_kv_heads=2, num_q_heads=8)
    inp = W.make_append(wl, 5, contexts=(0,), n_new=48, device=DEV)
    bt, kp, vp = inp.block_table.clone(), inp.k_pool.view(torch.uint8).clone(), inp.v_pool.view(torch.uint8).clone()
    ks, vs = inp.k_scale.clone(), inp.v_scale.clone()
    rc, fs, ft = inp.refcount.clone(), inp.free_stack.clone(), ints([inp.free_top])
    err = ints([0])
    svpa.kv_append(inp.new_k, inp.new_v, bt, inp.context_lens, rc, fs, ft, kp, vp, error_flag=err, k_scale=ks,
                   v_scale=vs, scale_tile=64)
    pos = torch.arange(48, device=DEV)
    slots = (bt[0, pos // BS] * BS + pos % BS).to(torch.int32)
    k2, v2 = torch.zeros_like(kp), torch.zeros_like(vp)
    s2 = [torch.zeros_like(ks), torch.zeros_like(vs)]
    svpa.kv_write(inp.new_k[0], inp.new_v[0], slots, k2, v2, error_flag=err, k_scale=s2[0], v_scale=s2[1], scale_tile=64)
    assert svpa.check_error(err) == 0
    used = bt[0, :3].long()
    for a, b in ((kp, k2), (vp, v2), (ks, s2[0]), (vs, s2[1])):
        assert torch.equal(a[used], b[used])


def test_a_slot_past_the_pool_raises_and_is_skipped():
    k, v, slots, pools, _ = write_case(20, 2, 64, False, False)
    slots[4] = pools[0].shape[0] * BS
    slots[9] = 2 ** 31 - 1
    before = slots.clone()
    want = [write_expected(x, torch.where(slots >= pools[0].shape[0] * BS, -1, slots), p, None, False)[0]
            for x, p in zip((k, v), pools)]
    err = ints([0])
    svpa.kv_write(k, v, slots, pools[0].view(torch.bfloat16), pools[1].view(torch.bfloat16), error_flag=err)
    assert svpa.STATUS[svpa.check_error(err)] == "SVPA_ERR_BAD_BLOCK"
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1]) and torch.equal(slots, before)


# ---------------------------------------------------------------- logits
class Logits:
    def __init__(self, b, rows, v, bf16=False, hist=50, bias=5, mask=True, parent=None, seed=0, history=True,
                 drafts=True, penalties=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = random.Random(seed)
        x = torch.randn((b, rows, v), generator=g, device=DEV) * 3
        self.x = x.to(torch.bfloat16) if bf16 else x
        self.b, self.rows, self.v, self.parent = b, rows, v, parent

        def tokens(*s):
            return (torch.rand(s, generator=g, device=DEV) ** 3 * v).clamp(max=v - 1).to(torch.int32)

        hl = [rng.randrange(0, hist + 1) for _ in range(b)]
        self.hist_lens, self.prompt_lens = ints(hl), ints([rng.randrange(0, n + 1) for n in hl])
        self.history = tokens(b, hist) if history else None
        n = rows if parent else rows - 1
        self.drafts = tokens(b, n) if drafts and n else None
        if self.drafts is not None and self.history is not None:  # a draft repeats the history, and another draft
            self.drafts[:, -1] = self.history[:, 0]
            if n > 2:
                self.drafts[:, 1] = self.drafts[:, -1]
        if parent and self.drafts is not None:
            self.drafts[:, 0] = -1000  # the root's entry is not read
        u = torch.rand((3, b), generator=g, device=DEV)
        self.pen = (1.0 + u[0], u[1], u[2]) if penalties else (None, None, None)
        self.bias = None
        if bias:
            counts = [rng.randrange(0, bias + 1) for _ in range(b)] if b > 1 else [bias]
            counts[0] = bias
            off = [sum(counts[:i]) for i in range(b + 1)]
            tok = tokens(off[-1])
            tok[bias - 1] = tok[0]  # named twice: the last entry holds
            if self.drafts is not None:
                tok[0] = tok[bias - 1] = self.drafts[0, -1]
            self.bias = (ints(off), tok, torch.randn(off[-1], generator=g, device=DEV))
        self.mask = None
        if mask:
            self.mask = torch.randint(-2 ** 31, 2 ** 31, (b, rows, -(-v // 32)), generator=g, device=DEV).to(torch.int32)
            self.mask[0, 0] = 0  # nothing allowed
        self.out = torch.full((b, rows, v), 1e30, device=DEV)
        self.err = ints([0])

    def call(self, out=None, stream=None):
        r, p, f = self.pen
        bo, bt, bv = self.bias or (None, None, None)
        svpa.logits_process(self.x, self.out if out is None else out, error_flag=self.err, history=self.history,
                            prompt_lens=self.prompt_lens, hist_lens=self.hist_lens, draft_tokens=self.drafts,
                            parent=self.parent, repetition=r, presence=p, frequency=f, bias_offsets=bo,
                            bias_tokens=bt, bias_values=bv, mask=self.mask, stream=stream)

    def expected(self):
        """64 bits, and the magnitude the bound is relative to."""
        x = self.x.double().clone()
        size = x.abs() * 2
        anc = W.ancestor_masks(self.parent or [i - 1 for i in range(self.rows)])
        for b in range(self.b):
            base, given = torch.zeros(self.v, device=DEV), torch.zeros(self.v, device=DEV)
            if self.history is not None:
                h, n, p = self.history[b].long(), int(self.hist_lens[b]), int(self.prompt_lens[b])
                base = torch.bincount(h[p:n], minlength=self.v)
                given = torch.bincount(h[:p], minlength=self.v)
            r, p, f = (torch.as_tensor(d if q is None else q[b], device=DEV).double()
                       for q, d in zip(self.pen, (1.0, 0.0, 0.0)))
            for j in range(self.rows):
                count = base.clone()
                if self.drafts is not None:
                    path = [i for i in range(1, self.rows) if anc[j] >> i & 1]
                    for i in path:
                        count[int(self.drafts[b, i if self.parent else i - 1])] += 1
                y = x[b, j]
                seen = (count > 0) | (given > 0)
                y = torch.where(seen, torch.where(y > 0, y / r, y * r), y)
                y = y - f * count - p * (count > 0)
                size[b, j] += f * count + p
                if self.bias:
                    off, tok, val = self.bias
                    for i in range(int(off[b]), int(off[b + 1])):
                        if not bool((tok[i + 1:int(off[b + 1])] == tok[i]).any()):
                            y[int(tok[i])] += val[i].double()
                            size[b, j, int(tok[i])] += val[i].double().abs()
                if self.mask is not None:
                    bits = (self.mask[b, j].long() & 0xFFFFFFFF)[:, None] >> torch.arange(32, device=DEV) & 1
                    y = torch.where(bits.reshape(-1)[:self.v] > 0, y, -torch.inf)
                x[b, j] = y
        return x, size

    def check(self, got=None):
        got = self.out if got is None else got
        assert svpa.check_error(self.err) == 0
        want, size = self.expected()
        assert torch.equal(torch.isneginf(got), torch.isneginf(want))
        ok = torch.isfinite(want)
        # five operations, each rounded once to fp32 (2^-24 of a value no larger than `size`)
        assert bool(((got.double() - want).abs()[ok] <= 5 * 2.0 ** -24 * size[ok]).all())


TREE = W.tree_parents((3, 2))


@pytest.mark.parametrize("kw", [
    dict(b=1, rows=1, v=1, hist=3, bias=1), dict(b=2, rows=3, v=31), dict(b=2, rows=5, v=4096),
    dict(b=1, rows=6, v=4097), dict(b=2, rows=4, v=50257, hist=900), dict(b=2, rows=4, v=50257, bf16=True),
    dict(b=2, rows=9, v=8200, bf16=True, hist=2000, bias=300), dict(b=2, rows=len(TREE), v=5000, parent=TREE),
    dict(b=1, rows=64, v=1000, parent=[i - 1 for i in range(64)]), dict(b=2, rows=64, v=1000, hist=5),
    dict(b=3, rows=4, v=9000, history=False), dict(b=3, rows=4, v=9000, drafts=False),
    dict(b=3, rows=4, v=9000, penalties=False), dict(b=3, rows=4, v=9000, bias=0, mask=False),
    dict(b=3, rows=4, v=9000, history=False, drafts=False, bias=0),
    dict(b=3, rows=4, v=9000, history=False, drafts=False, bias=0, mask=False, bf16=True),
    dict(b=20, rows=2, v=32000, hist=1),
])
def test_logits_against_64_bits(kw):
    c = Logits(**kw)
    c.call()
    c.check()


def test_logits_in_place_and_unaligned_rows():
    c = Logits(2, 5, 8192)
    keep = c.x.clone()
    c.call(out=c.x)
    got, c.x = c.x, keep
    c.check(got)
    for bf16 in (False, True):  # rows that start off any vector boundary
        d = Logits(2, 3, 8192, bf16=bf16, seed=4)
        wide = torch.zeros(d.x.numel() + 1, dtype=d.x.dtype, device=DEV)
        wide[1:] = d.x.reshape(-1)
        d.x = wide[1:].view(d.x.shape)
        d.call()
        d.check()


def test_special_logits_pass_through():
    """-inf stays, +inf and NaN of allowed tokens stay, masked ones become -inf."""
    c = Logits(1, 2, 4096, history=False, drafts=False, bias=0)
    c.x[0, :, :6] = torch.tensor([float("nan"), float("inf"), -float("inf")] * 2, device=DEV)
    c.mask[0] = -1
    c.mask[0, :, 0] = -1 ^ 0b111000
    c.call()
    assert svpa.check_error(c.err) == 0
    got = c.out[0, 1, :6].tolist()
    assert got[0] != got[0] and got[1:] == [float("inf")] + [-float("inf")] * 4


@pytest.mark.parametrize("what", ["history", "negative history", "length", "prompt", "drafts", "bias", "offsets"])
def test_bad_ids_and_lengths_raise(what):
    c = Logits(2, 4, 5000, hist=20)
    c.hist_lens.fill_(20)
    c.prompt_lens.fill_(5)
    if what == "history":
        c.history[1, 3] = 5000
    elif what == "negative history":
        c.history[1, 3] = -1
    elif what == "length":
        c.hist_lens[1] = 21
    elif what == "prompt":
        c.prompt_lens[1] = 21
    elif what == "drafts":
        c.drafts[0, 1] = 1 << 30
    elif what == "bias":
        c.bias[1][0] = -4
    else:
        c.bias[0][1] = -1
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_INVALID_ARG"

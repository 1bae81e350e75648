"""GPU tests of svpa_paged_prompt_attn: causal attention of packed prompts and
chunks over their pages, against 64 bits."""
import math

import pytest
import torch

import packed_ref as R
from speculative_verify_paged_attn_gb300 import svpa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Case:
    def __init__(self, new, cached, hq, hkv, d, seed=1, fused=False, pad=0, width=None, scale=None, spare=0):
        g = R.gen(seed, DEV)
        self.new, self.kv = list(new), [n + c for n, c in zip(new, cached)]
        self.hq, self.hkv, self.d = hq, hkv, d
        pages = [-(-n // R.BS) for n in self.kv]
        ids, pool = R.make_pool(pages, hkv, d, g, DEV)
        width = width or max(max(pages), 1)
        self.table = torch.full((len(new), width), -7, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(self.kv):
            mine = ids[at:at + pages[b]]
            at += pages[b]
            self.table[b, :pages[b]] = mine
            for x in range(2):  # valid tokens only; every other slot stays NaN
                rows = torch.randn((pages[b] * R.BS, hkv, d), generator=g, device=DEV).to(torch.bfloat16)
                rows[n:] = float("nan")
                pool[x, mine.long()] = rows.view(pages[b], R.BS, hkv, d).transpose(1, 2)
        self.k, self.v = pool[0], pool[1]
        self.t = sum(new) + pad
        wide = hq + (2 * hkv if fused else 0)
        self.q = torch.randn((self.t, wide, d), generator=g, device=DEV).to(torch.bfloat16)[:, :hq]
        self.cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(self.kv, dtype=torch.int32, device=DEV)
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.p = svpa.prompt_params(len(new), self.t, hq, hkv, d, width, self.k.shape[0], q_stride=self.q.stride(0),
                                    sm_scale=scale)
        self.ws = torch.zeros(svpa.paged_prompt_attn_workspace_size(self.p), dtype=torch.uint8, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.out = torch.full((self.t, hq, d), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.t, hq), 77.0, device=DEV)

    def call(self, stream=None, lse=True):
        svpa.paged_prompt_attn(self.p, self.q, self.k, self.v, self.table, self.cu, self.lens, self.out,
                               workspace=self.ws, error_flag=self.err, lse=self.lse if lse else None, stream=stream)

    def reference(self):
        firsts = self.cu.tolist()[:-1]
        limits = [[m - n + i + 1 for i in range(n)] for n, m in zip(self.new, self.kv)]
        return R.reference(self.q, self.k, self.v, self.table, firsts, self.new, self.kv, limits, self.hkv, self.scale)

    def check(self, what=""):
        assert svpa.check_error(self.err) == 0
        assert int(self.ws[:256].view(torch.int32).abs().sum()) == 0  # counters back at zero
        n = sum(self.new)
        out, lse, spread = self.reference()
        R.check(self.out[:n], self.lse[:n], (out[:n], lse[:n], spread[:n]), what)
        assert bool((self.out[n:] == 77.0).all()) and bool((self.lse[n:] == 77.0).all())


CASES = [
    # new tokens, cached tokens, Hq, Hkv, D
    ([1], [0], 4, 4, 64),
    ([1], [0], 8, 1, 128),
    ([37], [0], 4, 4, 64),
    ([16, 17, 15], [0, 0, 0], 8, 2, 128),
    ([128], [0], 2, 2, 128),
    ([129, 127], [0, 0], 2, 2, 64),
    ([256, 257, 1], [0, 0, 0], 2, 1, 128),
    ([300, 1, 0, 5, 700], [0, 0, 0, 0, 0], 4, 4, 128),
    ([0, 0, 33, 0], [0, 9, 4, 0], 4, 2, 64),
    ([90, 13], [0, 0], 14, 2, 128),          # a group of seven heads
    ([65, 200], [0, 0], 6, 2, 64),           # of three
    ([40, 3], [0, 0], 16, 1, 128),
    ([7, 2], [0, 0], 128, 1, 64),            # one token a tile
    ([5], [0], 80, 1, 128),                  # tiles of 80 rows
    ([1, 1, 1, 1, 1], [31, 32, 33, 0, 500], 8, 2, 128),   # single tokens behind a cache
    ([64, 1, 130], [100, 129, 1], 4, 1, 128),
    ([20], [5000], 8, 2, 128),               # a chunk behind a long cache: split over the kv range
    ([300], [3000], 2, 1, 64),               # pairs of tiles, split
    ([1], [9000], 4, 1, 128),
    ([130, 1], [1, 4000], 1, 1, 128),
    ([1500, 900], [0, 700], 8, 1, 128),
]


@pytest.mark.parametrize("new,cached,hq,hkv,d", CASES)
def test_against_64_bits(new, cached, hq, hkv, d):
    c = Case(new, cached, hq, hkv, d)
    c.call()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_sliced_queries_padding_rows_and_wide_tables(d):
    """q sliced out of a fused projection, rows behind the last sequence left
    as they were, table columns behind the last page ignored."""
    c = Case([33, 0, 70], [4, 0, 0], 8, 2, d, fused=True, pad=21, width=40)
    c.call()
    c.check()


def test_random_ragged_batches():
    import random
    rng = random.Random(3)
    for i in range(12):
        hkv, g = rng.choice([(1, 1), (2, 4), (1, 7), (3, 2), (1, 16)])
        n = rng.randrange(1, 9)
        new = [rng.choice([0, 1, rng.randrange(1, 400)]) for _ in range(n)]
        if sum(new) == 0:
            new[0] = 3
        cached = [rng.choice([0, rng.randrange(0, 300)]) for _ in range(n)]
        c = Case(new, cached, hkv * g, hkv, rng.choice([64, 128]), seed=i, fused=i % 2 == 0, pad=i % 3)
        c.call()
        c.check(f"{new} {cached} {hkv} {g}")


def test_mixed_units_repeated():
    """Pairs and single tiles in turn on every SM, the same bits every time."""
    new = [(131 * i) % 700 + 1 for i in range(60)]
    c = Case(new, [(577 * i) % 900 for i in range(60)], 16, 8, 128)
    c.call()
    c.check()
    first = c.out.clone()
    flush = torch.empty(64 << 20, device=DEV)
    for i in range(10):
        c.out.zero_()
        flush.fill_(float(i))
        c.call()
        assert torch.equal(c.out, first), i
    c.check()


def test_large_scores_and_growing_maxima():
    """Scores that grow along the sequence (the running maximum is replaced
    many times) and a sharp softmax."""
    c = Case([700], [0], 4, 2, 128, scale=0.25)
    ramp = torch.linspace(0.1, 1.5, 704, device=DEV)[:700]
    ids = c.table[0].long()
    k = c.k[ids].transpose(1, 2).reshape(-1, 2, 128)
    k[:700] = (k[:700].float() * ramp[:, None, None]).to(torch.bfloat16)
    c.k[ids] = k.view(-1, 16, 2, 128).transpose(1, 2)
    c.call()
    assert svpa.check_error(c.err) == 0
    out, lse, spread = c.reference()
    # sum |q k| * scale is up to 128 * E|q||k| * 1.5 * 0.25 < 64: twice the score error of the other cases
    err = (c.out.double() - out).abs()
    assert ((err / (R.out_bound(out, spread) + 4 * R.FP32 * spread)).max().item()) <= 1.0
    assert ((c.lse.double() - lse).abs() / (2 * R.lse_bound(lse))).max().item() <= 1.0


def test_the_same_call_twice_and_without_lse():
    c = Case([90, 260, 31], [0, 10, 700], 8, 2, 128)
    c.call()
    first, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    c.call(lse=False)
    assert torch.equal(c.out, first) and torch.equal(c.lse, lse)
    c.check()


def test_side_stream_and_captured_replay():
    c = Case([90, 260, 1], [0, 0, 2000], 4, 1, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    side.synchronize()
    c.check()
    eager = c.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    for _ in range(2):
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, eager)
    # new lengths in the same buffers: the plan holds for every length that fits the shapes
    c.new, c.kv = [200, 1, 150], [200, 77, 160]
    pages = [-(-n // 16) for n in c.kv]
    ids = torch.randperm(c.k.shape[0], device=DEV).to(torch.int32)
    c.k.copy_(torch.randn(c.k.shape, device=DEV))
    c.v.copy_(torch.randn(c.v.shape, device=DEV))
    at = 0
    for b, n in enumerate(pages):
        c.table[b, :n] = ids[at:at + n]
        at += n
    c.cu.copy_(torch.tensor([0, 200, 201, 351], dtype=torch.int32))
    c.lens.copy_(torch.tensor(c.kv, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check()


BAD = {
    "a length below the query tokens": lambda c: c.lens.__setitem__(1, 3),
    "a length past the table": lambda c: c.lens.__setitem__(1, 16 * c.table.shape[1] + 1),
    "a negative length": lambda c: c.lens.__setitem__(1, -5),
    "offsets past the rows": lambda c: c.cu.__setitem__(3, c.t + 40),
    "falling offsets": lambda c: c.cu.__setitem__(2, 1),
}


@pytest.mark.parametrize("what", sorted(BAD))
def test_bad_rows_raise_and_the_next_call_is_right(what):
    c = Case([40, 50, 60], [0, 0, 0], 4, 2, 64)
    keep = [c.cu.clone(), c.lens.clone()]
    BAD[what](c)
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_INVALID_ARG"
    c.cu.copy_(keep[0])
    c.lens.copy_(keep[1])
    c.err.zero_()
    c.call()
    c.check()


def test_bad_block_raises():
    c = Case([40, 50], [0, 0], 4, 2, 64)
    for bad in (-1, c.k.shape[0], 1 << 30):
        keep = int(c.table[1, 2])
        c.table[1, 2] = bad
        c.err.zero_()
        c.call()
        assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_BAD_BLOCK"
        c.table[1, 2] = keep
    c.err.zero_()
    c.call()
    c.check()


@pytest.mark.parametrize("new,cached,hq,hkv,cu", [
    # the falling row owns no tile: 0 -> 1000 -> 500 -> 1200 with 256 tokens a unit
    ([1000, 500, 700], [0, 0, 0], 2, 2, {1: 1000, 2: 500, 3: 1200}),
    # every length fits its (wrong) row
    ([600, 300, 600], [0, 0, 0], 8, 1, {1: 600, 2: 300, 3: 900}),
    # rows before the first sequence
    ([40, 20], [0, 0], 2, 2, {0: 5}),
    ([40, 20], [0, 0], 2, 2, {0: -5}),
    # more sequences than one round of loads finds
    ([300] * 50, [3000 if b == 20 else 0 for b in range(50)], 16, 2, {20: 3100}),
    ([300] * 50, [0] * 50, 16, 2, {49: -2 ** 31}),
    ([3] * 700, [0] * 700, 2, 2, {650: 40}),
])
def test_offsets_that_fall_or_start_late_raise(new, cached, hq, hkv, cu):
    c = Case(new, cached, hq, hkv, 64)
    keep = c.cu.clone()
    for i, v in cu.items():
        c.cu[i] = v
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_INVALID_ARG"
    c.cu.copy_(keep)
    c.err.zero_()
    c.out.fill_(77.0)
    c.call()
    c.check()


@pytest.mark.parametrize("new,cached,hq,hkv,d", [
    ([300, 1, 0, 5, 700], [0, 0, 0, 0, 0], 4, 4, 128), ([64, 1, 130], [100, 129, 1], 4, 1, 64), ([20], [5000], 8, 2, 128),
])
def test_outputs_on_a_16_byte_boundary(new, cached, hq, hkv, d):
    """Results stored in pieces of 16 bytes, not of 32."""
    c = Case(new, cached, hq, hkv, d, pad=2)
    wide = torch.full((c.out.numel() + 16,), 77.0, dtype=torch.bfloat16, device=DEV)
    c.out = wide[8:-8].view(c.out.shape)
    c.call()
    c.check()
    assert bool((wide[:8] == 77.0).all()) and bool((wide[-8:] == 77.0).all())


@pytest.mark.parametrize("new,cached,hq,hkv,d", [
    ([300, 40], [0, 0], 4, 4, 128),      # pairs of tiles
    ([37, 5], [0, 600], 8, 2, 64),       # single tiles
    ([20], [5000], 8, 2, 128), ([300], [3000], 2, 1, 64),  # split over the kv range
])
def test_a_nan_query_stays_in_its_row(new, cached, hq, hkv, d):
    """The row's result is NaN, not zeros; every other row is as it was."""
    c = Case(new, cached, hq, hkv, d)
    c.call()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    t, h = new[0] - 3, hq - 1
    c.q[t, h, 5] = float("nan")
    c.call()
    assert svpa.check_error(c.err) == 0
    assert bool(torch.isnan(c.out[t, h]).all()) and bool(torch.isnan(c.lse[t, h]))
    c.out[t, h], c.lse[t, h] = out[t, h], lse[t, h]
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)

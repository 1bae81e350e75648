"""GPU tests of svpa_prefix_verify_attn: verification attention of a batch that
shares a prefix, against 64 bits and against svpa_paged_verify_attn."""
import math

import pytest
import torch

import packed_ref as R
from speculative_verify_paged_attn_gb300 import svpa
from speculative_verify_paged_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Case:
    def __init__(self, own, prefix, n_q, hq, hkv, d, seed=1, masks=None, loners=(), width=None):
        """own: each sequence's committed tokens behind the prefix; loners:
        sequences that hold a copy of their own instead of the shared blocks."""
        g = R.gen(seed, DEV)
        self.n_q, self.hq, self.hkv, self.d, self.prefix = n_q, hq, hkv, d, prefix
        self.b, self.masks = len(own), masks
        shared = prefix // R.BS
        self.ctx = [prefix + n for n in own]
        pages = [-(-(n + n_q) // R.BS) for n in self.ctx]
        ids, pool = R.make_pool([shared] + pages, hkv, d, g, DEV)
        width = width or max(pages)
        self.table = torch.full((self.b, width), -9, dtype=torch.int32, device=DEV)
        self.blocks = ids[:shared].clone()

        def rows(n):
            return torch.randn((2, n, hkv, R.BS, d), generator=g, device=DEV).to(torch.bfloat16)

        pool[:, self.blocks.long()] = rows(shared)
        at = shared
        for b in range(self.b):
            first = 0 if b in loners else shared
            mine = ids[at:at + pages[b] - first]
            at += pages[b] - first
            self.table[b, :first] = self.blocks[:first]
            self.table[b, first:pages[b]] = mine
            fresh = rows(pages[b] - first)
            tail = self.ctx[b] + n_q - (pages[b] - 1) * R.BS  # slots behind the last draft stay NaN
            if pages[b] > first:
                fresh[:, -1, :, tail:] = float("nan")
            pool[:, mine.long()] = fresh
        self.k, self.v = pool[0], pool[1]
        self.q = torch.randn((self.b, n_q, hq, d), generator=g, device=DEV).to(torch.bfloat16)
        self.lens = torch.tensor(self.ctx, dtype=torch.int32, device=DEV)
        self.p = svpa.attn_params(self.b, n_q, hq, hkv, d, width, self.k.shape[0])
        self.ws = torch.zeros(svpa.prefix_verify_attn_workspace_size(self.p, prefix), dtype=torch.uint8, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.out = torch.full((self.b, n_q, hq, d), 5.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.b, n_q, hq), 5.0, device=DEV)

    def call(self, stream=None, lse=True):
        svpa.prefix_verify_attn(self.p, self.q, self.k, self.v, self.blocks if self.prefix else None, self.table,
                                self.lens, self.out, workspace=self.ws, error_flag=self.err,
                                ancestor_mask=self.masks, lse=self.lse if lse else None, stream=stream)

    def reference(self):
        n = self.n_q
        masks = self.masks or [(1 << (j + 1)) - 1 for j in range(n)]
        bits = torch.tensor([[m >> i & 1 for i in range(n)] for m in masks], dtype=torch.bool, device=DEV)
        extra = [torch.cat([bits.new_zeros((n, c)), bits], 1) for c in self.ctx]
        return R.reference(self.q.view(-1, self.hq, self.d), self.k, self.v, self.table,
                           [b * n for b in range(self.b)], [n] * self.b, [c + n for c in self.ctx],
                           [[c] * n for c in self.ctx], self.hkv, 1 / math.sqrt(self.d), extra)

    def check(self, what=""):
        assert svpa.check_error(self.err) == 0
        assert int(self.ws[:256].view(torch.int32).abs().sum()) == 0
        R.check(self.out.view(-1, self.hq, self.d), self.lse.view(-1, self.hq), self.reference(), what)


TREE = W.ancestor_masks(W.tree_parents((4, 2, 2)))

CASES = [
    # own tokens, prefix, n_q, Hq, Hkv, D
    ([3], 16, 1, 4, 4, 64),
    ([0, 5, 90], 32, 1, 8, 2, 128),
    ([0, 0], 128, 5, 4, 4, 128),                 # nothing of their own but the drafts
    ([100, 17, 260, 1], 800, 6, 16, 2, 128),
    ([40] * 9, 272, 3, 14, 2, 128),              # seven heads a group
    ([40, 1, 130], 144, 64, 2, 1, 64),           # 64 queries
    ([10, 700, 128, 127, 129], 2048, 4, 8, 8, 64),
    ([5, 6], 4096, 2, 64, 1, 128),
    ([3000, 10], 512, 2, 8, 1, 128),             # own parts split over idle SMs
    ([1500], 1024, 8, 4, 1, 64),
    ([70, 20, 0], 0, 4, 4, 2, 128),              # no prefix
    ([33, 12] * 20, 480, 5, 8, 4, 128),
]


@pytest.mark.parametrize("own,prefix,n_q,hq,hkv,d", CASES)
def test_against_64_bits(own, prefix, n_q, hq, hkv, d):
    c = Case(own, prefix, n_q, hq, hkv, d)
    c.call()
    c.check()


@pytest.mark.parametrize("own", [[30, 200, 77], [2500, 3]])
def test_draft_tree(own):
    c = Case(own, 320, len(TREE), 8, 2, 128, masks=TREE)
    c.call()
    c.check()


@pytest.mark.parametrize("own,hkv", [([30, 200, 77, 5] * 50, 4), ([900, 30, 77], 1), ([3000, 2500, 77], 1)])
def test_sequences_without_the_prefix(own, hkv):
    """Rows whose table does not begin with the shared blocks, and rows shorter
    than the prefix, attend their own history: the result is that of
    paged_verify_attn whatever prefix is named."""
    c = Case(own, 256, 4, 4 * hkv, hkv, 128, loners=(1,))
    # a third one holds all shared blocks but the last
    c.lens[2] = 250 - 16
    c.ctx[2] = 250 - 16
    c.call()
    c.check()
    assert svpa.check_error(c.err) == 0
    ws = torch.zeros(svpa.attn_workspace_size(c.p), dtype=torch.uint8, device=DEV)
    other = torch.empty_like(c.out)
    svpa.paged_verify_attn(c.p, c.q, c.k, c.v, c.table, c.lens, other, workspace=ws, error_flag=c.err)
    assert svpa.check_error(c.err) == 0
    # both within their bound of the same value
    ref, _, spread = c.reference()
    gap = (c.out.double() - other.double()).abs().view(ref.shape)
    assert bool((gap <= 2 * R.out_bound(ref, spread)).all())


def test_many_sequences_and_repeated_calls():
    c = Case([(37 * i) % 300 for i in range(96)], 512, 6, 16, 2, 128)
    c.call()
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.out.zero_()
        c.call()
    assert torch.equal(c.out, first)


def test_streams_of_own_blocks_behind_a_tree():
    """More units than SMs, streamed from memory, odd numbers of blocks: the
    ring's slots pass between the two tiles in every order."""
    c = Case([200 + (997 * i) % 2500 for i in range(64)], 800, len(TREE), 32, 8, 128, masks=TREE)
    c.call()
    c.check()
    first, lse = c.out.clone(), c.lse.clone()
    flush = torch.empty(64 << 20, device=DEV)
    for i in range(12):
        c.out.zero_()
        c.lse.zero_()
        if i % 2:
            flush.fill_(float(i))
        c.call()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse), i
    c.check()


def test_captured_replay_with_new_lengths():
    c = Case([90, 26, 140, 3], 256, 4, 8, 2, 128)
    c.call()
    c.check()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    c.ctx = [256 + n for n in (80, 26, 9, 3)]
    c.lens.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_bad_inputs_raise_and_the_next_call_is_right():
    c = Case([90, 26, 140], 256, 4, 8, 2, 128)
    keep = c.lens.clone()
    for bad in (-1, 16 * c.table.shape[1] - 3):
        c.lens[1] = bad
        c.err.zero_()
        c.call()
        assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_INVALID_ARG"
    c.lens.copy_(keep)
    for spot in (0, 17):  # in the prefix of one row (which then stands alone), and behind it
        was = int(c.table[2, spot])
        c.table[2, spot] = c.k.shape[0]
        c.err.zero_()
        c.call()
        assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_BAD_BLOCK"
        c.table[2, spot] = was
    was = int(c.blocks[3])
    c.blocks[3] = -2
    c.err.zero_()
    c.call()
    assert svpa.STATUS[svpa.check_error(c.err)] == "SVPA_ERR_BAD_BLOCK"
    c.blocks[3] = was
    c.err.zero_()
    c.call()
    c.check()


@pytest.mark.parametrize("own,prefix,n_q,hq,hkv,loners", [
    ([200, 33], 4096, 1, 32, 32, ()), ([100 + 29 * i for i in range(8)], 2048, 1, 32, 32, (3,)),
    ([300, 7, 64, 1000, 0, 450], 3200, 5, 16, 8, (0, 5)),
])
def test_few_ctas_wait_for_a_long_prefix(own, prefix, n_q, hq, hkv, loners):
    """CTAs without a prefix unit wait most of the call: what they hold back, and
    what the others take, does not change the result."""
    c = Case(own, prefix, n_q, hq, hkv, 128, loners=loners)
    c.call()
    c.check()
    first, lse = c.out.clone(), c.lse.clone()
    flush = torch.empty(64 << 20, device=DEV)
    for i in range(6):
        c.out.zero_()
        c.lse.zero_()
        if i % 2:
            flush.fill_(float(i))
        c.call()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse), i
    c.check()


def test_two_calls_at_once_with_their_own_workspaces():
    cases = [Case([90, 260, 140, 33] * 5, 1024, 4, 16, 4, 128, seed=3), Case([12, 700], 4096, 1, 16, 16, 128, seed=4)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.call()
        c.check()
    want = [c.out.clone() for c in cases]
    torch.cuda.synchronize()
    for _ in range(8):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.out.zero_()
                c.call(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        c.check()
        assert torch.equal(c.out, w)


@pytest.mark.parametrize("own,prefix,n_q,hq,hkv", [
    ([100, 17, 260, 1], 800, 6, 16, 2), ([70, 20, 0], 16, 4, 4, 2), ([33, 12] * 20, 480, 5, 8, 4),
])
def test_outputs_on_a_16_byte_boundary(own, prefix, n_q, hq, hkv):
    """Results stored in pieces of 16 bytes, not of 32."""
    c = Case(own, prefix, n_q, hq, hkv, 128)
    wide = torch.full((c.out.numel() + 16,), 5.0, dtype=torch.bfloat16, device=DEV)
    c.out = wide[8:-8].view(c.out.shape)
    c.call()
    c.check()
    assert bool((wide[:8] == 5.0).all()) and bool((wide[-8:] == 5.0).all())


@pytest.mark.parametrize("own,prefix,n_q,hq,hkv", [
    ([100, 17, 260, 1], 800, 6, 16, 2), ([33, 12] * 40, 480, 5, 16, 4), ([3000, 10], 512, 2, 8, 1),
])
def test_a_nan_query_stays_in_its_row(own, prefix, n_q, hq, hkv):
    """Behind a shared prefix, joined at once or from split parts: the row's
    result is NaN, every other row is as it was."""
    c = Case(own, prefix, n_q, hq, hkv, 128)
    c.call()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    c.q[1, n_q - 1, 3, 7] = float("nan")
    c.call()
    assert svpa.check_error(c.err) == 0
    spot = (1, n_q - 1, 3)
    assert bool(torch.isnan(c.out[spot]).all()) and bool(torch.isnan(c.lse[spot]))
    c.out[spot], c.lse[spot] = out[spot], lse[spot]
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)

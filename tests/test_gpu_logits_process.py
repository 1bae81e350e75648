"""GPU tests of svpa_logits_process at the sizes of full batches (every kernel
that the launch chooses among), with long histories and long bias lists."""
import math
import random

import pytest
import torch

from speculative_verify_paged_attn_gb300 import svpa
from speculative_verify_paged_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Case:
    """Everything present; `biases`: entries of each sequence's list, drawn from
    the vocabulary's first `span` tokens (repeated ones among them)."""

    def __init__(self, b, rows, v, bf16=False, hist=50, biases=5, span=None, parent=None, seed=0, masked=True):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = random.Random(seed)
        self.b, self.rows, self.v, self.parent = b, rows, v, parent
        x = torch.randn((b, rows, v), generator=g, device=DEV) * 3
        self.x = x.to(torch.bfloat16) if bf16 else x

        def ints(t):
            return torch.as_tensor(t, dtype=torch.int32, device=DEV)

        def tokens(shape, below=v):  # low ids are the common ones
            return (torch.rand(shape, generator=g, device=DEV) ** 3 * below).clamp(max=below - 1).to(torch.int32)

        n = [hist if i == 0 else rng.randrange(0, hist + 1) for i in range(b)]
        self.hist_lens, self.prompt_lens = ints(n), ints([rng.randrange(0, m + 1) for m in n])
        self.history = tokens((b, hist))
        self.drafts = tokens((b, rows if parent else rows - 1)) if rows > 1 or parent else None
        if self.drafts is not None and hist:
            self.drafts[:, -1] = self.history[:, 0]
        u = torch.rand((3, b), generator=g, device=DEV)
        self.rep, self.pres, self.freq = 1.0 + u[0], u[1].clone(), u[2].clone()
        counts = [biases if i == 0 else rng.randrange(0, biases + 1) for i in range(b)]
        self.offsets = ints([sum(counts[:i]) for i in range(b + 1)])
        self.tok = tokens((sum(counts),), span or v)
        self.val = torch.randn(sum(counts), generator=g, device=DEV)
        self.mask = None
        if masked:
            self.mask = torch.randint(-2 ** 31, 2 ** 31, (b, rows, -(-v // 32)), generator=g, device=DEV).to(torch.int32)
            self.mask[0, 0] = 0  # nothing allowed
        self.out = torch.full((b, rows, v), 1e30, device=DEV)
        self.err = ints([0])

    def call(self, out=None):
        svpa.logits_process(self.x, self.out if out is None else out, error_flag=self.err, history=self.history,
                            prompt_lens=self.prompt_lens, hist_lens=self.hist_lens, draft_tokens=self.drafts,
                            parent=self.parent, repetition=self.rep, presence=self.pres, frequency=self.freq,
                            bias_offsets=self.offsets, bias_tokens=self.tok, bias_values=self.val, mask=self.mask)

    def expected(self, j):
        """Row j of every sequence in 64 bits, and the magnitude its bound is relative to."""
        b, v = self.b, self.v
        pos = torch.arange(self.history.shape[1], device=DEV)
        new = (pos >= self.prompt_lens[:, None]) & (pos < self.hist_lens[:, None])
        count = torch.zeros((b, v), dtype=torch.float64, device=DEV)
        given = torch.zeros((b, v), dtype=torch.float64, device=DEV)
        count.scatter_add_(1, self.history.long(), new.double())
        given.scatter_add_(1, self.history.long(), (pos < self.prompt_lens[:, None]).double())
        anc = W.ancestor_masks(self.parent or [i - 1 for i in range(self.rows)])
        for i in range(1, self.rows):
            if anc[j] >> i & 1:
                count.scatter_add_(1, self.drafts[:, i if self.parent else i - 1, None].long(),
                                   torch.ones((b, 1), dtype=torch.float64, device=DEV))
        entries = self.tok.numel()
        row = torch.repeat_interleave(torch.arange(b, device=DEV), self.offsets.diff().long(), output_size=entries)
        last = torch.full((b * v,), -1, dtype=torch.int64, device=DEV)
        last.scatter_reduce_(0, row * v + self.tok.long(), torch.arange(entries, device=DEV), "amax")
        bias = torch.where(last >= 0, self.val.double()[last.clamp(min=0)] if entries else 0.0, 0.0).view(b, v)
        rep, pres, freq = (t.double()[:, None] for t in (self.rep, self.pres, self.freq))
        y = self.x[:, j].double()
        size = 2 * y.abs() + freq * count + pres + bias.abs()
        y = torch.where((count > 0) | (given > 0), torch.where(y > 0, y / rep, y * rep), y)
        y = y - freq * count - pres * (count > 0) + bias
        if self.mask is not None:
            bits = self.mask[:, j, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32) & 1
            y = torch.where(bits.view(b, -1)[:, :v] != 0, y, -math.inf)
        return y, size

    def check(self, got=None):
        got = self.out if got is None else got
        assert svpa.check_error(self.err) == 0
        for j in range(self.rows):
            want, size = self.expected(j)
            mine = got[:, j].double()
            finite = torch.isfinite(want)
            assert torch.equal(torch.isnan(mine), torch.isnan(want)), j
            assert torch.equal(mine.nan_to_num(0.0, 1.0, -1.0)[~finite], want.nan_to_num(0.0, 1.0, -1.0)[~finite]), j
            # five operations, each rounded once to fp32 (2^-24 of a value no larger than `size`)
            assert bool(((mine - want).abs()[finite] <= 5 * 2.0 ** -24 * size[finite]).all()), j


# vocabulary and batch of the three slabs: a row a CTA, 2048 tokens, 4096 tokens
SMALL, MIDDLE, LARGE = dict(b=3, v=50257), dict(b=10, v=128256), dict(b=30, v=128256)


@pytest.mark.parametrize("size", [SMALL, MIDDLE, LARGE], ids=["small", "middle", "large"])
@pytest.mark.parametrize("biases,span", [(700, 600), (3000, 4096), (5000, None)])
def test_more_biased_tokens_than_a_slab_lists(size, biases, span):
    c = Case(rows=2, biases=biases, span=span, hist=300, bf16=biases == 3000, **size)
    c.call()
    c.check()


def test_a_bias_for_every_token():
    """One list that names the whole vocabulary twice: the second half holds."""
    c = Case(2, 3, 128256, biases=1)
    order = torch.cat([torch.randperm(c.v, device=DEV) for _ in range(2)]).to(torch.int32)
    c.tok = torch.cat([order, order.new_zeros(1)])
    c.val = torch.randn(2 * c.v + 1, device=DEV)
    c.offsets = torch.tensor([0, 2 * c.v, 2 * c.v + 1], dtype=torch.int32, device=DEV)
    c.call()
    c.check()


TREE = W.tree_parents((3, 2))

# the batch of each slab's smallest call, to the sequence, and odd vocabularies
@pytest.mark.parametrize("kw", [
    dict(b=25, rows=3, v=50257), dict(b=25, rows=3, v=50257, bf16=True), dict(b=24, rows=3, v=50257),
    dict(b=75, rows=2, v=50257, bf16=True), dict(b=75, rows=3, v=50257), dict(b=74, rows=2, v=50257),
    dict(b=10, rows=4, v=128256), dict(b=30, rows=3, v=128256, bf16=True), dict(b=30, rows=2, v=128255),
    dict(b=30, rows=len(TREE), v=128256, parent=TREE), dict(b=75, rows=len(TREE), v=50257, parent=TREE, bf16=True),
    dict(b=75, rows=1, v=50257), dict(b=30, rows=3, v=128256, masked=False, biases=0),
    dict(b=75, rows=2, v=50257, hist=5001), dict(b=30, rows=2, v=128256, hist=9000, bf16=True),
    dict(b=10, rows=2, v=128256, hist=4096), dict(b=25, rows=2, v=50257, hist=8191), dict(b=2, rows=3, v=32000, hist=6001),
    dict(b=3, rows=2, v=50257, hist=2048), dict(b=25, rows=64, v=50257, hist=30),
], ids=lambda k: "-".join(str(k[x]) for x in ("b", "rows", "v")) + ("-bf16" if k.get("bf16") else ""))
def test_full_batches_against_64_bits(kw):
    c = Case(**kw)
    c.call()
    c.check()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("b,v", [(25, 50257), (75, 50257), (30, 128256)])
def test_full_batches_off_every_vector_boundary(b, v, bf16):
    c = Case(b, 2, v, bf16=bf16, hist=700)
    wide = torch.zeros(c.x.numel() + 1, dtype=c.x.dtype, device=DEV)
    wide[1:] = c.x.reshape(-1)
    c.x = wide[1:].view(c.x.shape)
    out = torch.full((c.out.numel() + 1,), 5.0, device=DEV)
    c.call(out=out[1:].view(c.out.shape))
    c.check(out[1:].view(c.out.shape))
    assert float(out[0]) == 5.0


@pytest.mark.parametrize("b,v", [(25, 50257), (30, 128256)])
def test_full_batches_in_place(b, v):
    c = Case(b, 3, v, hist=5000)
    keep = c.x.clone()
    c.call(out=c.x)
    got, c.x = c.x, keep
    c.check(got)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("b,v", [(2, 5000), (25, 50257), (30, 128256)])
def test_special_logits_of_marked_tokens(b, v, bf16):
    """NaN and infinities among prompt, generated, drafted and biased tokens, in
    allowed and masked places."""
    c = Case(b, 4, v, bf16=bf16, hist=400, biases=400, span=3000)
    low = c.x[:, :, :3000]
    pick = torch.arange(3000, device=DEV) % 7
    for k, value in enumerate((math.nan, math.inf, -math.inf)):
        low[:, :, pick == k] = value
    c.call()
    c.check()


def test_the_same_bits_every_time():
    """Marks are listed in any order and counted by atomics: the result is the same."""
    c = Case(30, 3, 128256, hist=9000, biases=300, span=4096, bf16=True)
    c.call()
    c.check()
    first = c.out.clone()
    for _ in range(4):
        c.out.zero_()
        c.call()
        assert torch.equal(c.out, first)

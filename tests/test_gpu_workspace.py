"""One zero-filled buffer as the workspace of several attention calls in turn:
shared and unshared prefixes, prompts and plain verification, whatever their
batch, draft length and prefix."""
import pytest
import torch

import gpu_util as G
import test_gpu_prefix as P
import test_gpu_prompt as Q
from speculative_verify_paged_attn_gb300 import svpa
from speculative_verify_paged_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HEAD = 256 + 65536  # counters and split tickets: zero again after every completed call


class Alone(P.Case):
    """svpa_paged_verify_attn on the same inputs."""

    def __init__(self, *args, split_pages=0, **kw):
        super().__init__(*args, **kw)
        self.p.split_pages = split_pages
        self.ws = torch.zeros(svpa.attn_workspace_size(self.p), dtype=torch.uint8, device=DEV)

    def call(self, stream=None, lse=True):
        svpa.paged_verify_attn(self.p, self.q, self.k, self.v, self.table, self.lens, self.out, workspace=self.ws,
                               error_flag=self.err, ancestor_mask=self.masks, lse=self.lse if lse else None,
                               stream=stream)


CALLS = {
    # shared, the own parts split (a flag a sequence in the workspace); partials behind it
    "shared, split": lambda: P.Case([8500, 30, 4000, 7], 1024, 5, 8, 2, 128, width=600),
    # the same call but for its prefix: read by every sequence, histories split
    "unshared, split": lambda: P.Case([9000, 30, 4000, 7], 16, 5, 8, 2, 128, width=600),
    # shared, the sequences ranked by length
    "shared, ranked": lambda: P.Case([(37 * i) % 300 for i in range(40)], 512, 6, 64, 8, 128, width=600),
    # a larger batch that splits
    "unshared, batch 40": lambda: P.Case([(97 * i) % 2500 for i in range(40)], 0, 6, 64, 8, 128, width=600),
    "unshared, single tokens": lambda: P.Case([(57 * i) % 3000 for i in range(24)], 0, 1, 8, 2, 64, width=600),
    "verify, batch 9": lambda: Alone([6000, 30, 4000, 7, 900, 1, 2000, 3000, 64], 0, 5, 8, 2, 128, width=600),
    "prompt chunks, split": lambda: Q.Case([130, 1, 40], [1, 4000, 6000], 8, 2, 128),
}


@pytest.mark.parametrize("second", sorted(CALLS))
@pytest.mark.parametrize("first", sorted(CALLS))
def test_one_workspace_for_calls_in_turn(first, second):
    a, b = CALLS[first](), CALLS[second]()
    ws = torch.zeros(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device=DEV)
    a.ws = b.ws = ws
    for i in range(2):
        for name, c in ((first, a), (second, b)):
            c.out.fill_(77.0)
            c.lse.fill_(77.0)
            c.call()
            c.check(f"{name}, round {i}")
    assert int(ws[:HEAD].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("make", [
    lambda: Alone([(7 * i) % 50 for i in range(4200)], 0, 1, 16, 4, 128, split_pages=1),
    lambda: P.Case([(7 * i) % 50 for i in range(4200)], 0, 1, 16, 4, 128),
])
def test_more_tickets_than_the_workspace_keeps(make):
    """16800 (sequence, kv head) pairs: their tickets reach past the part that
    every call leaves at zero, where an earlier call's partials may stand."""
    c = make()
    c.p.split_pages = 1
    c.ws = torch.zeros(svpa.attn_workspace_size(c.p), dtype=torch.uint8, device=DEV)
    c.call()
    assert svpa.check_error(c.err) == 0
    out, lse = c.out.clone(), c.lse.clone()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for _ in range(2):
        c.ws[HEAD:] = 0x11
        c.out.zero_()
        c.lse.zero_()
        c.call()
        assert svpa.check_error(c.err) == 0
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
        assert int(c.ws[:HEAD].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("name", ["fp8", "fp8_t64"])
def test_fp8_pages_on_the_same_workspace(name):
    """FP8 pages, whose blocks are split over all SMs, between calls of the other kinds."""
    wl = W.WORKLOADS[name].scaled(num_q_heads=16, num_kv_heads=2)
    inp = G.to_dev(W.make_attention(wl, 3, contexts=(3000, 17, 900, 5000)))
    b, n_q, hq, d = inp.q.shape
    p = svpa.attn_params(b, n_q, hq, 2, d, inp.block_table.shape[1], inp.num_blocks, kv_fp8=True,
                         sm_scale=wl.sm_scale, scale_tile=wl.scale_tile)
    out, err = torch.zeros((b, n_q, hq, d), dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(ws):
        out.zero_()
        svpa.paged_verify_attn(p, inp.q, inp.k_pool.view(torch.uint8), inp.v_pool.view(torch.uint8), inp.block_table,
                               inp.context_lens, out, workspace=ws, error_flag=err, k_scale=inp.k_scale,
                               v_scale=inp.v_scale, ancestor_mask=G.mask_list(inp))
        assert svpa.check_error(err) == 0
        return out.clone()

    size = svpa.attn_workspace_size(p)
    want = call(torch.zeros(size, dtype=torch.uint8, device=DEV))
    others = [CALLS[k]() for k in ("shared, split", "unshared, split", "prompt chunks, split")]
    ws = torch.zeros(max([size] + [c.ws.numel() for c in others]), dtype=torch.uint8, device=DEV)
    for c in others:
        c.ws = ws
        c.call()
        c.check()
        assert torch.equal(call(ws), want)
        c.call()
        c.check()
    assert int(ws[:HEAD].view(torch.int32).abs().sum()) == 0

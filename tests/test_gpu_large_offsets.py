"""Pools and logits of more than 2^31 elements: the same results as in small ones."""
import pytest
import torch

import test_gpu_prefix as P
import test_gpu_prompt as Q
import test_gpu_logits_process as L
from speculative_verify_paged_attn_gb300 import svpa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FAR = 140000  # pages of 8 x 16 x 128 values: 2.3e9 elements before the first one used


def moved(pool, at):
    big = torch.empty((at + pool.shape[0],) + pool.shape[1:], dtype=pool.dtype, device=DEV)
    big[at:] = pool
    return big


@pytest.mark.parametrize("new,cached", [([300, 1, 700], [0, 900, 40]), ([20], [5000])])
def test_prompts_at_the_end_of_a_large_pool(new, cached):
    c = Q.Case(new, cached, 16, 8, 128)
    c.call()
    out, lse = c.out.clone(), c.lse.clone()
    c.k, c.v = moved(c.k, FAR), moved(c.v, FAR)
    c.table += FAR
    c.p.num_blocks += FAR
    c.out.zero_()
    c.call()
    assert svpa.check_error(c.err) == 0
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("own,prefix,n_q", [([100, 17, 260, 1], 800, 6), ([33, 12] * 20, 480, 5), ([3000, 10], 512, 2),
                                            ([900, 30], 16, 5)])
def test_prefixes_at_the_end_of_a_large_pool(own, prefix, n_q):
    c = P.Case(own, prefix, n_q, 16, 8, 128)
    c.call()
    out, lse = c.out.clone(), c.lse.clone()
    c.k, c.v = moved(c.k, FAR), moved(c.v, FAR)
    c.table += FAR
    c.blocks += FAR
    c.p.num_blocks += FAR
    c.out.zero_()
    c.call()
    assert svpa.check_error(c.err) == 0
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_scattered_to_the_end_of_a_large_pool(fp8):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    t = 333
    k, v = (torch.randn((t, 8, 128), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    slots = torch.randperm(30 * 16, generator=g, device=DEV)[:t].to(torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    results = []
    for at in (0, FAR * (2 if fp8 else 1)):  # (bytes, and scales, past 2^32)
        pools = [torch.empty((at + 30, 8, 16, 128), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
                 for _ in range(2)]
        scales = [torch.empty((at + 30, 8, 16, 2), device=DEV) for _ in range(2)] if fp8 else [None, None]
        for x in pools + scales:
            if x is not None:
                x[at:] = 0
        svpa.kv_write(k, v, slots + at * 16, *pools, error_flag=err, k_scale=scales[0], v_scale=scales[1],
                      scale_tile=64 if fp8 else 0)
        assert svpa.check_error(err) == 0
        results.append([x[at:].clone() for x in pools + scales if x is not None])
        del pools, scales
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bf16", [False, True])
def test_logits_past_2_31_elements(bf16):
    """300 sequences of 60 rows: the last one's rows as of a call of its own."""
    b, rows, v = 300, 60, 128255
    small = L.Case(1, rows, v, bf16=bf16, hist=500)
    small.call()
    small.check()
    x = torch.zeros((b, rows, v), dtype=small.x.dtype, device=DEV)
    x[-1] = small.x[0]
    out = torch.empty((b, rows, v), device=DEV)

    def last(t):
        full = torch.zeros((b,) + t.shape[1:], dtype=t.dtype, device=DEV)
        full[-1] = t[0]
        return full

    offsets = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    offsets[-1] = small.tok.numel()
    svpa.logits_process(x, out, error_flag=small.err, history=last(small.history), prompt_lens=last(small.prompt_lens),
                        hist_lens=last(small.hist_lens), draft_tokens=last(small.drafts), repetition=last(small.rep),
                        presence=last(small.pres), frequency=last(small.freq), bias_offsets=offsets,
                        bias_tokens=small.tok, bias_values=small.val, mask=last(small.mask))
    assert svpa.check_error(small.err) == 0
    assert torch.equal(out[-1], small.out[0])
    assert bool(torch.isneginf(out[:-1:37]).all())  # their masks allow nothing

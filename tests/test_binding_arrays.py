"""The binding refuses arrays that the library would misread (CPU only: nothing
is launched)."""
import pytest
import torch

from speculative_verify_paged_attn_gb300 import svpa


@pytest.fixture(scope="module", autouse=True)
def lib():
    from speculative_verify_paged_attn_gb300 import build
    build.build()
    svpa.load()


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


BF, F32 = torch.bfloat16, torch.float32


def refused(call, good, **bad):
    args = dict(good, **bad)
    with pytest.raises(svpa.SvpaError) as e:
        call(**args, stream=0)
    assert e.value.status == 1


@pytest.mark.parametrize("bad", [
    dict(logits=z(2, 3, 100, dtype=torch.float16)), dict(logits=z(2, 3, 100, dtype=torch.float64)),
    dict(logits=z(2, 3, 128, dtype=F32)[:, :, :100]),       # out of a padded vocabulary
    dict(logits=z(2, 4, 100, dtype=BF)[:, 1:]), dict(logits=z(2, 100, 3, dtype=F32).transpose(1, 2)),
    dict(out=z(2, 3, 100, dtype=BF)), dict(out=z(2, 3, 128, dtype=F32)[:, :, :100]), dict(out=z(2, 3, 99, dtype=F32)),
    dict(history=z(2, 20, dtype=torch.int64)), dict(history=z(2, 30)[:, :20]), dict(history=z(1, 20)),
    dict(draft_tokens=z(2, 1)), dict(draft_tokens=z(2, 3)[:, 1:]), dict(draft_tokens=z(2, 2, dtype=torch.int64)),
    dict(draft_tokens=z(2, 2), parent=[-1, 0, 0]),          # a tree has an entry a row
    dict(mask=z(2, 3, 3)), dict(mask=z(2, 3, 8)[:, :, :4]), dict(mask=z(2, 3, 4, dtype=torch.bool)),
])
def test_logits(bad):
    good = dict(logits=z(2, 3, 100, dtype=F32), out=z(2, 3, 100, dtype=F32), error_flag=z(1), history=z(2, 20),
                hist_lens=z(2), draft_tokens=z(2, 2), mask=z(2, 3, 4))
    refused(svpa.logits_process, good, **bad)


@pytest.mark.parametrize("bad", [
    dict(slot_map=z(4)), dict(slot_map=z(10)[::2]), dict(slot_map=z(5, dtype=torch.int64)),
    dict(new_k=z(5, 2, 64, dtype=torch.float16)), dict(new_v=z(5, 2, 64, dtype=F32)), dict(new_v=z(4, 2, 64, dtype=BF)),
    dict(new_k=z(1, 64, 2, dtype=BF).transpose(1, 2), new_v=z(1, 2, 64, dtype=BF)),
    dict(k_pool=z(9, 2, 16, 32, dtype=BF)), dict(v_pool=z(8, 2, 16, 64, dtype=BF)), dict(k_pool=z(9, 2, 16, 64, dtype=F32)),
    dict(v_pool=z(9, 16, 2, 64, dtype=BF).transpose(1, 2)),
    dict(k_pool=z(9, 2, 16, 64, dtype=torch.uint8), v_pool=z(9, 2, 16, 64, dtype=torch.uint8),
         k_scale=z(9, 2, 16, 1, dtype=F32), v_scale=z(9, 2, dtype=F32), scale_tile=64),
])
def test_write(bad):
    good = dict(new_k=z(5, 2, 64, dtype=BF), new_v=z(5, 2, 64, dtype=BF), slot_map=z(5),
                k_pool=z(9, 2, 16, 64, dtype=BF), v_pool=z(9, 2, 16, 64, dtype=BF), error_flag=z(1))
    refused(svpa.kv_write, good, **bad)


@pytest.mark.parametrize("bad", [
    dict(q=z(6, 4, 64, dtype=BF)), dict(q=z(7, 2, 64, dtype=BF)), dict(q=z(7, 4, 64, dtype=torch.float16)),
    dict(q=z(7, 4, 128, dtype=BF)[:, :, ::2]), dict(q=z(7, 64, 4, dtype=BF).transpose(1, 2)),
    dict(block_table=z(2, 9)[:, :4]), dict(block_table=z(2, 3)), dict(block_table=z(2, 4, dtype=torch.int64)),
    dict(cu_seqlens=z(2)), dict(kv_lens=z(1)), dict(kv_lens=z(2, dtype=torch.int64)), dict(lse=z(7, 3, dtype=F32)),
    dict(out=z(7, 4, 64, dtype=F32)), dict(out=z(7, 8, 64, dtype=BF)[:, :4]), dict(k_pool=z(8, 2, 16, 64, dtype=BF)),
    dict(v_pool=z(9, 2, 16, 64, dtype=F32)),
])
def test_prompt(bad):
    good = dict(params=svpa.prompt_params(2, 7, 4, 2, 64, 4, 9), q=z(7, 4, 64, dtype=BF), out=z(7, 4, 64, dtype=BF),
                k_pool=z(9, 2, 16, 64, dtype=BF), v_pool=z(9, 2, 16, 64, dtype=BF), block_table=z(2, 4),
                cu_seqlens=z(3), kv_lens=z(2), lse=z(7, 4, dtype=F32), workspace=z(1), error_flag=z(1))
    refused(svpa.paged_prompt_attn, good, **bad)


def test_prompt_of_one_scattered_token():
    """A single token has no stride to compare, but its values have to be contiguous all the same."""
    q = z(1, 64, 4, dtype=BF).transpose(1, 2)
    x = z(64)
    with pytest.raises(svpa.SvpaError):
        svpa.paged_prompt_attn(svpa.prompt_params(1, 1, 4, 2, 64, 4, 9), q, x, x, x, x, x, q, workspace=x, error_flag=x,
                               stream=0)


@pytest.mark.parametrize("bad", [
    dict(q=z(2, 3, 8, 64, dtype=BF)[:, :, :4]), dict(q=z(2, 3, 4, 64, dtype=torch.float16)),
    dict(prefix_blocks=z(4)[::2]), dict(prefix_blocks=z(2, dtype=torch.int64)), dict(block_table=z(2, 8)[:, :4]),
    dict(block_table=z(1, 4)), dict(context_lens=z(1)), dict(out=z(2, 3, 4, 64, dtype=F32)),
    dict(lse=z(2, 3, 3, dtype=F32)), dict(k_pool=z(8, 2, 16, 64, dtype=BF)), dict(ancestor_mask=[1, 3]),
])
def test_prefix(bad):
    good = dict(params=svpa.attn_params(2, 3, 4, 2, 64, 4, 9), q=z(2, 3, 4, 64, dtype=BF), out=z(2, 3, 4, 64, dtype=BF),
                k_pool=z(9, 2, 16, 64, dtype=BF), v_pool=z(9, 2, 16, 64, dtype=BF), prefix_blocks=z(2),
                block_table=z(2, 4), context_lens=z(2), workspace=z(1), error_flag=z(1))
    refused(svpa.prefix_verify_attn, good, **bad)


@pytest.mark.parametrize("bad", [
    dict(seq_lens=z(1)), dict(seq_lens=z(2, dtype=torch.int64)), dict(cu_seqlens=z(2)), dict(free_stack=z(8)),
    dict(block_table=z(2, 8)[:, :4]), dict(slot_map=z(20)[::2]), dict(refcount=z(9, dtype=torch.int64)),
    dict(prefix_blocks=z(4)[::2]), dict(free_top=z(0)),
])
def test_build(bad):
    good = dict(seq_lens=z(2), block_table=z(2, 4), cu_seqlens=z(3), slot_map=z(10), refcount=z(9), free_stack=z(9),
                free_top=z(1), workspace=z(64), error_flag=z(1), prefix_blocks=z(2))
    refused(svpa.block_table_build, good, **bad)

"""Host-side refusals of the packed-query attention calls (CPU only)."""
import ctypes

import pytest

NZ = ctypes.c_void_p(256)  # never dereferenced: validation returns before any launch
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from speculative_verify_paged_attn_gb300 import build, svpa
    build.build()
    return svpa.load()


PROMPT = dict(batch=3, total_q=100, num_q_heads=8, num_kv_heads=2, head_dim=128, max_blocks_per_seq=20, num_blocks=70)


def prompt_status(lib, what="size", **kw):
    from speculative_verify_paged_attn_gb300 import svpa
    d = dict(PROMPT)
    d.update(kw)
    n = ctypes.c_size_t(0)
    return lib.svpa_paged_prompt_attn_workspace_size(ctypes.byref(svpa.prompt_params(**d)), ctypes.byref(n))


@pytest.mark.parametrize("bad,status", [
    (dict(), 0), (dict(batch=-1), 1), (dict(total_q=-1), 1), (dict(num_kv_heads=3), 1), (dict(num_q_heads=0), 1),
    (dict(block_size=32), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1), (dict(sm_scale=0.0), 1),
    (dict(sm_scale=float("nan")), 1), (dict(sm_scale=float("inf")), 1), (dict(q_stride=8 * 128 + 4), 1),
    (dict(q_stride=8 * 128 - 8), 1), (dict(q_stride=12 * 128), 0), (dict(head_dim=96), 2), (dict(kv_fp8=True), 2),
    (dict(num_q_heads=258), 2), (dict(num_q_heads=256), 0), (dict(max_blocks_per_seq=1 << 28), 2),
    (dict(num_blocks=1 << 30), 2), (dict(batch=(1 << 20) + 1), 2), (dict(total_q=(1 << 28) + 1), 2),
    (dict(total_q=1 << 28, batch=1 << 20, num_q_heads=128, num_kv_heads=128, num_blocks=7), 0),
])
def test_prompt_shapes(lib, bad, status):
    assert prompt_status(lib, **bad) == status


def test_prompt_call_arguments(lib):
    from speculative_verify_paged_attn_gb300 import svpa
    p = svpa.prompt_params(**PROMPT)
    r = ctypes.byref(p)
    size = svpa.paged_prompt_attn_workspace_size(p)
    call = lib.svpa_paged_prompt_attn
    good = [NZ] * 9
    for i in (0, 1, 2, 3, 4, 5, 6):  # every array but lse is required
        args = list(good)
        args[i] = None
        assert call(r, *args, size, NZ, None) == 1, i
    for i in (0, 1, 2, 6):
        args = list(good)
        args[i] = ODD
        assert call(r, *args, size, NZ, None) == 1, i
    assert call(r, *good, size, None, None) == 1  # the error word
    assert call(r, *good[:8], None, size, NZ, None) == 6
    assert call(r, *good[:8], ODD, size, NZ, None) == 6
    assert call(r, *good, size - 1, NZ, None) == 6
    assert call(None, *good, size, NZ, None) == 1
    for none in (dict(batch=0), dict(total_q=0)):  # nothing to do
        q = svpa.prompt_params(**dict(PROMPT, **none))
        assert call(ctypes.byref(q), *([None] * 9), 0, None, None) == 0


def test_prompt_binding_refuses_rows_other_than_its_stride(lib):
    import torch

    from speculative_verify_paged_attn_gb300 import svpa
    p = svpa.prompt_params(1, 5, 2, 2, 64, 4, 4)
    q = torch.zeros(5, 6, 64, dtype=torch.bfloat16)[:, :2]  # sliced, but q_stride not said
    x = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(svpa.SvpaError):
        svpa.paged_prompt_attn(p, q, x, x, x, x, x, q, workspace=x, error_flag=x, stream=0)


@pytest.mark.parametrize("prefix,kw,status", [
    (0, {}, 0), (512, {}, 0), (-16, {}, 1), (100, {}, 1), (16 * 71, {}, 1), (16 * 70, {}, 0),
    (512, dict(kv_fp8=True), 2), (512, dict(variant=1), 2), (512, dict(variant=2), 0), (512, dict(n_q=40), 2),
    (512, dict(head_dim=96), 2), (512, dict(num_kv_heads=3), 1), (512, dict(n_q=0), 1), (512, dict(n_q=65), 1),
    (512, dict(batch=65536), 2),
    # more units than 31 bits count
    (512, dict(batch=65535, n_q=8, num_q_heads=131070, num_kv_heads=65535), 2),
])
def test_prefix_shapes(lib, prefix, kw, status):
    from speculative_verify_paged_attn_gb300 import svpa
    d = dict(batch=3, n_q=5, num_q_heads=8, num_kv_heads=2, head_dim=128, max_blocks_per_seq=60, num_blocks=70)
    d.update(kw)
    n = ctypes.c_size_t(0)
    assert lib.svpa_prefix_verify_attn_workspace_size(ctypes.byref(svpa.attn_params(**d)), prefix,
                                                      ctypes.byref(n)) == status


def test_prefix_call_arguments(lib):
    from speculative_verify_paged_attn_gb300 import svpa
    p = svpa.attn_params(3, 5, 8, 2, 128, 60, 70)
    r = ctypes.byref(p)
    size = svpa.prefix_verify_attn_workspace_size(p, 512)
    call = lib.svpa_prefix_verify_attn

    def run(ptrs, prefix=512, bytes_=size, err=NZ, mask=None):
        q, k, v, blocks, table, lens, out, ws = ptrs
        return call(r, q, k, v, blocks, prefix, table, lens, mask, out, None, ws, bytes_, err, None)

    good = [NZ] * 8
    for i in range(7):
        args = list(good)
        args[i] = None
        assert run(args) == 1, i
    for i in (0, 1, 2, 6):
        args = list(good)
        args[i] = ODD
        assert run(args) == 1, i
    assert run(good, err=None) == 1
    assert run(good[:7] + [None]) == 6
    assert run(good[:7] + [ODD]) == 6
    assert run(good, bytes_=size - 1) == 6
    blind = (ctypes.c_uint64 * 5)(1, 2, 4, 8, 0)  # a query that does not see itself
    assert run(good, mask=ctypes.cast(blind, ctypes.c_void_p)) == 1
    p0 = svpa.attn_params(0, 5, 8, 2, 128, 60, 70)
    assert call(ctypes.byref(p0), None, None, None, None, 0, None, None, None, None, None, None, 0, None, None) == 0


def test_workspaces_keep_room_for_tickets(lib):
    """Counters and 64 KB of tickets head every attention workspace; the
    allocation-free call, whose array is its own, takes what it took without them."""
    from speculative_verify_paged_attn_gb300 import svpa
    head = 256 + (64 << 10)
    assert svpa.attn_workspace_size(svpa.attn_params(1, 1, 8, 8, 128, 4, 16)) >= head
    assert svpa.paged_prompt_attn_workspace_size(svpa.prompt_params(**PROMPT)) >= head
    for prefix in (0, 512):
        assert svpa.prefix_verify_attn_workspace_size(svpa.attn_params(3, 5, 8, 2, 128, 60, 70), prefix) >= head

    def needs(b):  # 2 heads, 25 splits of 20 rows: partials behind the head
        return svpa.attn_workspace_size(svpa.attn_params(b, 5, 8, 2, 128, 500, 16, split_pages=20)) - head

    # the largest batch that 32 MiB hold with 8 bytes of tickets a sequence in the head's place
    batch = max(b for b in range(1, 200) if needs(b) + 256 + (b * 8 + 255) // 256 * 256 <= 32 << 20)
    for b, status in ((batch, 1), (batch + 1, 6)):  # null arrays, or too large
        p = svpa.attn_params(b, 5, 8, 2, 128, 500, 16, split_pages=20)
        assert svpa.paged_verify_attn_noalloc(p, None, None, None, None, None, None, error_flag=None, stream=0,
                                              check=False) == status, b


def test_units_leave_room_for_the_counter(lib):
    # 1038435 sequences of 2068 kv heads: 67 units below 2^31, and the kernel's
    # counter goes up to one for each CTA past the last unit
    heads = dict(total_q=1, num_q_heads=2068, num_kv_heads=2068, head_dim=64, num_blocks=5)
    assert prompt_status(lib, batch=1038435, **heads) == 2
    assert prompt_status(lib, batch=1038435 - 64, **heads) == 0

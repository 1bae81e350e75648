"""Host-side refusals of the block-table build, the K/V scatter and the logits
processing (CPU only)."""
import ctypes

import pytest

NZ = ctypes.c_void_p(256)  # never dereferenced: validation returns before any launch
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from speculative_verify_paged_attn_gb300 import build, svpa
    build.build()
    return svpa.load()


def build_status(lib, sizes=None, prefix_len=32, ptrs=None, ws=NZ, bytes_=256, err=NZ):
    d = dict(batch=3, block_size=16, max_blocks=20, num_blocks=70, slots=100)
    d.update(sizes or {})
    # lengths, prefix blocks, table, offsets, slots, counts, stack, top
    p = [NZ] * 8
    for i in ptrs or ():
        p[i] = None
    return lib.svpa_block_table_build(d["batch"], d["block_size"], d["max_blocks"], d["num_blocks"], d["slots"], p[0],
                                      p[1], prefix_len, *p[2:], ws, bytes_, err, None)


@pytest.mark.parametrize("sizes,status", [
    (dict(batch=-1), 1), (dict(block_size=8), 1), (dict(max_blocks=0), 1), (dict(num_blocks=0), 1),
    (dict(slots=-1), 1), (dict(batch=8193), 2), (dict(num_blocks=1 << 27), 2), (dict(max_blocks=1 << 27), 2),
    (dict(slots=(1 << 30) + 1), 2), (dict(batch=0), 0),
])
def test_build_sizes(lib, sizes, status):
    assert build_status(lib, sizes) == status


def test_build_arguments(lib):
    for prefix in (-16, 8, 16 * 21):
        assert build_status(lib, prefix_len=prefix) == 1, prefix
    for i in range(8):
        assert build_status(lib, ptrs=[i]) == 1, i
    assert build_status(lib, err=None) == 1
    assert build_status(lib, ws=None) == 6 and build_status(lib, ws=ODD) == 6 and build_status(lib, bytes_=255) == 6
    n = ctypes.c_size_t(0)
    assert lib.svpa_block_table_build_workspace_size(8192, ctypes.byref(n)) == 0 and n.value == 256
    assert lib.svpa_block_table_build_workspace_size(8193, ctypes.byref(n)) == 2
    assert lib.svpa_block_table_build_workspace_size(-1, ctypes.byref(n)) == 1
    assert lib.svpa_block_table_build_workspace_size(1, None) == 1


def write_status(lib, ptrs=None, odd=(), err=NZ, **kw):
    d = dict(t=5, h=4, d=64, bs=16, nb=9, dt=0, tile=0, ks=256, vs=256)
    d.update(kw)
    p = [NZ] * 7  # k, v, slots, k pool, v pool, k scale, v scale
    for i in ptrs or ():
        p[i] = None
    for i in odd:
        p[i] = ODD
    return lib.svpa_kv_write(d["t"], d["h"], d["d"], d["bs"], d["nb"], d["dt"], d["tile"], p[0], p[1], d["ks"], d["vs"],
                             *p[2:], err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), 1), (dict(h=0), 1), (dict(h=4097, ks=1 << 20, vs=1 << 20), 1), (dict(d=60), 1), (dict(d=0), 1),
    (dict(d=1032, ks=8192, vs=8192), 1), (dict(bs=32), 1), (dict(nb=0), 1), (dict(dt=2), 1), (dict(tile=64), 1),
    (dict(dt=1, tile=32), 1), (dict(ks=248), 1), (dict(vs=260), 1), (dict(dt=1), 2),
    (dict(dt=1, tile=64, d=72, ks=288, vs=288), 2), (dict(t=(1 << 28) + 1), 2),
    (dict(t=1 << 28, h=64, d=1024, ks=65536, vs=65536), 2), (dict(t=0), 0),
])
def test_write_sizes(lib, kw, status):
    assert write_status(lib, **kw) == status


def test_write_arguments(lib):
    for i in range(5):
        assert write_status(lib, ptrs=[i]) == 1, i
    for i in (0, 1, 3, 4):
        assert write_status(lib, odd=[i]) == 1, i
    for i in (5, 6):
        assert write_status(lib, ptrs=[i], dt=1, tile=64) == 1, i
    assert write_status(lib, err=None) == 1


def test_write_binding_refuses_scattered_rows(lib):
    import torch

    from speculative_verify_paged_attn_gb300 import svpa
    x = torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)  # the head's values are not contiguous
    slots, pool, err = torch.zeros(5, dtype=torch.int32), torch.zeros(9, 4, 16, 64, dtype=torch.bfloat16), torch.zeros(1)
    with pytest.raises(svpa.SvpaError):
        svpa.kv_write(x, x, slots, pool, pool, error_flag=err, stream=0)


def logits_status(lib, ptrs=(), logits=NZ, out=NZ, err=NZ, parent=None, history=NZ, **kw):
    from speculative_verify_paged_attn_gb300 import svpa
    d = dict(batch=2, rows=3, vocab=100, max_history=10, logits_dtype=0)
    d.update(kw)
    p = dict(prompt=NZ, hist_lens=NZ, drafts=NZ, rep=NZ, pres=NZ, freq=NZ, off=NZ, tok=NZ, val=NZ, mask=NZ)
    for k in ptrs:
        p[k] = None
    par = None
    if parent is not None:
        par = ctypes.cast((ctypes.c_int32 * len(parent))(*parent), ctypes.c_void_p)
    return lib.svpa_logits_process(ctypes.byref(svpa.LogitsParams(**d)), logits, history, p["prompt"], p["hist_lens"],
                                   p["drafts"], par, p["rep"], p["pres"], p["freq"], p["off"], p["tok"], p["val"],
                                   p["mask"], out, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(rows=0), 1), (dict(rows=65), 1), (dict(vocab=0), 1), (dict(max_history=-1), 1),
    (dict(max_history=0), 1), (dict(logits_dtype=2), 1), (dict(vocab=(1 << 24) + 1), 2), (dict(batch=65536), 2),
    (dict(logits=None), 1), (dict(out=None), 1), (dict(err=None), 1), (dict(ptrs=["hist_lens"]), 1),
    (dict(ptrs=["off"]), 1), (dict(ptrs=["val"]), 1), (dict(parent=[0, 0, 0]), 1), (dict(parent=[-1, 1, 0]), 1),
    (dict(parent=[-1, 0, -1]), 1), (dict(logits_dtype=1), 1),  # bf16 in place
    (dict(logits=ctypes.c_void_p(258)), 1), (dict(out=ctypes.c_void_p(262)), 1),
    (dict(logits=ctypes.c_void_p(257), logits_dtype=1), 1), (dict(batch=0, logits=None, out=None, err=None), 0),
])
def test_logits_arguments(lib, kw, status):
    assert logits_status(lib, **kw) == status


@pytest.mark.parametrize("n,status", [((1 << 28) + 1, 2), (0x7fffffff, 2)])
def test_logits_history_limit(lib, n, status):
    # a count has 29 bits and the history's index runs a step past its end: neither may wrap
    assert logits_status(lib, max_history=n) == status

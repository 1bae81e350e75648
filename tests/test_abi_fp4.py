"""Host-side refusals of the norms and rotation, the page writes and reads, and
the append and the attention on 4-bit pages; the 4-bit definitions (CPU only)."""
import ctypes

import pytest
import torch

import fp4_ref as F

NZ = ctypes.c_void_p(256)  # never dereferenced: validation returns before any launch
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    from speculative_verify_paged_attn_gb300 import build, svpa
    build.build()
    return svpa.load()


def params(**kw):
    from speculative_verify_paged_attn_gb300 import svpa
    d = dict(num_tokens=5, num_q_heads=8, num_kv_heads=2, head_dim=64, rotary_dim=64, interleaved=0, max_position=100,
             block_size=16, num_blocks=9, kv_dtype=0, scale_tile=0, eps=1e-6, q_stride=512, k_stride=128, v_stride=128,
             q_out_stride=512, k_out_stride=128)
    d.update(kw)
    return svpa.RopeParams(**d)


def rope_status(lib, null=(), odd=(), write=False, **kw):
    names = ["q", "k"] + (["v"] if write else []) + ["positions"] + (["slots"] if write else []) + \
            ["cos_sin", "qw", "kw", "q_out"] + \
            (["k_pool", "v_pool", "k_scale", "v_scale", "kf", "vf"] if write else ["k_out"]) + ["err"]
    ptrs = {n: ctypes.c_void_p(256 * (i + 1)) for i, n in enumerate(names)}
    ptrs.update({n: None for n in null})
    ptrs.update({n: ODD for n in odd})
    for n in ("q_out", "k_out"):
        if n in kw:
            ptrs[n] = ptrs[kw.pop(n)]
    f = lib.svpa_rope_kv_write if write else lib.svpa_qk_norm_rope
    return f(ctypes.byref(params(**kw)), *[ptrs[n] for n in names], None)


BAD = [(dict(num_tokens=-1), 1), (dict(num_q_heads=-1), 1), (dict(num_kv_heads=0), 1),
       (dict(num_kv_heads=4097, k_stride=1 << 20, v_stride=1 << 20, k_out_stride=1 << 20), 1), (dict(rotary_dim=-2), 1),
       (dict(rotary_dim=80), 1), (dict(rotary_dim=31), 1), (dict(rotary_dim=24), 2), (dict(interleaved=2), 1),
       (dict(max_position=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(head_dim=96), 2),
       (dict(q_stride=504), 1), (dict(k_stride=120), 1), (dict(k_stride=132), 1), (dict(q_out_stride=508), 1),
       (dict(num_tokens=(1 << 28) + 1), 2), (dict(num_tokens=0), 0)]


@pytest.mark.parametrize("kw,status", BAD + [(dict(k_out_stride=120), 1)])
def test_rope_sizes(lib, kw, status):
    assert rope_status(lib, **kw) == status


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(v_stride=120), 1), (dict(block_size=8), 1), (dict(num_blocks=0), 1), (dict(num_blocks=1 << 27), 2),
    (dict(kv_dtype=3), 1), (dict(scale_tile=64), 1), (dict(kv_dtype=1), 2), (dict(kv_dtype=1, scale_tile=32), 1),
    (dict(kv_dtype=2, scale_tile=64), 1)])
def test_rope_write_sizes(lib, kw, status):
    assert rope_status(lib, write=True, **kw) == status


def test_rope_arguments(lib):
    for n in ("q", "k", "positions", "cos_sin", "q_out", "k_out", "err"):
        assert rope_status(lib, null=[n]) == 1, n
    for n in ("q", "k", "v", "positions", "slots", "cos_sin", "q_out", "k_pool", "v_pool", "err"):
        assert rope_status(lib, null=[n], write=True) == 1, n
    for n in ("k_scale", "v_scale"):
        assert rope_status(lib, null=[n], write=True, kv_dtype=1, scale_tile=64) == 1, n
    for n in ("q", "k", "cos_sin", "qw", "kw", "q_out", "k_out"):
        assert rope_status(lib, odd=[n]) == 1, n
    for n in ("q", "k", "v", "cos_sin", "qw", "kw", "q_out", "k_pool", "v_pool"):
        assert rope_status(lib, odd=[n], write=True) == 1, n
    # in place needs one stride
    assert rope_status(lib, q_out="q", q_out_stride=1024) == 1
    assert rope_status(lib, k_out="k", k_out_stride=1024) == 1


def read_status(lib, null=(), odd=(), **kw):
    d = dict(t=5, h=2, d=64, bs=16, nb=9, dt=2, tile=0, ks=128, vs=128)
    d.update(kw)
    p = [None if i in null else ODD if i in odd else NZ for i in range(9)]
    return lib.svpa_kv_read(*[d[x] for x in ("t", "h", "d", "bs", "nb", "dt", "tile")], *p, d["ks"], d["vs"],
                            None if "err" in null else NZ, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), 1), (dict(h=0), 1), (dict(h=4097, ks=1 << 20, vs=1 << 20), 1), (dict(d=0), 1), (dict(d=60), 1),
    (dict(d=24, dt=2), 1), (dict(d=1040, ks=4096, vs=4096), 1), (dict(bs=8), 1), (dict(nb=0), 1), (dict(nb=1 << 27), 2),
    (dict(dt=3), 1), (dict(tile=64), 1), (dict(dt=1), 2), (dict(dt=1, tile=64, d=72, ks=144, vs=144), 2),
    (dict(ks=120), 1), (dict(vs=132), 1), (dict(t=(1 << 28) + 1), 2), (dict(t=0), 0),
])
def test_read_sizes(lib, kw, status):
    assert read_status(lib, **kw) == status


def test_read_arguments(lib):
    for i in (0, 1, 2, 7, 8, "err"):
        assert read_status(lib, null=[i]) == 1, i
    for i in (1, 2, 7, 8):
        assert read_status(lib, odd=[i]) == 1, i
    for i in (3, 4):
        assert read_status(lib, null=[i], dt=1, tile=64) == 1, i


def append_status(lib, null=(), odd=(), **kw):
    d = dict(b=2, n=5, h=2, d=64, bs=16, mb=8, nb=9)
    d.update(kw)
    p = [None if i in null else ODD if i in odd else NZ for i in range(11)]
    return lib.svpa_kv_append_fp4(*[d[x] for x in ("b", "n", "h", "d", "bs", "mb", "nb")], *p,
                                  None if "err" in null else NZ, None)


@pytest.mark.parametrize("kw,status", [
    (dict(b=-1), 1), (dict(n=0), 1), (dict(n=4097), 1), (dict(h=0), 1), (dict(h=4097), 1), (dict(d=8), 1), (dict(d=72), 1),
    (dict(d=1040), 1), (dict(bs=32), 1), (dict(mb=0), 1), (dict(nb=0), 1), (dict(b=0), 0),
])
def test_append_sizes(lib, kw, status):
    assert append_status(lib, **kw) == status


def test_append_arguments(lib):
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, "err"):
        assert append_status(lib, null=[i]) == 1, i
    for i in (0, 1, 7, 8):
        assert append_status(lib, odd=[i]) == 1, i


def attn_status(lib, null=(), odd=(), mask=None, bytes_=1 << 40, **kw):
    from speculative_verify_paged_attn_gb300 import svpa
    d = dict(batch=2, n_q=3, num_q_heads=8, num_kv_heads=2, head_dim=64, max_blocks_per_seq=8, num_blocks=9, kv_fp4=True)
    d.update(kw)
    p = svpa.attn_params(**{k: v for k, v in d.items() if k != "kv_dtype"})
    if "kv_dtype" in d:
        p.kv_dtype = d["kv_dtype"]
    ptr = [None if i in null else ODD if i in odd else NZ for i in range(7)]
    m = None if mask is None else ctypes.cast((ctypes.c_uint64 * len(mask))(*mask), ctypes.c_void_p)
    tail = [None if i in null else ODD if i in odd else NZ for i in ("out", "lse", "ws")]
    return lib.svpa_paged_verify_attn_fp4(ctypes.byref(p), *ptr, m, *tail, bytes_, None if "err" in null else NZ, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(n_q=0), 1), (dict(n_q=65), 1), (dict(num_q_heads=0), 1), (dict(num_kv_heads=3), 1),
    (dict(num_kv_heads=0), 1), (dict(block_size=8), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1),
    (dict(sm_scale=0.0), 1), (dict(sm_scale=float("inf")), 1), (dict(split_pages=-1), 1), (dict(variant=1), 1),
    (dict(scale_tile=64), 1), (dict(kv_dtype=0), 1), (dict(kv_dtype=1), 1), (dict(head_dim=96), 2),
    (dict(n_q=33), 2), (dict(batch=65536), 2), (dict(num_blocks=1 << 30, num_kv_heads=2), 2),
    (dict(max_blocks_per_seq=1 << 27), 2), (dict(max_blocks_per_seq=(1 << 27) - 8), 2), (dict(batch=0), 0),
    (dict(mask=[1, 2, 3]), 1), (dict(mask=[1, 3, 15]), 1),
    (dict(bytes_=255), 6),
])
def test_attention_sizes(lib, kw, status):
    assert attn_status(lib, **kw) == status


def test_attention_arguments(lib):
    for i in (0, 1, 2, 5, 6, "out", "err"):
        assert attn_status(lib, null=[i]) == 1, i
    for i in (0, 1, 2, "out"):
        assert attn_status(lib, odd=[i]) == 1, i
    assert attn_status(lib, null=["ws"]) == 6 and attn_status(lib, odd=["ws"]) == 6
    from speculative_verify_paged_attn_gb300 import svpa
    p = svpa.attn_params(2, 3, 8, 2, 64, 8, 9, kv_fp4=True)
    assert lib.svpa_paged_verify_attn_fp4_workspace_size(ctypes.byref(p), None) == 1
    # other calls keep refusing 4-bit pages
    n = ctypes.c_size_t(0)
    assert lib.svpa_attn_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 1


def test_commit_of_a_tree_knows_4_bit_pages(lib):
    base = [0, 5, 16, 8, 16]
    assert lib.svpa_block_table_commit(*base, *([None] * 7), 0, None, None, 4, 64, 2, None, None) == 0
    base[0] = 2
    # a tree path: FP8 pages are refused, 4-bit ones need their pools
    assert lib.svpa_block_table_commit(*base, *([NZ] * 7), 3, NZ, NZ, 4, 64, 1, NZ, None) == 2
    assert lib.svpa_block_table_commit(*base, *([NZ] * 7), 3, None, NZ, 4, 64, 2, NZ, None) == 1
    assert lib.svpa_block_table_commit(*base, *([NZ] * 7), 3, NZ, ODD, 4, 64, 2, NZ, None) == 1


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.mark.parametrize("bad", [
    dict(k=z(5, 2, 64, dtype=torch.float16)), dict(k=z(5, 64, 2, dtype=BF).transpose(1, 2)), dict(q=z(4, 4, 64, dtype=BF)),
    dict(q=z(5, 4, 128, dtype=BF)), dict(q_out=None), dict(q_out=z(5, 2, 64, dtype=BF)), dict(k_out=z(5, 2, 64, dtype=F32)),
    dict(positions=z(5, dtype=torch.int64)), dict(positions=z(4)), dict(cos_sin=z(9, 64, dtype=torch.float64)),
    dict(cos_sin=z(64, dtype=F32)), dict(cos_sin=z(9, 128, dtype=F32)[:, ::2]), dict(q_weight=z(64, dtype=F32)),
    dict(k_weight=z(63, dtype=BF)), dict(error_flag=z(1, dtype=F32)),
])
def test_binding_refuses_wrong_rows(lib, bad):
    from speculative_verify_paged_attn_gb300 import svpa
    good = dict(q=z(5, 4, 64, dtype=BF), k=z(5, 2, 64, dtype=BF), positions=z(5), cos_sin=z(9, 64, dtype=F32),
                q_out=z(5, 4, 64, dtype=BF), k_out=z(5, 2, 64, dtype=BF), q_weight=z(64, dtype=BF),
                k_weight=z(64, dtype=BF), error_flag=z(1))
    good.update(bad)
    with pytest.raises(svpa.SvpaError):
        svpa.qk_norm_rope(**good, stream=0)


@pytest.mark.parametrize("bad", [
    dict(v=z(5, 3, 64, dtype=BF)), dict(slot_map=z(10)[::2]), dict(slot_map=z(4)), dict(k_pool=z(9, 2, 575, dtype=U8)),
    dict(v_pool=z(8, 2, 576, dtype=U8)), dict(k_pool=z(9, 2, 576, dtype=BF)), dict(k_factor=z(1, dtype=F32)),
    dict(v_factor=z(2, dtype=torch.float64)), dict(q=z(5, 4, 64, dtype=BF)),
])
def test_binding_refuses_wrong_pages(lib, bad):
    from speculative_verify_paged_attn_gb300 import svpa
    good = dict(k=z(5, 2, 64, dtype=BF), v=z(5, 2, 64, dtype=BF), positions=z(5), slot_map=z(5),
                cos_sin=z(9, 64, dtype=F32), k_pool=z(9, 2, 576, dtype=U8), v_pool=z(9, 2, 576, dtype=U8),
                k_factor=z(2, dtype=F32), v_factor=z(2, dtype=F32), error_flag=z(1), fp4=True)
    good.update(bad)
    with pytest.raises(svpa.SvpaError):
        svpa.rope_kv_write(**good, stream=0)


@pytest.mark.parametrize("bad", [
    dict(k_out=z(5, 2, 64, dtype=F32)), dict(v_out=z(4, 2, 64, dtype=BF)), dict(slot_map=z(4)),
    dict(k_pool=z(9, 2, 500, dtype=U8)), dict(k_factor=z(1, dtype=F32)),
])
def test_binding_refuses_wrong_reads(lib, bad):
    from speculative_verify_paged_attn_gb300 import svpa
    good = dict(slot_map=z(5), k_pool=z(9, 2, 576, dtype=U8), v_pool=z(9, 2, 576, dtype=U8),
                k_out=z(5, 2, 64, dtype=BF), v_out=z(5, 2, 64, dtype=BF), error_flag=z(1), fp4=True)
    good.update(bad)
    with pytest.raises(svpa.SvpaError):
        svpa.kv_read(**good, stream=0)


@pytest.mark.parametrize("bad", [
    dict(q=z(2, 3, 8, 32, dtype=BF)), dict(q=z(2, 3, 8, 64, dtype=torch.float16)), dict(k_pool=z(9, 2, 575, dtype=U8)),
    dict(v_pool=z(9, 2, 576, dtype=BF)), dict(block_table=z(2, 16)[:, :8]), dict(context_lens=z(1)),
    dict(out=z(2, 3, 8, 64, dtype=F32)), dict(lse=z(2, 3, 7, dtype=F32)), dict(ancestor_mask=[1, 3]),
    dict(k_factor=z(1, dtype=F32)),
])
def test_binding_refuses_wrong_attention(lib, bad):
    from speculative_verify_paged_attn_gb300 import svpa
    good = dict(params=svpa.attn_params(2, 3, 8, 2, 64, 8, 9, kv_fp4=True), q=z(2, 3, 8, 64, dtype=BF),
                k_pool=z(9, 2, 576, dtype=U8), v_pool=z(9, 2, 576, dtype=U8), block_table=z(2, 8), context_lens=z(2),
                out=z(2, 3, 8, 64, dtype=BF), workspace=z(1), error_flag=z(1))
    good.update(bad)
    with pytest.raises(svpa.SvpaError):
        svpa.paged_verify_attn_fp4(**good, stream=0)


def test_definition_worked_example():
    # 16 values with the largest 6: scale 1, codes the values themselves; borders go to the even code
    row = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.26, 0, 4.9, 5.1, -6.0])
    code, byte = F.encode(row.bfloat16()[None, None], torch.ones(1))
    assert byte.tolist() == [[[0x38]]]
    assert code.flatten().tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 0, 6, 7, 15]
    assert F.values(code, byte, torch.ones(1)).flatten().tolist()[:8] == [6, 0, 1, 1, 2, 2, 4, 4]
    # a group of zeros, one too small for its scale, one past the largest scale
    x = torch.tensor([[0.0] * 16, [2.0 ** -10] * 16, [3000.0, 1000.0] + [0.0] * 14]).bfloat16()
    code, byte = F.encode(x[:, None], torch.ones(1))
    assert byte.flatten().tolist() == [0, 0, 0x7e] and code[0].sum() == 0 and code[1].sum() == 0
    assert code[2].flatten().tolist()[:2] == [7, 4]


def test_pool_layout_round_trip():
    g = torch.Generator().manual_seed(1)
    code = torch.randint(0, 16, (3, 16, 2, 32), generator=g)
    byte = torch.randint(0, 127, (3, 16, 2, 2), generator=g)
    pool = F.to_pool(F.pack(code, byte))
    assert pool.shape == (3, 2, 9 * 32)
    c, b = F.from_pool(pool)
    assert torch.equal(c, code) and torch.equal(b, byte)
    # element 5 of row 7, head 1, page 2: byte 2 of the row, its high half
    assert int(pool[2, 1, 7 * 16 + 2]) >> 4 == int(code[2, 7, 1, 5])
    assert int(pool[2, 1, 16 * 16 + 7 * 2 + 1]) == int(byte[2, 7, 1, 1])

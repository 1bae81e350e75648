"""GPU tests of the padding and bad rows of svpa_rope_kv_write among good ones."""
import pytest
import torch

from speculative_verify_paged_attn_gb300 import svpa
from test_gpu_rope import DEV, Rows, empty_pool, factors, ints

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def write(x, slots, kind, blocks=4):
    """The pools, scales and queries after a call into pages of that kind."""
    (kp, ks), (vp, vs) = [empty_pool(kind, blocks, x.hkv, x.d) for _ in range(2)]
    kf, vf = (factors(x.hkv, 1), factors(x.hkv, 2)) if kind == "fp4" else (None, None)
    q_out = torch.full((x.t, x.hq, x.d), 9.0, dtype=torch.bfloat16, device=DEV)
    svpa.rope_kv_write(x.k, x.v, x.pos, ints(slots), x.table, kp, vp, error_flag=x.err, q=x.q, q_out=q_out,
                       q_weight=x.qw, k_weight=x.kw, k_scale=ks, v_scale=vs, scale_tile=64 if kind == "fp8" else 0,
                       fp4=kind == "fp4", k_factor=kf, v_factor=vf)
    status = svpa.STATUS[svpa.check_error(x.err)]
    x.err.zero_()
    return status, [t for t in (q_out, kp, vp, ks, vs) if t is not None]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("norm", [True, False])
def test_what_a_padding_row_holds_does_not_matter(kind, norm):
    slots = [0, 17, -1, 3, -2 ** 31, 40, 63]
    x = Rows(7, 9, 3, 128, 128, norm=norm, fused=True, seed=1)
    status, want = write(x, slots, kind)
    assert status == "SVPA_OK"
    for t, bad in ((2, NAN), (4, INF)):
        x.q[t], x.k[t], x.v[t], x.pos[t] = bad, -bad, bad, 2 ** 31 - 1 if t == 2 else -1
    status, got = write(x, slots, kind)
    assert status == "SVPA_OK" and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_a_row_past_the_pool_is_reported_and_left_out(kind):
    x = Rows(5, 2, 2, 64, 64, seed=2)
    _, want = write(x, [0, 17, -1, 3, 60], kind)
    for bad in (64, 2 ** 31 - 1):
        status, got = write(x, [0, 17, bad, 3, 60], kind)
        assert status == "SVPA_ERR_BAD_BLOCK" and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_value_that_4_bits_cannot_hold_spoils_its_16_elements_alone(bad):
    x = Rows(5, 2, 2, 64, 0, norm=False, seed=3)
    slots = [0, 17, 9, 3, 60]
    _, (_, kp, vp) = write(x, slots, "fp4")
    x.k[2, 1, 21] = bad  # slot 9, head 1, elements 16 .. 31
    x.v[3, 0, 63] = bad  # slot 3, head 0, elements 48 .. 63
    status, (_, kb, vb) = write(x, slots, "fp4")
    assert status == "SVPA_ERR_INVALID_ARG"
    for pool, got, head, slot, group in ((kp, kb, 1, 9, 1), (vp, vb, 0, 3, 3)):
        keep = torch.ones_like(pool[0], dtype=torch.bool)
        keep[head, slot * 32 + group * 8:slot * 32 + group * 8 + 8] = False
        keep[head, 512 + slot * 4 + group] = False
        assert torch.equal(pool[0][keep], got[0][keep]) and torch.equal(pool[1:], got[1:])

"""GPU tests of svpa_kv_append_fp4 with rows and factors that 4-bit pages cannot
hold: the error is reported and no row is written."""
import pytest
import torch

from speculative_verify_paged_attn_gb300 import svpa
from test_gpu_rope import Append

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def refused(a):
    """The append of `a` reports a bad value; the pools are as they were and the tables are consistent."""
    pools = a.kp.clone(), a.vp.clone()
    svpa.kv_append_fp4(a.k, a.v, a.table, a.cl, a.count, a.free, a.top, a.kp, a.vp, error_flag=a.err, k_factor=a.kf,
                       v_factor=a.vf)
    assert svpa.STATUS[svpa.check_error(a.err)] == "SVPA_ERR_INVALID_ARG"
    assert torch.equal(a.kp, pools[0]) and torch.equal(a.vp, pools[1])
    held = torch.bincount(a.table[a.table >= 0].long(), minlength=a.blocks)
    assert torch.equal(held.int(), a.count)
    a.err.zero_()


SHAPES = [([9], 1, 1, 16), ([3, 15, 16, 31, 100], 5, 8, 128), ([0, 1, 40], 40, 3, 64),
          ([7 + i for i in range(160)], 8, 32, 128)]


@pytest.mark.parametrize("ctx,n_new,hkv,d", SHAPES)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_values_that_are_not_finite(ctx, n_new, hkv, d, where):
    a = Append(ctx, n_new, hkv, d, seed=2)
    good = a.k.clone(), a.v.clone()
    at = {"first": 0, "middle": a.k.numel() // 2 + 1, "last": a.k.numel() - 1}[where]
    for name, bad in (("k", NAN), ("v", INF), ("k", -INF)):
        getattr(a, name).view(-1)[at] = bad
        refused(a)
        a.k.copy_(good[0])
        a.v.copy_(good[1])
    a.run()  # the same call with finite values


@pytest.mark.parametrize("ctx,n_new,hkv,d", SHAPES)
def test_factors_out_of_range(ctx, n_new, hkv, d):
    a = Append(ctx, n_new, hkv, d, seed=3)
    good = a.kf.clone(), a.vf.clone()
    for i, bad in enumerate((0.0, -1.0, NAN, INF, 2.0 ** -61, 2.0 ** 61)):
        (a.kf if i % 2 else a.vf)[i * hkv // 6] = bad
        refused(a)
        a.kf.copy_(good[0])
        a.vf.copy_(good[1])
    a.run()


def test_a_replayed_append_reports_what_a_later_step_brings():
    """One captured append: finite values, a NaN, finite values again."""
    a = Append([20, 5, 33], 4, 2, 128, seed=4)
    a.run()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        svpa.kv_append_fp4(a.k, a.v, a.table, a.cl, a.count, a.free, a.top, a.kp, a.vp, error_flag=a.err,
                           k_factor=a.kf, v_factor=a.vf)
    pools = a.kp.clone(), a.vp.clone()
    keep = a.v[1, 2, 1, 77].item()
    a.k.neg_()
    a.v[1, 2, 1, 77] = NAN
    graph.replay()
    assert svpa.STATUS[svpa.check_error(a.err)] == "SVPA_ERR_INVALID_ARG"
    assert torch.equal(a.kp, pools[0]) and torch.equal(a.vp, pools[1])
    a.err.zero_()
    a.v[1, 2, 1, 77] = keep
    graph.replay()
    assert svpa.check_error(a.err) == 0
    want, values = a.kp.clone(), a.vp.clone()
    a.run()  # the same rows by an eager call, held to the definition
    assert torch.equal(a.kp, want) and torch.equal(a.vp, values)

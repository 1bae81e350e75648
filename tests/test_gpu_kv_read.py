"""GPU tests of the roundings of svpa_kv_read: one fp32 product, then bf16."""
from fractions import Fraction

import pytest
import torch

import fp4_ref as F
from speculative_verify_paged_attn_gb300 import svpa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def factors_beside_ties():
    """(factor, expected): 3 * factor lies beside a tie of bf16 (by less than half an
    fp32 step, so that the fp32 product is the tie), on the side away from the even
    neighbour; expected is that neighbour."""
    out = []
    for j in range(1, 250, 2):
        tie = Fraction(1) + Fraction(j, 256)
        f = torch.tensor(float(tie / 3), dtype=torch.float64).float()
        off = 3 * Fraction(f.item()) - tie
        down, up = tie - Fraction(1, 256), tie + Fraction(1, 256)
        even = down if (j - 1) // 2 % 2 == 0 else up
        if 0 < abs(off) < Fraction(1, 1 << 24) and (off > 0) == (even == down):
            out.append((f.item(), float(even)))
    assert len(out) > 20
    return out


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_product_in_fp32_and_then_bf16(kind):
    pairs = factors_beside_ties()
    heads, d = len(pairs), 64
    f = torch.tensor([p[0] for p in pairs], device=DEV)
    want = torch.tensor([p[1] for p in pairs], device=DEV).to(BF)[None, :, None].expand(16, heads, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.arange(16, dtype=torch.int32, device=DEV)
    k, v = [torch.zeros((16, heads, d), dtype=BF, device=DEV) for _ in range(2)]
    if kind == "fp4":  # code 3, scale 1
        rows = torch.full((1, 16, heads, d), 5, device=DEV), torch.full((1, 16, heads, d // 16), 0x38, device=DEV)
        pool = F.to_pool(F.pack(*rows))
        svpa.kv_read(slots, pool, pool, k, v, error_flag=err, fp4=True, k_factor=f, v_factor=f)
    else:
        pool = torch.full((1, heads, 16, d), 3.0, device=DEV).to(torch.float8_e4m3fn)
        scale = f[None, :, None, None].expand(1, heads, 16, 1).contiguous()
        svpa.kv_read(slots, pool, pool, k, v, error_flag=err, k_scale=scale, v_scale=scale, scale_tile=64)
    assert svpa.check_error(err) == 0
    assert torch.equal(k, want) and torch.equal(v, want)

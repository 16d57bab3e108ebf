"""Scales of the scores at the ends of fp32's range, over the 4-bit cache, against
the 64-bit model.  Tolerances: see check_attn."""
import pytest
import torch

from test_gpu_kv4 import BF16, F32, check_attn, filled, queries, sp  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(1, BF16), (150, BF16), (3, F32)]


# Products q k of up to some 1e38, which fp32 still holds (queries of 1e36, keys
# of ordinary size, 128 terms of either sign).
@pytest.mark.parametrize("Lq,dtype", SHAPES)
@pytest.mark.parametrize("tau", [0.0, -0.0, 2.0 ** -125, -2.0 ** -125, 2.0 ** -130])
def test_small_scales_of_large_products(sp, tau, Lq, dtype):
    cache = filled(sp, [700, 130], 1, 128)
    check_attn(sp, cache, queries(2, 2, Lq, 128, dtype, scale=1e36), tau=tau, causal=True)


@pytest.mark.parametrize("Lq,dtype", SHAPES)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_scale_of_zero_keeps_what_is_not_a_number(sp, bad, Lq, dtype):
    cache = filled(sp, [700], 1, 128)
    q = queries(1, 2, Lq, 128, dtype)
    want, want_lse = sp.sparstar_kv4_attn(cache, q, tau=0.0)
    q[0, 1, Lq // 2, 7] = bad
    out, lse = sp.sparstar_kv4_attn(cache, q, tau=0.0)
    assert torch.isnan(out[0, 1, Lq // 2]).all()
    out[0, 1, Lq // 2], lse[0, 1, Lq // 2] = want[0, 1, Lq // 2], want_lse[0, 1, Lq // 2]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)

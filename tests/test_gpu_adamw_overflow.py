"""A moment that leaves FP32's range shows: a block of 8-bit states with a
non-finite m or v becomes NaN as a whole from the next step on, and no other."""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("betas", [(0.9, 0.95), (0.9, 0.999), (0.95, 0.999)])
@pytest.mark.parametrize("large", [1e25, -1e20, 3e38, float("inf"), float("-inf"), float("nan")])
def test_a_block_whose_moments_overflow_becomes_nan(large, betas):
    g = torch.Generator().manual_seed(1)
    p = torch.randn(1000, generator=g).cuda()
    x = torch.randn(1000, generator=g).cuda()
    opt = M.AdamW([p], state_bits=8, betas=betas)
    opt.step([x])
    bad = x.clone()
    bad[300] = large   # its square is infinite
    opt.step([bad])
    for _ in range(2):
        opt.step([x])
        nan = torch.isnan(p)
        assert nan[256:512].all() and int(nan.sum()) == 256
        assert torch.isnan(opt.exp_avg_sq_scale[1]) and torch.isfinite(opt.exp_avg_sq_scale[[0, 2, 3]]).all()


def test_moments_near_the_top_of_the_range_stay_finite():
    p, x = torch.zeros(512, device="cuda"), torch.full((512,), 1e18, device="cuda")
    opt = M.AdamW([p], state_bits=8, betas=(0.9, 0.95))
    for _ in range(20):
        opt.step([x])
    assert torch.isfinite(p).all() and torch.isfinite(opt.exp_avg_sq_scale).all()

"""What the temperature costs a probability of a drafted token (derived in the test)."""
import math

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, I32 = torch.float32, torch.int32


@pytest.mark.parametrize("t", [2.175, 4.35, 8.7, 9.425, 6.475])
def test_the_temperature_costs_one_rounding(t):
    """A draft of probability p = 2^-y, y near 120, beside one certain token, with uniforms
    next to p. The kernel's exponent is d k for the logit's distance d, which is exact here,
    and k = log2(e) / T rounded to FP32 (off by `off` of it): an error of y off, half a step
    of FP32 at y (2^-18), and 2 units of the exponential. (A product of two rounded factors
    in place of k is off by 1.37 to 1.44 times 2^-24 at these temperatures.)"""
    T = float(np.float32(t))
    exact = math.log2(math.e) / T
    off = abs(float(np.float32(exact)) / exact - 1)
    d = torch.linspace(115.0, 125.0, 64).mul(T * math.log(2)).float()
    y = d.double() * exact
    p = torch.exp2(-y) / (1 + torch.exp2(-y))
    tol = math.log(2) * (y * off + 2.0 ** -18) + 2.0 ** -22 + 2.0 ** -24    # the last: the uniform's own rounding
    B = d.numel()
    target = torch.zeros(B, 2, 2)
    target[:, 0, 1] = -d
    tokens = torch.ones(B, 1, dtype=I32)
    for sign, stands in ((1, 0), (-1, 1)):
        u = (p * (1 + sign * tol)).float()[:, None]
        r = M.verify_drafts(target.to(DEV), tokens.to(DEV), u.to(DEV), torch.ones(B, 2, device=DEV), temperature=T)
        assert r["accepted"].tolist() == [stands] * B

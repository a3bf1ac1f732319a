"""Steps whose denominator sqrt(v) / sqrt(1 - beta2^t) + eps is small, down to
2^-49 with eps below it or 0: equal bit for bit to IEEE operations one by one."""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-30, 2.0 ** -40, 1e-10])
@pytest.mark.parametrize("betas", [(0.9, 0.95), (0.95, 0.999)])
def test_small_denominators(eps, betas):
    n, (b1, b2), lr = 1 << 16, betas, 1e-3
    g = torch.Generator().manual_seed(1)
    p = torch.zeros(n, device="cuda")
    opt = M.AdamW([p], lr=lr, betas=betas, eps=eps, weight_decay=0.0)
    m = v = want = torch.zeros(n, device="cuda")
    e = torch.randint(-46, 20, (n,), generator=g).float()
    for t in range(1, 4):
        x = torch.ldexp(torch.rand(n, generator=g) + 1, e).cuda() * (1 if t % 2 else -1)
        opt.step([x])
        m, v = m * b1 + x * (1 - b1), v * b2 + (x * x) * (1 - b2)
        r = v.sqrt() * (1 / math.sqrt(1 - b2 ** t)) + eps
        assert r.min() < 2.0 ** -38 + 2 * eps
        want = want - (m / r) * (lr / (1 - b1 ** t))
        assert torch.equal(opt.exp_avg[:n], m) and torch.equal(opt.exp_avg_sq[:n], v)
        assert torch.equal(p, want)

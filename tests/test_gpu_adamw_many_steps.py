"""8-bit AdamW states over many steps, against 32-bit ones, and the draws behind
them.

Bounds. Between two neighbouring E4M3 values lie 6 to 12.5% (u), so a drawn code
moves sqrt(v) by up to that, with a probability of the distance that one step
asks for, d / u: d is about (1 - beta2) / 2 for gradients as large as before, as
much again for the change of the block's scale. Per step the relative variance of
v grows by 4 u^2 (d / u) = 4 u d <= (1 - beta2) / 2, while a step forgets 1 - beta2
of it: the stationary distribution of that process is an inverse gamma one of
shape 1 + 2 / (1/2) = 5 at the worst, whose 1st and 99th percentiles are 0.43 and
3.2 times its mean: 0.65 and 1.8 for the root, which the true v's own noise
(gradients in the window of beta2) widens. Asserted: the median within 0.7 and
1.3, 98% of the elements within 0.4 and 2.5. Codes that do not move stay at 1 /
0.01 = 100 times the true value.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def values(opt, name):
    """A moment's values (sqrt(v) for the second) of an optimizer with 8-bit states."""
    s = getattr(opt, name + "_scale").repeat_interleave(256)
    return getattr(opt, name).float() * s


@pytest.mark.parametrize("beta2,before,after", [(0.96, 150, 600), (0.99, 500, 2000), (0.995, 1000, 4000),
                                                (0.999, 4000, 14000)])
def test_second_moment_follows_falling_gradients(beta2, before, after):
    n, g = 16 * 256, torch.Generator(device=DEV).manual_seed(1)
    p, q = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    a = M.AdamW([p], state_bits=8, betas=(0.9, beta2))
    b = M.AdamW([q], state_bits=32, betas=(0.9, beta2))
    small = torch.arange(n, device=DEV) % 256 >= 8
    factor = torch.where(small, 0.01, 1.0)
    for i in range(before + after):
        x = torch.randn(n, generator=g, device=DEV)
        if i >= before:
            x *= factor
        a.step([x])
        b.step([x])
    ratio = values(a, "exp_avg_sq").double() / b.exp_avg_sq.double().sqrt()
    for part in (ratio[small], ratio[~small]):
        assert 0.7 <= part.median() <= 1.3, part.median()
    assert ((ratio >= 0.4) & (ratio <= 2.5)).double().mean() >= 0.98


@pytest.mark.parametrize("beta2", [0.95, 0.99])
def test_first_moment_dies_out_without_gradients(beta2):
    """beta1 = 0.95: a parameter whose gradients stop moves by what is left of its
    first moment, some steps of lr, not on and on."""
    n, g = 16 * 256, torch.Generator(device=DEV).manual_seed(2)
    p, q = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    kinds = dict(betas=(0.95, beta2), lr=1.0, weight_decay=0.0)
    a, b = M.AdamW([p], state_bits=8, **kinds), M.AdamW([q], state_bits=32, **kinds)
    small = torch.arange(n, device=DEV) % 256 >= 8
    for i in range(2300):
        x = torch.randn(n, generator=g, device=DEV)
        if i == 300:
            p0, q0 = p.clone(), q.clone()
        if i >= 300:
            x = torch.where(small, 0.0, x)
        a.step([x])
        b.step([x])
    moved, want = (p - p0).abs()[small], (q - q0).abs()[small]
    assert moved.median() <= 2 * want.median() and moved.max() <= 4 * want.max()


@pytest.mark.parametrize("gdtype,pdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                           (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("shift", [0, 1])
def test_drawn_codes_are_neighbours_and_right_on_average(gdtype, pdtype, shift):
    """One step from zero: m = (1 - beta1) g and v = (1 - beta2) g^2. Every code is
    one of the two around the exact value, and over n elements of one value in a
    block's range their mean is within 5 standard deviations of it (a draw between
    neighbours a < b has variance (b - a)^2 / 4 at most; the block's scale, the
    quotient and the draw's 20 bits add 2^-20)."""
    blocks, beta1, beta2 = 2000, 0.97, 0.999
    n = 256 * blocks
    value = torch.logspace(0, -3.5, 255, device=DEV).to(gdtype)
    x = torch.zeros(blocks, 256, device=DEV, dtype=gdtype)
    x[:, 0] = 2.0
    x[:, 1:] = value
    x[:, 3::2] *= -1
    store = torch.zeros(n + shift, device=DEV, dtype=gdtype)
    store[shift:] = x.view(-1)
    p = torch.zeros(n + shift, device=DEV, dtype=pdtype)[shift:]
    opt = M.AdamW([p], state_bits=8, betas=(beta1, beta2))
    opt.step([store[shift:]])
    c1, c2 = torch.tensor([1 - beta1, 1 - beta2], device=DEV)
    m, v = x.float() * c1, (x.float() * x.float()) * c2
    grid = torch.arange(127, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    for name, exact in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
        code = getattr(opt, name).double().view(blocks, 256)
        want = exact.double() / getattr(opt, name + "_scale").double()[:, None]
        assert (code * want >= 0).all()
        code, want = code.abs(), want.abs()
        hi = grid[torch.searchsorted(grid, want * (1 - 2.0 ** -21)).clamp(max=126)]
        lo = grid[(torch.searchsorted(grid, want * (1 + 2.0 ** -21), right=True) - 1).clamp(min=0)]
        near = (code == hi) | (code == lo)
        assert near.all() or (name == "exp_avg_sq" and (code[~near] == 2.0 ** -9).all())
        sd = (hi - lo).amax(0) / 2 / blocks ** 0.5
        off = (code.mean(0) - want.mean(0)).abs()
        above = want[0] >= 2.0 ** -9   # below, the second moment's codes stay above zero
        assert (off <= 5 * sd + 2.0 ** -20 * want[0])[above].all(), name
        assert (code.std(0) > 0).sum() > 150   # draws, not one rounding for all


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.95, 0.95), (0.95, 0.99)])
def test_draws_are_repeatable_and_do_not_depend_on_the_grouping(betas):
    sizes = [(37 * i) % 701 + 1 for i in range(600)]
    g = torch.Generator().manual_seed(3)
    start = [torch.randn(n, generator=g) for n in sizes]
    grads = [[torch.randn(n, generator=g).cuda() for n in sizes] for _ in range(3)]

    def run(which):
        p = [start[i].cuda() for i in which]
        opt = M.AdamW(p, state_bits=8, betas=betas)
        for gs in grads:
            opt.step([gs[i] for i in which])
        return p, opt

    p, a = run(range(600))
    q, b = run(range(600))
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    for name in ("exp_avg", "exp_avg_sq"):
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8))
    for i in range(0, 600, 71):
        r, c = run([i])
        assert torch.equal(r[0], p[i])
        at = a.starts[i]
        for name in ("exp_avg", "exp_avg_sq"):
            assert torch.equal(getattr(c, name)[:sizes[i]].view(torch.uint8),
                               getattr(a, name)[at:at + sizes[i]].view(torch.uint8))

"""AdamW over many tensors against the formula, in 64 bits and, for the 8-bit
states, operation by operation in FP32 (IEEE operations in a fixed order, so
codes and scales have to be equal bit for bit).

Tolerances in 64 bits. Each FP32 operation rounds by 2^-24; m and v take three,
the step about eight more, and s steps add up: s * 12 * 2^-24 of the largest
magnitudes in a sum (|p| + lr |u| with |u| <= 10 here). A BF16 result adds half
a unit in the last place, 2^-9, at each step.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SIZES = [1, 7, 255, 256, 257, 4096, 5001, 0, 100003]
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def tensors(seed, sizes, dtype, std, shift=0):
    """Tensors of these sizes, each `shift` elements into an allocation of its own."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + shift, generator=g) * std).to(dtype).to(DEV)[shift:] for n in sizes]


def blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,copies", [(0, True), (1, False), (3, True)])
def test_three_steps(bits, pdtype, gdtype, shift, copies):
    """Every operation in FP32 by torch (no contraction): equal bit for bit, or, for
    the 32-bit states, also within the 64-bit formula's bound."""
    params = tensors(1, SIZES, pdtype, 0.5, shift)
    start = [p.clone() for p in params]
    outs = [torch.full((n + 5,), 9.0, dtype=torch.bfloat16, device=DEV) for n in SIZES]
    cp = [o[shift:shift + n] for o, n in zip(outs, SIZES)] if copies else None
    opt = M.AdamW(params, copies=cp, state_bits=bits, **HYPER)
    scale = torch.full((1,), 0.25, device=DEV)
    steps = [tensors(10 + s, SIZES, gdtype, 0.1, shift) for s in range(3)]
    for grads in steps:
        opt.step(grads, grad_scale=scale)
    b1, b2 = HYPER["betas"]
    lr, eps, wd = HYPER["lr"], HYPER["eps"], HYPER["weight_decay"]
    for i, n in enumerate(SIZES):
        p = start[i].float()
        m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        P, Mo, V = start[i].double(), m.double(), v.double()
        for s, grads in enumerate(steps):
            g = grads[i].float() * 0.25
            bc1, bc2 = 1 - b1 ** (s + 1), 1 - b2 ** (s + 1)
            m = m * b1 + g * (1 - b1)
            v = v * b2 + (g * g) * (1 - b2)
            r = v.sqrt()
            p = p * (1 - lr * wd) - (m / (r * (1 / math.sqrt(bc2)) + eps)) * (lr / bc1)
            exact_copy = p.to(torch.bfloat16)
            p = p.to(pdtype).float()
            G = grads[i].double() * 0.25
            Mo, V = b1 * Mo + (1 - b1) * G, b2 * V + (1 - b2) * G * G
            P = P * (1 - lr * wd) - lr / bc1 * Mo / ((V / bc2).sqrt() + eps)
            if bits == 8:
                mb, rb = blocks(m), blocks(r)
                sm = (mb.abs().amax(1) / 448.0).clamp(min=2.0 ** -126)
                sv = (rb.amax(1) / 448.0).clamp(min=2.0 ** -126)
                cm = (mb * (1.0 / sm)[:, None]).to(torch.float8_e4m3fn)
                cv = ((rb * (1.0 / sv)[:, None]).clamp(min=2.0 ** -9) * (rb > 0)).to(torch.float8_e4m3fn)
                m = (cm.float() * sm[:, None]).view(-1)[:n]
                v = (cv.float() * sv[:, None]).square().view(-1)[:n]
        at = opt.starts[i]
        assert torch.equal(params[i].float(), p), f"parameter {i}"
        if copies:
            assert torch.equal(cp[i], exact_copy)
            rest = outs[i].clone()
            rest[shift:shift + n] = 9.0
            assert (rest == 9.0).all()
        if bits == 8:
            if n:
                first, count = at // 256, cm.shape[0]
                assert torch.equal(opt.exp_avg_scale[first:first + count], sm)
                assert torch.equal(opt.exp_avg_sq_scale[first:first + count], sv)
                assert torch.equal(opt.exp_avg[at:at + n].view(torch.uint8), cm.view(-1)[:n].view(torch.uint8))
                assert torch.equal(opt.exp_avg_sq[at:at + n].view(torch.uint8), cv.view(-1)[:n].view(torch.uint8))
            continue
        assert torch.equal(opt.exp_avg[at:at + n], m) and torch.equal(opt.exp_avg_sq[at:at + n], v)
        lim = 3 * 12 * 2.0 ** -24 * (P.abs() + 10 * lr) + (3 * 2.0 ** -8 * (P.abs() + 10 * lr) if pdtype == torch.bfloat16 else 0)
        if pdtype == torch.float32:
            assert ((params[i].double() - P).abs() <= lim).all()
        assert ((opt.exp_avg[at:at + n].double() - Mo).abs() <= 36 * 2.0 ** -24 * 0.1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    """Results do not depend on how tensors are grouped: 1000 tensors in one
    optimizer, and each hundredth in one of its own."""
    sizes = [(37 * i) % 701 + 1 for i in range(1000)]
    params = tensors(2, sizes, torch.float32, 1.0)
    alone = [p.clone() for p in params[::100]]
    grads = tensors(3, sizes, torch.bfloat16, 0.1)
    opt = M.AdamW(params, state_bits=bits, **HYPER)
    single = [M.AdamW([p], state_bits=bits, **HYPER) for p in alone]
    for _ in range(2):
        opt.step(grads)
        for o, g in zip(single, grads[::100]):
            o.step([g])
    for i, (p, o) in enumerate(zip(alone, single)):
        assert torch.equal(p, params[100 * i])
        at, n = opt.starts[100 * i], sizes[100 * i]
        for name in ("exp_avg", "exp_avg_sq"):
            a, b = getattr(o, name)[:n], getattr(opt, name)[at:at + n]
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_continuing_from_a_saved_state():
    params = tensors(4, [300, 5000], torch.float32, 1.0)
    grads = [tensors(5 + s, [300, 5000], torch.float32, 0.1) for s in range(4)]
    twin = [p.clone() for p in params]
    a = M.AdamW(params, state_bits=8, **HYPER)
    for g in grads:
        a.step(g)
    b = M.AdamW(twin, state_bits=8, **HYPER)
    b.step(grads[0])
    b.step(grads[1])
    names = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    c = M.AdamW(twin, state_bits=8, state={**{k: getattr(b, k).clone() for k in names}, "step": 2}, **HYPER)
    c.step(grads[2])
    c.step(grads[3])
    assert c.step_count == 4
    for p, q in zip(params, twin):
        assert torch.equal(p, q)


def test_zero_gradients_and_a_small_second_moment():
    """Without gradients a fresh state only decays the parameter; a second moment
    far below its block's largest keeps a code above zero, so the step stays bounded."""
    p = torch.ones(512, device=DEV)
    opt = M.AdamW([p], state_bits=8, lr=0.1, weight_decay=0.5, betas=(0.9, 0.99))
    opt.step([torch.zeros(512, device=DEV)])
    assert torch.equal(p, torch.full_like(p, 1 - 0.1 * 0.5))
    assert (opt.exp_avg.view(torch.uint8) == 0).all() and (opt.exp_avg_sq.view(torch.uint8) == 0).all()
    g = torch.full((512,), 1e-6, device=DEV)
    g[0] = 1e3
    before = p.clone()
    opt.step([g])
    assert (opt.exp_avg_sq.view(torch.uint8)[:256] > 0).all()
    opt.step([torch.zeros(512, device=DEV)])
    opt.step([torch.zeros(512, device=DEV)])
    assert torch.isfinite(p).all() and ((p - before).abs() < 10).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_nan_gradient_stays_in_its_place(bits):
    """32-bit states: its element; 8-bit states: its block of 256 from the next step on."""
    p = tensors(6, [1024], torch.float32, 1.0)
    opt = M.AdamW(p, state_bits=bits, **HYPER)
    g = tensors(7, [1024], torch.float32, 0.1)[0]
    opt.step([g])
    g[300] = float("nan")
    opt.step([g])
    bad = torch.isnan(p[0])
    assert bad[300] and int(bad.sum()) == 1
    g[300] = 0.0
    opt.step([g])
    bad = torch.isnan(p[0])
    if bits == 32:
        assert int(bad.sum()) == 1
    else:
        assert bad[256:512].all() and int(bad.sum()) == 256


def test_another_stream_and_lr_override():
    p = tensors(8, [70000], torch.float32, 1.0)
    q = [p[0].clone()]
    g = tensors(9, [70000], torch.bfloat16, 0.1)
    a, b = M.AdamW(p, **HYPER), M.AdamW(q, **{**HYPER, "lr": 0.5})
    a.step(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.step(g, lr=HYPER["lr"], stream=s)
    s.synchronize()
    assert torch.equal(p[0], q[0])


def test_roots_and_quotients_are_the_ieee_ones():
    c = torch.zeros(2, dtype=torch.int64, device=DEV)
    M.minite_test_adamw_math(c)
    assert c.tolist() == [0, 0]


def test_moments_outside_the_usual_range():
    """Second moments from 2^-140 to 2^120 and zero, in one block: the same
    operations as anywhere else (the usual range takes another path)."""
    n = 512
    g = torch.ldexp(torch.ones(n), torch.randint(-70, 60, (n,), generator=torch.Generator().manual_seed(3)).float())
    g[::7] = 0.0
    g = g.to(DEV)
    p = torch.zeros(n, device=DEV)
    opt = M.AdamW([p], state_bits=32, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0)
    opt.step([g])
    m, v = g * (1 - 0.9), (g * g) * (1 - 0.95)
    want = -(m / (v.sqrt() * (1 / math.sqrt(1 - 0.95)) + 1e-8)) * (1e-3 / (1 - 0.9))
    assert torch.equal(opt.exp_avg[:n], m) and torch.equal(opt.exp_avg_sq[:n], v)
    assert torch.equal(p, want)


def test_refusals():
    p = [torch.zeros(8, device=DEV)]
    opt = M.AdamW(p)
    for bad in ([], [torch.zeros(7, device=DEV)], [torch.zeros(8)],
                [torch.zeros(8, device=DEV, dtype=torch.float16)], [torch.zeros(16, device=DEV)[::2]]):
        with pytest.raises(M.MiniteError):
            opt.step(bad)
    assert opt.step_count == 0
    for make in (lambda: M.AdamW([]), lambda: M.AdamW(p, state_bits=16), lambda: M.AdamW([torch.zeros(8)]),
                 lambda: M.AdamW([p[0], torch.zeros(8, device=DEV, dtype=torch.bfloat16)]),
                 lambda: M.AdamW([torch.zeros((8, 8), device=DEV).t()[:, :4]]),
                 lambda: M.AdamW(p, copies=[torch.zeros(8, device=DEV)]),
                 lambda: M.AdamW(p, betas=(1.0, 0.9)).step([torch.zeros(8, device=DEV)])):
        with pytest.raises(M.MiniteError):
            make()

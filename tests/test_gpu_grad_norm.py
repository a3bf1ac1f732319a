"""The global gradient norm, its clipping factor and clipped gradients against 64
bits.

Tolerances. At most 16 squares follow one another in FP32 (64 where they had to be
scaled), all positive, each addition off by 2^-24 of the sum, three more additions
join the four chains; the rest is in 64 bits. The root halves it: 10 * 2^-24 (34 *
2^-24 scaled), and one rounding to FP32. The factor takes the norm's error and one
rounding. A clipped element is one FP32 product and one rounding to its type.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NEAR, SCALED = 12 * 2.0 ** -24, 36 * 2.0 ** -24


def tensors(seed, sizes, types, std=1e-3, shift=0):
    """Tensors of a flat buffer each, the first element `shift` in."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + shift, generator=g) * std).to(t).to(DEV)[shift:] for n, t in zip(sizes, types)]


def exact(grads, order):
    if order == 2:
        return math.sqrt(sum(float(torch.dot(g.double().view(-1), g.double().view(-1))) for g in grads))
    return max([float(g.double().abs().max()) for g in grads if g.numel()], default=0.0)


SIZES = [[1], [7], [0, 3, 0], [255, 256, 257], [4096] * 20, [8191, 1, 16385, 32768, 5], [524288], [524289],
         [100] * 33, [17, 100000] * 80, [3] * 1001 + [70000], [3_000_000, 1], [20_000_003]]


@pytest.mark.parametrize("order", [2.0, math.inf])
@pytest.mark.parametrize("types", [[BF], [F32], [BF, F32]], ids=["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("shift", [0, 1, 13])
def test_norm_and_factor(sizes, types, order, shift):
    grads = tensors(len(sizes), sizes, types * len(sizes), shift=shift)
    want = exact(grads, order)
    for max_norm in (math.inf, want / 3, 0.0):
        r = M.grad_norm(grads, max_norm=max_norm, order=order)
        got, factor = float(r["norm"]), float(r["scale"])
        assert abs(got - want) <= (NEAR if order == 2 else 0) * want
        f = min(1.0, max_norm / (want + 1e-6))
        assert abs(factor - f) <= (NEAR + 2.0 ** -24) * f
    again = M.grad_norm(grads, order=order)
    assert float(again["norm"]) == got   # the same call, the same bits


@pytest.mark.parametrize("n", [1000, 3_000_000])
@pytest.mark.parametrize("size", [1e-45, 1e-40, 3e-38, 1e-25, 1e-15, 1e-12, 1e8, 1e18, 1e25, 1e38])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sizes_whose_squares_leave_fp32(size, n, dtype):
    g = torch.Generator().manual_seed(2)
    x = (torch.rand(n, generator=g, dtype=torch.float64) + 0.5).mul_(size).to(dtype).to(DEV)
    want = exact([x], 2)
    got = float(M.grad_norm([x])["norm"])
    if want > 3.4028235e38:
        assert got == math.inf
    else:
        assert abs(got - want) <= SCALED * want + 2.0 ** -150
    assert float(M.grad_norm([x], order=math.inf)["norm"]) == float(x.double().abs().max())


def test_large_and_small_gradients_side_by_side():
    x = torch.zeros(2_000_000, device=DEV)
    x[::7], x[5], x[1_999_999] = 1e-30, 3.0, 4.0
    assert abs(float(M.grad_norm([x])["norm"]) - 5.0) <= NEAR * 5
    assert float(M.grad_norm([torch.zeros(999, device=DEV)], max_norm=1.0)["norm"]) == 0.0


@pytest.mark.parametrize("n", [5, 3_000_000])
@pytest.mark.parametrize("order", [2.0, math.inf])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_non_finite_gradients(n, order, dtype):
    for bad, want, factor in ((math.inf, math.inf, 0.0), (-math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)):
        for at in (0, n // 2, n - 1):
            x = torch.full((n,), 0.5, dtype=dtype, device=DEV)
            x[at] = bad
            r = M.grad_norm([torch.ones(3, device=DEV), x], max_norm=1.0, order=order)
            for got, w in ((float(r["norm"]), want), (float(r["scale"]), factor)):
                assert got == w or (math.isnan(got) and math.isnan(w))


def test_without_a_limit_the_factor_is_one():
    for n in (10, 3_000_000):
        x = torch.ones(n, device=DEV)
        for bad, factor in ((1.0, 1.0), (math.inf, 1.0), (math.nan, math.nan)):
            x[n // 3] = bad
            got = float(M.grad_norm([x])["scale"])
            assert got == factor or (math.isnan(got) and math.isnan(factor))


def test_no_elements():
    r = M.grad_norm([torch.empty(0, device=DEV)], max_norm=2.0)
    assert float(r["norm"]) == 0.0 and float(r["scale"]) == 1.0


@pytest.mark.parametrize("gtype", [BF, F32])
@pytest.mark.parametrize("otype", [BF, F32])
@pytest.mark.parametrize("sizes", [[1], [1000, 7, 33000], [3] * 1001, [5_000_000]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("gshift,oshift", [(0, 0), (1, 0), (0, 3), (5, 5)])
def test_clipped_into_other_tensors(gtype, otype, sizes, gshift, oshift):
    grads = tensors(1, sizes, [gtype] * len(sizes), shift=gshift)
    flat = [torch.full((n + oshift + 2,), 9.0, dtype=otype, device=DEV) for n in sizes]
    out = [f[oshift: oshift + n] for f, n in zip(flat, sizes)]
    before = [g.clone() for g in grads]
    want = exact(grads, 2)
    r = M.clip_grads(grads, want / 2, out=out)
    f = float(r["scale"])
    assert abs(f - want / 2 / (want + 1e-6)) <= (NEAR + 2.0 ** -24)
    for g, b, o, whole in zip(grads, before, out, flat):
        assert torch.equal(g, b)
        assert torch.equal(o, (b.float() * f).to(otype))     # one product, one rounding
        assert (whole[:oshift] == 9).all() and (whole[oshift + o.numel():] == 9).all()


@pytest.mark.parametrize("types", [[BF], [F32], [BF, F32]])
def test_clipped_in_place(types):
    sizes = [100, 70000, 1, 3_000_001]
    grads = tensors(4, sizes, types * 4)
    before = [g.clone() for g in grads]
    n = exact(grads, 2)
    assert float(M.clip_grads(grads, 2 * n)["scale"]) == 1.0
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    f = float(M.clip_grads(grads, n / 10)["scale"])
    assert all(torch.equal(g, (b.float() * f).to(b.dtype)) for g, b in zip(grads, before))
    assert abs(exact(grads, 2) - n / 10) <= n / 10 * 2.0 ** -9 + 1e-6


def test_a_factor_of_nan_reaches_the_gradients():
    x = torch.ones(10, device=DEV)
    x[3] = math.nan
    M.clip_grads([x], 1.0)
    assert torch.isnan(x).all()


def test_streams_and_graphs():
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = tensors(1, [3_000_000], [F32])[0], tensors(2, [4_000_000], [BF])[0]
    torch.cuda.synchronize()
    for _ in range(5):
        ra, rb = M.grad_norm([a], stream=one), M.grad_norm([b], stream=two)
    torch.cuda.synchronize()
    assert abs(float(ra["norm"]) / exact([a], 2) - 1) <= NEAR and abs(float(rb["norm"]) / exact([b], 2) - 1) <= NEAR
    x = [torch.zeros_like(a), torch.zeros(50, dtype=BF, device=DEV)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = M.clip_grads(x, 1.0)
    for scale in (1.0, 1e3, 1e-3):
        x[0].copy_(a * scale)
        x[1].fill_(scale)
        n = exact(x, 2)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(r["norm"]) - n) <= NEAR * n
        assert exact(x, 2) <= min(n, 1.0) * (1 + 2.0 ** -8)


def test_more_than_two_to_the_31_elements():
    x = torch.zeros((1 << 31) + 4096 * 3, dtype=BF, device=DEV)
    x[0], x[1 << 31], x[-1] = 2.0, 3.0, 6.0
    assert float(M.grad_norm([x])["norm"]) == 7.0
    M.clip_grads([x], 3.5)
    assert [round(float(v), 3) for v in (x[0], x[1 << 31], x[-1])] == [1.0, 1.5, 3.0]

"""BF16 products grouped by expert against 64-bit products.

Tolerances. A product of two BF16 values is exact in FP32. Every K = 16 step
adds its products to the running sum with an error of at most 2^-22 of the
magnitudes summed so far (the alignment of the 16 products and the truncated
result, 2^-23 each), so a sum of n values is within ceil(n / 16) 2^-22
sum |a b|. FP32 outputs are summed in chunks of 256 values that are added in
FP32 (round to nearest, 2^-24 each): 16 * 2^-22 + ceil(n / 256) 2^-24. A BF16
output adds half a unit in the last place, 2^-9 of the result (twice that here,
for a result that the error above moves over a rounding boundary).
"""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).to(DEV)


def check(got, exact, mag, n, what):
    got = got.double()
    if got.numel() == 0:
        return
    steps = -(-n // 16)
    lim = mag * (min(steps, 16) * 2.0 ** -22 + -(-n // 256) * 2.0 ** -24)
    if what[0] == torch.bfloat16:
        lim = mag * (steps * 2.0 ** -22) + exact.abs() * 2.0 ** -8
    bad = ~((got - exact).abs() <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{((got - exact).abs() / lim.clamp(min=1e-300)).max().item():.2f} times the bound"


CASES = [  # rows of each expert, N, K
    ([1], 8, 8),
    ([1], 1536, 2048),
    ([0, 0, 3, 0], 16, 24),
    ([5, 0, 130, 1, 64], 200, 136),
    ([127, 128, 129], 264, 72),
    ([300, 1], 256, 64),
    ([17, 0, 0, 500, 33, 2, 0], 520, 1000),
    ([700], 248, 2056),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_forward_and_activation_gradient(counts, N, K, stored, out_dtype):
    m, e = sum(counts), len(counts)
    x, w = randn(1, m, K), randn(2, e, K, N) if stored else randn(2, e, N, K)
    off = offsets_of(counts)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = M.grouped_gemm_bf16(x, w, off, w_as_stored=stored, out_dtype=out_dtype, status=status)
    at = 0
    for i, c in enumerate(counts):
        a, b = x[at:at + c].double(), w[i].double()
        b = b if stored else b.t()
        check(out[at:at + c], a @ b, a.abs() @ b.abs(), K, (out_dtype, i, c))
        at += c
    assert int(status.item()) == 0


@pytest.mark.parametrize("kind", ["bfloat16", "float32", "accumulate"])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_weight_gradient(counts, N, K, kind):
    m, e = sum(counts), len(counts)
    dy, x = randn(3, m, N), randn(4, m, K)
    dtype = torch.bfloat16 if kind == "bfloat16" else torch.float32
    before = torch.randn(e, N, K, generator=torch.Generator().manual_seed(5)).to(DEV)
    acc = kind == "accumulate"
    out = before.clone() if acc else torch.full((e, N, K), float("nan"), device=DEV, dtype=dtype)
    got = M.grouped_wgrad_bf16(dy, x, offsets_of(counts), out=out, accumulate=acc)
    assert got is out
    at = 0
    for i, c in enumerate(counts):
        a, b = dy[at:at + c].double().t(), x[at:at + c].double()
        exact, mag = a @ b, a.abs() @ b.abs()
        if acc:  # one more FP32 rounding of the sum, 2^-24 (2^-23 of the magnitudes covers it)
            exact = exact + before[i].double()
            mag = mag + 2 * before[i].double().abs()
        check(out[i], exact, mag, max(c, 1), (dtype, i, c))
        if c == 0:
            assert torch.equal(out[i], before[i] if acc else torch.zeros_like(out[i]))
        at += c


@pytest.mark.parametrize("mode", ["forward", "stored", "wgrad"])
@pytest.mark.parametrize("E,N,K,seed", [(37, 256, 64, 0), (300, 520, 136, 1), (1024, 72, 72, 2), (5, 1280, 320, 3)])
def test_random_routings(mode, E, N, K, seed):
    """Experts of 0 to about 900 rows: every way a cluster's pairs share a tile,
    every number of rows in a tile, and tables too long for all stages."""
    g = torch.Generator().manual_seed(seed)
    counts = (900 * torch.rand(E, generator=g) ** (6 if E > 100 else 1)).long()
    counts[::5] = 0
    counts = counts.tolist()
    off, m = offsets_of(counts), sum(counts)
    x = randn(seed + 50, m, K)
    if mode == "wgrad":
        dy = randn(seed + 51, m, N)
        got = M.grouped_wgrad_bf16(dy, x, off)
    else:
        w = randn(seed + 52, E, K, N) if mode == "stored" else randn(seed + 52, E, N, K)
        got = M.grouped_gemm_bf16(x, w, off, w_as_stored=mode == "stored", out_dtype=torch.float32)
    at = 0
    for e, c in enumerate(counts):
        r = slice(at, at + c)
        if mode == "wgrad":
            a, b, n, res = dy[r].double().t(), x[r].double(), max(c, 1), got[e]
        else:
            a, b, n, res = x[r].double(), w[e].double() if mode == "stored" else w[e].double().t(), K, got[r]
        check(res, a @ b, a.abs() @ b.abs(), n, (torch.float32, e, c))
        at += c


def test_more_units_of_work_than_are_listed():
    """160000 rows x 2048 features: over 64 units for each cluster."""
    counts, N, K = [100000, 59993, 7], 2048, 64
    x, w, off = randn(60, sum(counts), K), randn(61, 3, N, K), offsets_of(counts)
    out = M.grouped_gemm_bf16(x, w, off, out_dtype=torch.float32)
    for e, lo, hi in ((0, 0, 100000), (1, 100000, 159993), (2, 159993, 160000)):
        for a in range(lo, hi, 20000):
            r = slice(a, min(hi, a + 20000))
            A, B = x[r].double(), w[e].double().t()
            check(out[r], A @ B, A.abs() @ B.abs(), K, (torch.float32, e, a))


def test_long_sums_of_one_sign():
    """65536 positive products: what the tensor cores' sums lose at every step all
    goes one way, and the chunks keep it to a chunk's worth."""
    n = 65536
    a, b = randn(62, n, 64).abs(), randn(63, n, 128).abs()
    exact = a.double().t() @ b.double()
    check(M.grouped_wgrad_bf16(a, b, offsets_of([n]))[0], exact, exact, n, (torch.float32,))
    x, w = a.t().contiguous(), b.t().contiguous()[None]
    check(M.grouped_gemm_bf16(x, w, offsets_of([64]), out_dtype=torch.float32), exact, exact, n, (torch.float32,))


@pytest.mark.parametrize("mode", ["forward", "stored", "wgrad"])
def test_an_experts_values_do_not_reach_another(mode):
    """NaN and infinities in one expert's rows and weight stay with it, also where
    a tile or a sum's tail reads past an expert's end."""
    counts, N, K = [37, 70, 5], 72, 40
    off, m = offsets_of(counts), sum(counts)
    x, dy = randn(6, m, K), randn(7, m, N)
    w = randn(8, 3, K, N) if mode == "stored" else randn(8, 3, N, K)
    bad = [t.clone() for t in (x, dy, w)]
    bad[0][37:107] = float("nan")
    bad[1][37:107] = float("inf")
    bad[2][1] = float("nan")
    if mode == "wgrad":
        ref = M.grouped_wgrad_bf16(dy, x, off)
        got = M.grouped_wgrad_bf16(bad[1], bad[0], off)
        for e in (0, 2):
            assert torch.equal(got[e], ref[e])
        assert torch.isnan(got[1]).all()
    else:
        ref = M.grouped_gemm_bf16(x, w, off, w_as_stored=mode == "stored")
        got = M.grouped_gemm_bf16(bad[0], bad[2], off, w_as_stored=mode == "stored")
        assert torch.equal(got[:37], ref[:37]) and torch.equal(got[107:], ref[107:])
        assert torch.isnan(got[37:107]).all()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_strides_and_nothing_written_outside(out_dtype):
    counts, N, K = [50, 0, 83], 136, 200
    m = 150  # rows past the last expert's stay untouched
    off = offsets_of(counts)
    wide = randn(9, m, K + 56)
    x = wide[:, 24:24 + K]
    w = randn(10, 3, N, K)
    big = torch.full((m + 2, N + 24), 7.0, device=DEV, dtype=out_dtype)
    out = big[1:m + 1, 8:8 + N]
    M.grouped_gemm_bf16(x, w, off, out=out)
    ref = M.grouped_gemm_bf16(x.contiguous(), w, off, out_dtype=out_dtype)
    assert torch.equal(out[:133], ref[:133])
    big[1:134, 8:8 + N] = 7.0
    assert (big == 7.0).all()
    dy = randn(11, m, N + 8)[:, 8:]
    got = M.grouped_wgrad_bf16(dy, x, off)
    assert torch.equal(got, M.grouped_wgrad_bf16(dy.contiguous(), x.contiguous(), off))


def test_a_rows_result_does_not_depend_on_the_batch():
    K, N = 320, 384
    w = randn(12, 2, N, K)
    x = randn(13, 600, K)
    a = M.grouped_gemm_bf16(x, w, offsets_of([400, 200]))
    b = M.grouped_gemm_bf16(x[390:410].contiguous(), w, offsets_of([10, 10]))
    assert torch.equal(a[390:410], b)


def test_gradients_against_differences():
    """The product is bilinear: L(w + d) - L(w) = <dw, d> exactly, for steps d
    that keep w + d a BF16 value. Differences of FP32 results, so the bound is
    the sum of both sides' rounding: 2^-17 of the magnitudes for each product
    (K = 320 in chunks, from the bound above, 2^-18, both sides)."""
    counts, N, K = [40, 3, 90], 48, 320
    off, m = offsets_of(counts), sum(counts)
    x, w, dy = randn(14, m, K), randn(15, 3, N, K), randn(16, m, N)
    f32 = torch.float32

    def loss(x_, w_):
        return (M.grouped_gemm_bf16(x_, w_, off, out_dtype=f32).double() * dy.double()).sum()

    mag = (M.grouped_gemm_bf16(x.abs(), w.abs(), off, out_dtype=f32).double() * dy.double().abs()).sum()
    dw = M.grouped_wgrad_bf16(dy, x, off)
    dx = M.grouped_gemm_bf16(dy, w, off, w_as_stored=True, out_dtype=f32)
    for t, grad, f in ((w, dw, lambda s: loss(x, s)), (x, dx, lambda s: loss(s, w))):
        step = (t.float() * 0.5).to(torch.bfloat16)          # t + t / 2 is rounded once, here
        moved = (t.float() + step.float()).to(torch.bfloat16)
        d = moved.double() - t.double()
        assert abs((f(moved) - f(t)) - (grad.double() * d).sum()) <= 4 * 2.0 ** -17 * mag


def test_bad_offsets_write_nothing_and_set_the_status():
    x, w = randn(17, 64, 64), randn(18, 2, 64, 64)
    for bad in ([0, 40, 30], [1, 20, 64], [0, 20, 65]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full((64, 64), 5.0, device=DEV, dtype=torch.bfloat16)
        M.grouped_gemm_bf16(x, w, off, out=out, status=status)
        assert int(status.item()) == 1 << 1 and (out == 5.0).all()
        status.zero_()
        dw = torch.full((2, 64, 64), 5.0, device=DEV)
        M.grouped_wgrad_bf16(x, x, off, out=dw, status=status)
        assert int(status.item()) == 1 << 1 and (dw == 5.0).all()


def test_no_rows_at_all():
    w = randn(19, 3, 64, 32)
    x = torch.empty((0, 32), device=DEV, dtype=torch.bfloat16)
    dy = torch.empty((0, 64), device=DEV, dtype=torch.bfloat16)
    off = offsets_of([0, 0, 0])
    assert M.grouped_gemm_bf16(x, w, off).shape == (0, 64)
    assert (M.grouped_wgrad_bf16(dy, x, off) == 0).all()
    some = randn(20, 16, 32)   # rows, all of them past the last expert's
    out = torch.full((16, 64), 3.0, device=DEV, dtype=torch.bfloat16)
    M.grouped_gemm_bf16(some, w, off, out=out)
    assert (out == 3.0).all()


def test_another_stream():
    counts = [200, 56]
    x, w, off = randn(21, 256, 512), randn(22, 2, 640, 512), offsets_of(counts)
    ref = M.grouped_gemm_bf16(x, w, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.grouped_gemm_bf16(x, w, off, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)


def test_a_wait_that_runs_out_is_reported():
    """A budget of one nanosecond: the call still ends, with the status bit."""
    x, w, off = randn(23, 4096, 2048), randn(24, 1, 1024, 2048), offsets_of([4096])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.minite_set_wait_budget_ns(1)
    try:
        M.grouped_gemm_bf16(x, w, off, status=status)
        torch.cuda.synchronize()
    finally:
        M.minite_set_wait_budget_ns(0)
    assert int(status.item()) in (0, 1 << M.ERR_TIMEOUT)
    got = M.grouped_gemm_bf16(x, w, off)
    torch.cuda.synchronize()
    check(got, x.double() @ w[0].double().t(), x.double().abs() @ w[0].double().abs().t(), 2048,
          (torch.bfloat16,))

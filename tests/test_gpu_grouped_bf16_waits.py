"""BF16 products grouped by expert whose pipeline waits run out: the call ends with
exactly the timeout bit in its status, and the next call on the same operands
gives what it gave before.

A budget of one nanosecond ends a wait at its second failed attempt. An attempt
may itself sleep for some microseconds in the hardware, so a wait that is over
by then does not run out. The epilogue of a BF16 product waits for the whole sum
of a tile: 128 blocks of 64 values take at least 30 microseconds. FP32 products
have short waits alone (sums of four blocks), so that such a call may also be
complete: then its result has to be the right one.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).to(DEV)


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)


def out_of_time(call, surely=True):
    """The call with the default budget, with one nanosecond, and again."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = call(status).clone()
    assert int(status.item()) == 0
    for _ in range(3):
        status.zero_()
        M.minite_set_wait_budget_ns(1)
        try:
            got = call(status)
            torch.cuda.synchronize()
        finally:
            M.minite_set_wait_budget_ns(0)
        if surely or int(status.item()) != 0:
            assert int(status.item()) == 1 << M.ERR_TIMEOUT
        else:
            assert torch.equal(got, want)
        status.zero_()
        assert torch.equal(call(status), want)
        assert int(status.item()) == 0


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("counts", [[4096], [1], [700, 0, 33, 257, 5]])
def test_products(counts, stored, out_dtype):
    N, K, e = 1032, 8192, len(counts)
    x, off = randn(1, sum(counts), K), offsets_of(counts)
    w = randn(2, e, K, N) if stored else randn(2, e, N, K)
    out_of_time(lambda st: M.grouped_gemm_bf16(x, w, off, w_as_stored=stored, out_dtype=out_dtype, status=st),
                surely=out_dtype == torch.bfloat16)


@pytest.mark.parametrize("counts", [[4101], [3000, 0, 33, 2057, 5], [2048, 2048]])
@pytest.mark.parametrize("kind", ["bfloat16", "float32", "accumulate"])
def test_weight_gradients(kind, counts):
    """The odd CTA's tail waits for all of an expert's sum where that does not end
    on a step of 16 rows (64 blocks take at least 16 microseconds), and so does a
    BF16 result's epilogue."""
    N, K, e = 520, 1032, len(counts)
    dy, x, off = randn(3, sum(counts), N), randn(4, sum(counts), K), offsets_of(counts)
    before = torch.randn(e, N, K, generator=torch.Generator().manual_seed(5)).to(DEV)
    dtype = torch.bfloat16 if kind == "bfloat16" else torch.float32

    def call(st):
        out = before.clone() if kind == "accumulate" else None
        return M.grouped_wgrad_bf16(dy, x, off, out=out, out_dtype=dtype, accumulate=kind == "accumulate",
                                    status=st)

    out_of_time(call, surely=kind == "bfloat16" or any(c % 16 for c in counts))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_length_of_a_sum_uses_up_no_budget(dtype):
    """2^25 - 7 rows in one sum, 0.1 s at least, with 20 ms for each wait: no wait is
    for more than some blocks, but for the odd CTA's tail, which has more time."""
    n = (1 << 25) - 7
    a = torch.ones(n, 8, device=DEV, dtype=torch.bfloat16)
    b = torch.ones(n, 16, device=DEV, dtype=torch.bfloat16)
    a[::3], b[1::2] = 0.5, 0.25
    off, status = offsets_of([n]), torch.zeros(1, dtype=torch.int32, device=DEV)
    want = M.grouped_wgrad_bf16(a, b, off, out_dtype=dtype)
    M.minite_set_wait_budget_ns(20_000_000)
    try:
        got = M.grouped_wgrad_bf16(a, b, off, out_dtype=dtype, status=status)
        torch.cuda.synchronize()
    finally:
        M.minite_set_wait_budget_ns(0)
    assert int(status.item()) == 0 and torch.equal(got, want)

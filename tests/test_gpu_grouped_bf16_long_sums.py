"""BF16 results of very long sums, and calls repeated.

Tolerance. The tensor cores lose up to 2^-22 of the running sum at each step of 16
values, always towards zero. A BF16 result's sums are split after 16384 values:
1024 steps, 2^-12, then FP32 additions, round to nearest, of up to 2^11 parts
(2^-24 each, as random as a walk: below 2^-15), and half a unit of BF16, 2^-8 of the
result at most."""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -15


def positive(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(*shape, generator=g, device=DEV).add_(0.5).to(torch.bfloat16)


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("counts", [[1 << 25], [(1 << 25) - 7, 3, 0, 65536, 65537, 100]])
def test_weight_gradient(counts):
    off = offsets_of(counts)
    a, b = positive(1, sum(counts), 8), positive(2, sum(counts), 16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = M.grouped_wgrad_bf16(a, b, off, out_dtype=torch.bfloat16, status=status).double()
    assert int(status.item()) == 0
    at = 0
    for e, n in enumerate(counts):
        want = torch.zeros(8, 16, dtype=torch.float64, device=DEV)
        for lo in range(at, at + n, 1 << 22):
            part = slice(lo, min(at + n, lo + (1 << 22)))
            want += a[part].double().t() @ b[part].double()
        at += n
        assert ((got[e] - want).abs() <= TOL * want).all(), (e, ((got[e] - want) / want).abs().max().item())


@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 40], 136, 1 << 18), ([300], 264, 65536 + 64), ([70, 1], 8, 65536)])
def test_products(counts, N, K, stored):
    e, off = len(counts), offsets_of(counts)
    x, w = positive(3, sum(counts), K), positive(4, e, K, N) if stored else positive(4, e, N, K)
    got, at = M.grouped_gemm_bf16(x, w, off, w_as_stored=stored).double(), 0
    for i, n in enumerate(counts):
        wi = w[i].double() if stored else w[i].double().t()
        want = x[at:at + n].double() @ wi
        assert ((got[at:at + n] - want).abs() <= TOL * want).all()
        at += n


@pytest.mark.parametrize("kind", ["forward", "activation gradient", "weight gradient"])
def test_the_same_call_gives_the_same_bits(kind):
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 500, (64,), generator=g).tolist()
    off, m, N, K = offsets_of(counts), sum(counts), 1536, 512
    x, w = positive(6, m, K) - 1, positive(7, 64, N, K) - 1
    dy = positive(8, m, N) - 1
    call = {"forward": lambda: M.grouped_gemm_bf16(x, w, off),
            "activation gradient": lambda: M.grouped_gemm_bf16(dy, w, off, w_as_stored=True),
            "weight gradient": lambda: M.grouped_wgrad_bf16(dy, x, off)}[kind]
    want = call()
    for _ in range(20):
        assert torch.equal(call(), want)

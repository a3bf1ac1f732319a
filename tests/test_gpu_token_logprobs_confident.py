"""Log probabilities and entropies of tokens whose probability is almost 1: both
are small numbers, and have to keep their relative accuracy.

Derivation of the bound. With r = sum over all tokens but the likeliest of
exp(y), log p = -log1p(r) at that token and H = log1p(r) - t / (1 + r), both of
r's order. A term's exponent carries three roundings (the difference, the factor
1/T, the product), a relative error of 3 |y| 2^-24 in its exponential, which adds
2^-22 of its own; sums are at most V / 256 + 64 additions long on a thread's way
to the row, each with 2^-24; the logarithm and the last steps take 8 more. H adds
one product a term and a quotient, which the doubled bound covers.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu


def _rows(dtype, vocab, temperature, masked, seed):
    """Rows whose first-listed token leads by a growing margin."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    margins = torch.arange(8.0, 40.0, 1.0, device="cuda")
    n = margins.numel()
    x = torch.randn(n, vocab, generator=g, device="cuda")
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    if masked:
        x[:, torch.rand(vocab, generator=g, device="cuda") < 0.5] = float("-inf")
    x.scatter_(1, y.long()[:, None], (margins * temperature)[:, None])
    return x.to(dtype), y


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [33, 1000, 32003, 131072, 200001])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows", [1, 32])
def test_confident_tokens_keep_relative_accuracy(dtype, vocab, masked, rows):
    temperature = 0.8
    x, y = _rows(dtype, vocab, temperature, masked, vocab + rows)
    for at in range(0, x.shape[0], rows if rows > 1 else 5):
        xs, ys = x[at:at + rows].contiguous(), y[at:at + rows].contiguous()
        got = M.token_logprobs(xs, ys, temperature=temperature, alternatives=min(5, vocab))
        d = (xs.double() - xs.double().amax(1, keepdim=True)) / temperature
        top = d == 0
        assert (top.sum(1) == 1).all() and top.gather(1, ys.long()[:, None]).all()
        e = torch.where(top, 0.0, d.exp())
        r = e.sum(1)
        lp = -torch.log1p(r)
        h = torch.log1p(r) - torch.where(e > 0, d * e, 0.0).sum(1) / (1 + r)
        # terms below 2^-126 may be dropped
        far = -torch.where(e > 0, d, 0.0).amin(1)
        bound = (3 * far + 4 + vocab / 256 + 64 + 8) * 2.0 ** -24
        slack = vocab * 2.0 ** -126
        assert ((got["logprob"].double() - lp).abs() <= bound * lp.abs() + slack).all()
        assert ((got["entropy"].double() - h).abs() <= 2 * bound * h + 200 * slack).all()
        # the likeliest alternative is the token itself
        assert ((got["alt_logprobs"][:, 0].double() - lp).abs() <= bound * lp.abs() + slack).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_confident_tokens_do_not_depend_on_the_batch(dtype):
    x, y = _rows(dtype, 131072, 0.8, True, 5)
    full = M.token_logprobs(x, y, temperature=0.8)
    for i in (0, 7, 31):
        one = M.token_logprobs(x[i:i + 1], y[i:i + 1], temperature=0.8)
        assert torch.equal(one["logprob"], full["logprob"][i:i + 1])
        assert torch.equal(one["entropy"], full["entropy"][i:i + 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tied_maxima_share_the_probability(dtype):
    x = torch.full((3, 5003), -60.0, device="cuda", dtype=dtype)
    x[0, 100] = x[0, 101] = 5.0            # two in one vector
    x[1, 0] = x[1, 5002] = 5.0             # first and last
    x[2, 7::16] = 5.0                      # many threads
    n = (x == 5.0).sum(1).double()
    y = torch.tensor([101, 5002, 7], device="cuda", dtype=torch.int32)
    got = M.token_logprobs(x, y)
    bound = (8 + 5003 / 256 + 64) * 2.0 ** -24
    assert ((got["logprob"].double() + n.log()).abs() <= bound * n.log()).all()
    assert ((got["entropy"].double() - n.log()).abs() <= 2 * bound * n.log()).all()


@pytest.mark.parametrize("vocab", [33, 1000, 32003, 131072])
@pytest.mark.parametrize("offset", [0, 1])
def test_gradient_at_confident_tokens_keeps_relative_accuracy(vocab, offset):
    """At the target, d = (g_lp (1 - p) - g_H p (log p + H)) / T: each of the three
    numbers 1 - p, log p and H carries the bound above (H twice), and the result
    one rounding."""
    dtype, temperature = torch.float32, 0.8
    x, y = _rows(dtype, vocab, temperature, False, 3 * vocab)
    n = x.shape[0]
    if offset:   # rows that start off a 16-byte boundary
        wide = torch.zeros(n, vocab + 1, device="cuda", dtype=dtype)
        wide[:, 1:] = x
        x = wide[:, 1:]
    g = torch.Generator(device="cuda").manual_seed(vocab)
    gl = torch.randn(n, generator=g, device="cuda")
    ge = 0.1 * torch.randn(n, generator=g, device="cuda")
    fwd = M.token_logprobs(x, y, temperature=temperature)
    d = torch.empty(n, vocab, device="cuda", dtype=dtype)
    M.token_logprobs_backward(x, y, fwd, gl, ge, temperature=temperature, out=d)
    got = d.gather(1, y.long()[:, None])[:, 0].double()
    z = (x.double() - x.double().amax(1, keepdim=True)) / temperature
    e = torch.where(z == 0, 0.0, z.exp())
    r = e.sum(1)
    lp, q = -torch.log1p(r), r / (1 + r)
    h = torch.log1p(r) - (z * e).sum(1) / (1 + r)
    one, two = gl.double() * q, ge.double() * (1 - q)
    exact = (one - two * (lp + h)) / temperature
    far = -z.amin(1)
    bound = (3 * far + 4 + vocab / 256 + 64 + 16) * 2.0 ** -24
    slack = bound * (one.abs() + two.abs() * (lp.abs() + 2 * h)) / temperature
    unit = 2.0 ** -24
    assert ((got - exact).abs() <= slack * (1 + unit) + unit * exact.abs() + vocab * 2.0 ** -120).all()

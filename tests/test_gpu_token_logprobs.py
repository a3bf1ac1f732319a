"""Token log probabilities, entropy, alternatives and their gradient against
64-bit formulas.

Tolerances. Scaled logits y = x / T carry a relative error of 2^-23 (one
product), and differences y - M reach 2 max|y|; the exponentials and sums add
2^-20 relative at most (V terms summed by 256 threads and a tree, each partial
sum of at most V / 256 terms, random rounding; exp2f within 2 units). So log p
is within 2^-19 + 2^-22 * span for a row whose logits span `span` (scaled), the
entropy within that times (1 + its own size). A gradient row has two factors
of that kind: relative 2^-17 of |g_lp| + |g_H| (|log p| + H), and half a unit of
its type.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


def logits_of(seed, n, v, dtype, std=3.0, pad=0, shift=0):
    """[n, v] with rows v + pad elements apart, the first one `shift` elements in."""
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(n * (v + pad) + shift, generator=g) * std).to(dtype).to(DEV)
    return flat[shift:].view(n, v + pad)[:, :v]


def exact(logits, targets, t):
    y = logits.double() / t
    m = y.amax(1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(y - m)
    z = e.sum(1, keepdim=True)
    logp = y - m - z.log()
    p = e / z
    ent = torch.special.entr(p).sum(1)
    lp = None if targets is None else logp.gather(1, targets.long().clamp(min=0)[:, None])[:, 0]
    return logp, p, ent, lp


def span_of(logits, t):
    x = logits.double()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    return 2 * x.abs().amax(1) / t


SHAPES = [(1, 1), (3, 7), (2, 33), (5, 1000), (1, 4099), (4, 16384), (2, 100003), (33, 513), (200, 257),
          (1, 131072), (40, 20001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", SHAPES)
@pytest.mark.parametrize("t,pad,shift,wide", [(1.0, 0, 0, False), (0.7, 5, 1, True), (2.5, 8, 0, False)])
def test_forward(n, v, dtype, t, pad, shift, wide):
    x = logits_of(n * v, n, v, dtype, pad=pad, shift=shift)
    y = torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(1)).to(DEV)
    y = y if wide else y.to(torch.int32)
    k = min(v, 20)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = M.token_logprobs(x, y, temperature=t, alternatives=k, status=status)
    logp, p, ent, lp = exact(x, y, t)
    tol = 2.0 ** -19 + 2.0 ** -22 * span_of(x, t)
    assert ((r["logprob"].double() - lp).abs() <= tol).all()
    assert ((r["entropy"].double() - ent).abs() <= tol * (1 + ent)).all()
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r["alt_ids"].long(), ids)
    assert ((r["alt_logprobs"].double() - logp.gather(1, ids)).abs() <= tol[:, None]).all()
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 2, 31, 32])
def test_alternatives_with_ties_and_orders(dtype, k):
    """Equal logits (whole rows of them), sorted rows, signed zeros."""
    v = 5000
    rows = [torch.zeros(v), torch.arange(v).float() / 8, -torch.arange(v).float() / 8,
            (torch.arange(v) % 3).float(), torch.where(torch.arange(v) % 2 == 0, 0.0, -0.0),
            torch.arange(v).float().remainder(97).neg()]
    x = torch.stack(rows).to(dtype).to(DEV)
    r = M.token_logprobs(x, alternatives=k)
    assert r["logprob"] is None
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r["alt_ids"].long(), ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [64, 3001, 70001])
def test_masked_logits(dtype, v):
    """-inf almost everywhere, everywhere, the type's lowest value, few tokens left."""
    x = logits_of(v, 6, v, dtype)
    x[0, 5:] = -INF                       # five tokens left
    x[1] = -INF                           # nothing left
    x[2] = torch.finfo(dtype).min         # the mask's value everywhere: a uniform row
    x[3, 1:] = torch.finfo(dtype).min     # one token left
    x[4, :-1] = -INF                      # the last one left
    x[5, ::2] = -INF
    y = torch.tensor([3, 2, 7, 0, v - 1, 0], dtype=torch.int32, device=DEV)   # row 5: a masked token
    k = 8
    r = M.token_logprobs(x, y, alternatives=k)
    g1, g2 = torch.full((6,), 0.5, device=DEV), torch.full((6,), -0.25, device=DEV)
    d = M.token_logprobs_backward(x, y, r, g1, g2)
    lp, h = r["logprob"].double().cpu(), r["entropy"].double().cpu()
    logp, p, ent, want = exact(x, y, 1.0)
    tol = 2.0 ** -19 + 2.0 ** -22 * 30
    for i in (0, 4):
        assert abs(lp[i] - want[i].cpu()) <= tol and abs(h[i] - ent[i].cpu()) <= tol * (1 + ent[i].cpu())
    assert lp[1] == -INF and h[1] == 0 and (r["alt_ids"][1] == -1).all()
    assert (r["alt_logprobs"][1] == -INF).all() and (d[1] == 0).all()
    assert abs(lp[2] + math.log(v)) <= tol and abs(h[2] - math.log(v)) <= tol * (1 + math.log(v))
    assert torch.equal(r["alt_ids"][2].cpu(), torch.arange(k, dtype=torch.int32))
    assert lp[3] == 0 and h[3] == 0 and r["alt_ids"][3, 0] == 0
    assert r["alt_ids"][0, 5:].tolist() == [-1] * 3 and (r["alt_logprobs"][0, 5:] == -INF).all()
    assert sorted(r["alt_ids"][0, :5].tolist()) == [0, 1, 2, 3, 4]
    assert r["alt_ids"][4].tolist() == [v - 1] + [-1] * 7 and lp[4] == 0 and h[4] == 0
    assert lp[5] == -INF and (r["alt_ids"][5] % 2 == 1).all()
    assert torch.isfinite(d.float()).all()
    # masked tokens get no gradient, but for the given token's own part
    assert (d[0, 5:] == 0).all() and (d[5, 2::2] == 0).all() and d[5, 0] == 0.5
    # the uniform row: every probability is 1 / v, the entropy's gradient is 0
    uni = torch.full((v,), -0.5 / v, dtype=torch.float64)
    uni[7] += 0.5
    assert (d[2].double().cpu() - uni).abs().max() <= 0.5 * 2.0 ** -8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_and_nan_logits_stay_in_their_row(dtype):
    x = logits_of(7, 4, 2000, dtype)
    ref = M.token_logprobs(x, alternatives=4)
    x[1, 77] = INF
    x[2, 1999] = float("nan")
    y = torch.zeros(4, dtype=torch.int64, device=DEV)
    r = M.token_logprobs(x, y, alternatives=4)
    for i in (1, 2):
        assert torch.isnan(r["logprob"][i]) and torch.isnan(r["entropy"][i])
        assert (r["alt_ids"][i] == -1).all() and torch.isnan(r["alt_logprobs"][i]).all()
    for i in (0, 3):
        assert torch.equal(r["alt_ids"][i], ref["alt_ids"][i])
        assert torch.isfinite(r["logprob"][i])


def test_rows_without_a_token_and_tokens_out_of_range():
    n, v = 6, 3000
    x = logits_of(9, n, v, torch.bfloat16)
    x[1] = float("nan")       # never read
    y = torch.tensor([5, -1, v, 2, -100, v - 1], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = M.token_logprobs(x, y, alternatives=2, status=status)
    assert int(status.item()) == 1 << M.ERR_BAD_TOKEN
    for i in (1, 4):
        assert r["logprob"][i] == 0 and r["entropy"][i] == 0 and r["alt_ids"][i].tolist() == [-1, -1]
    assert torch.isnan(r["logprob"][2]) and torch.isfinite(r["entropy"][2])
    status.zero_()
    d = M.token_logprobs_backward(x, y, r, torch.ones(n, device=DEV), torch.ones(n, device=DEV), status=status)
    assert int(status.item()) == 1 << M.ERR_BAD_TOKEN
    for i in (1, 2, 4):
        assert (d[i] == 0).all()
    for i in (0, 3, 5):
        assert (d[i] != 0).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 7), (5, 1000), (2, 100003), (70, 257), (3, 16390)])
@pytest.mark.parametrize("t,pad,which,inplace", [(1.0, 0, "both", False), (0.7, 3, "both", True),
                                                 (1.5, 0, "logprob", False), (1.0, 8, "entropy", True)])
def test_gradient_against_the_formula(n, v, dtype, t, pad, which, inplace):
    x = logits_of(n + v, n, v, dtype, pad=pad)
    g = torch.Generator().manual_seed(3)
    y = torch.randint(0, v, (n,), generator=g).to(DEV)
    gl = torch.randn(n, generator=g).to(DEV) if which != "entropy" else None
    gh = torch.randn(n, generator=g).to(DEV) if which != "logprob" else None
    logp, p, ent, _ = exact(x, y, t)
    a = torch.zeros(n, device=DEV).double() if gl is None else gl.double()
    b = torch.zeros(n, device=DEV).double() if gh is None else gh.double()
    want = -p * (a[:, None] + b[:, None] * (logp + ent[:, None]))
    mag = p * (a.abs()[:, None] + b.abs()[:, None] * (logp.abs() + ent[:, None]))
    want.scatter_add_(1, y[:, None], a[:, None])
    mag.scatter_add_(1, y[:, None], a.abs()[:, None])
    want, mag = want / t, mag / t
    tol = mag * (2.0 ** -17 + 2.0 ** -21 * span_of(x, t)[:, None])
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8
    r = M.token_logprobs(x, y, temperature=t)
    d = M.token_logprobs_backward(x, y, r, gl, gh, temperature=t, out=x if inplace else None)
    assert d.dtype == dtype and (d.data_ptr() == x.data_ptr()) == inplace
    assert ((d.double() - want).abs() <= tol + 1e-38).all()


def test_gradient_against_differences():
    """Central differences of the forward along a direction u: truncation
    h^2 / 6 |f'''| with |f'''| <= 8 max|u|^3 (1 + H), rounding 2 * 2^-19 (1 + H) / 2h."""
    n, v, h = 8, 600, 2.0 ** -6
    x = logits_of(21, n, v, torch.float32, std=2.0)
    g = torch.Generator().manual_seed(4)
    u = (torch.rand(n, v, generator=g) - 0.5).to(DEV)
    y = torch.randint(0, v, (n,), generator=g).to(DEV)
    one, zero = torch.ones(n, device=DEV), None
    r = M.token_logprobs(x, y)
    up, down = M.token_logprobs(x + h * u, y), M.token_logprobs(x - h * u, y)
    tol = (h * h / 6 * 8 * 0.125 + 2 * 2.0 ** -18 / (2 * h)) * (1 + r["entropy"].double())
    for key, gl, gh in (("logprob", one, zero), ("entropy", zero, one)):
        d = M.token_logprobs_backward(x, y, r, gl, gh)
        slope = (up[key].double() - down[key].double()) / (2 * h)
        assert ((slope - (d.double() * u.double()).sum(1)).abs() <= tol).all()


@pytest.mark.parametrize("v", [4099, 32000, 50001, 100003])
def test_a_rows_results_do_not_depend_on_the_batch(v):
    """Alone (a cluster for a row), among 40 rows and among 1000: the same bits."""
    x = logits_of(31, 1000, v, torch.bfloat16, pad=3)
    y = torch.arange(1000, dtype=torch.int32, device=DEV) % v
    many = M.token_logprobs(x, y, temperature=0.9, alternatives=7)
    for n in (1, 40):
        few = M.token_logprobs(x[960:960 + n], y[960:960 + n], temperature=0.9, alternatives=7)
        for key in ("logprob", "entropy", "stats", "alt_ids", "alt_logprobs"):
            assert torch.equal(few[key], many[key][960:960 + n]), key


def test_no_targets_and_no_rows():
    x = logits_of(11, 9, 700, torch.bfloat16)
    r = M.token_logprobs(x)
    assert r["logprob"] is None and r["alt_ids"] is None
    d = M.token_logprobs_backward(x, None, r, None, torch.ones(9, device=DEV))
    logp, p, ent, _ = exact(x, None, 1.0)
    want = -p * (logp + ent[:, None])
    assert ((d.double() - want).abs() <= want.abs() * 2.0 ** -8 + p * (logp.abs() + ent[:, None]) * 2.0 ** -16).all()
    empty = M.token_logprobs(x[:0], torch.empty(0, dtype=torch.int32, device=DEV), alternatives=3)
    assert empty["logprob"].numel() == 0 and empty["alt_ids"].shape == (0, 3)


def test_rows_beyond_32_bit_offsets():
    """Logits of more than 2^31 elements: the last rows are read and written in place."""
    n, v = 16500, 131072
    x = torch.zeros((n, v), dtype=torch.bfloat16, device=DEV)
    x[-1] = logits_of(12, 1, v, torch.bfloat16)[0]
    y = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    y[-1] = 17
    r = M.token_logprobs(x, y, alternatives=4)
    ref = M.token_logprobs(x[-1:].clone(), y[-1:], alternatives=4)
    for key in ("logprob", "entropy", "alt_ids", "alt_logprobs"):
        assert torch.equal(r[key][-1:], ref[key])
    last = x[-1:].clone()
    d = M.token_logprobs_backward(x, y, r, torch.ones(n, device=DEV), None, out=x)
    assert torch.equal(d[-1:], M.token_logprobs_backward(last, y[-1:], ref, torch.ones(1, device=DEV), None))
    assert (d[-3:-1] == 0).all()


def test_another_stream():
    x = logits_of(13, 64, 30000, torch.bfloat16)
    y = torch.zeros(64, dtype=torch.int32, device=DEV)
    ref = M.token_logprobs(x, y, alternatives=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.token_logprobs(x, y, alternatives=5, stream=s)
    d = M.token_logprobs_backward(x, y, got, ref["entropy"], ref["entropy"], stream=s)
    s.synchronize()
    for key in ("logprob", "entropy", "alt_ids", "alt_logprobs"):
        assert torch.equal(got[key], ref[key])
    assert torch.equal(d, M.token_logprobs_backward(x, y, ref, ref["entropy"], ref["entropy"]))

"""Draft verification: which tokens a race can be won by, whatever the variates' signs.

A token whose variate is negative or NaN never wins, one whose variate is 0 (of either
sign) wins where its weight is above 0, and a token without weight (that the draft
distribution gives at least what the target does) never wins.

Tolerances. With at most 64 tokens and logits within 16 of each other a probability is off
by at most TOL = 2^-17 + 2^-22 (16 * 1.45 + 6) of itself (see test_gpu_verify_drafts.py), a
weight by TOL (p + q), a quotient by 2^-23 of it besides: of two quotients nearer to
each other than that either may win. A token is taken to have a weight, or to have
none, where |p - q| is beyond TOL (p + q); the others get a variate that never wins.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TOL = 2.0 ** -17 + 2.0 ** -22 * (16 * 1.45 + 6)


def case(seed, B, V, dtype):
    """A draft that falls in every sequence: p, q, the draft, and what the call takes."""
    g = torch.Generator().manual_seed(seed)
    target = (torch.randn(B, 2, V, generator=g) * 1.5).clamp(-8, 8).to(dtype)
    draft = (target[:, :1].float() + torch.randn(B, 1, V, generator=g)).clamp(-8, 8).to(dtype)
    p, q = torch.softmax(target[:, 0].double(), 1), torch.softmax(draft[:, 0].double(), 1)
    x = (q - p).argmax(1)
    u = torch.full((B, 1), 0.9999)
    assert (0.9999 * (q - p * 1.001).gather(1, x[:, None]) > 0).all()
    e = torch.empty(B, V).exponential_(generator=g).clamp_(min=1e-6)
    return target, draft, p, q, x, u, e, g


def expect(weights, both, e, got):
    """got[b] has a quotient that is the largest but for roundings; with variates of 0 it is
    the first token that has one and a weight."""
    for b in range(e.shape[0]):
        w, v = weights[b], e[b].double()
        may = (w > 0) & (v >= 0)              # NaN: no
        zero = may & (v == 0)
        new = int(got[b])
        if not may.any():
            assert new == -1, b
        elif zero.any():
            assert new == int(zero.nonzero()[0]), b
        else:
            race = torch.where(may, w / v.clamp(min=1e-30), 0.0)
            err = torch.where(may, (TOL * both[b] + 2.0 ** -23 * w) / v.clamp(min=1e-30), 0.0)
            assert new >= 0 and bool(may[new]) and race[new] + err[new] >= (race - err).max(), (b, new)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("odd", [-1.0, -1e-6, -0.0, 0.0, math.nan, -math.nan, -math.inf, math.inf, -1e-40])
@pytest.mark.parametrize("where", ["q above p", "p above q", "anywhere"])
def test_after_a_draft_that_falls(dtype, odd, where):
    B, V = 96, 61
    target, draft, p, q, x, u, e, g = case(11, B, V, dtype)
    unclear = (p - q).abs() <= TOL * (p + q)
    e[unclear] = -1.0
    some = torch.rand(B, V, generator=g) < 0.3
    if where == "q above p":
        some &= q > p
    elif where == "p above q":
        some &= p > q
    e[some & ~unclear] = odd
    status = torch.zeros(1, dtype=I32, device=DEV)
    r = M.verify_drafts(target.to(DEV), x[:, None].to(I32).to(DEV), u.to(DEV), e.to(DEV), draft_logits=draft.to(DEV),
                        status=status)
    assert int(status) == 0 and (r["accepted"] == 0).all()
    left = torch.where(q > p, 0.0, p - q)
    has = ((left > 0) & (e >= 0) & ~torch.isinf(e)).any(1)
    assert has.all()                          # every sequence has a token that may win
    e = torch.where(torch.isinf(e), -1.0, e)  # an infinite one wins nothing either
    expect(left, p + q, e, r["tokens"][:, 0].cpu())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("odd", [-1.0, -0.0, 0.0, math.nan, -1e-40])
@pytest.mark.parametrize("drafted", ["none", "missing", "looked up"])
def test_without_a_draft_distribution(dtype, odd, drafted):
    """One token sampled, by a sequence without drafts or after a looked-up one that fell."""
    B, V = 96, 53
    target, _, p, _, x, u, e, g = case(12, B, V, dtype)
    e[torch.rand(B, V, generator=g) < 0.3] = odd
    weights = p.clone()
    if drafted == "none":
        r = M.verify_drafts(target[:, :1].contiguous().to(DEV), torch.zeros(B, 0, dtype=I32, device=DEV),
                            torch.zeros(B, 0, device=DEV), e.to(DEV))
    else:
        tokens = x if drafted == "looked up" else torch.full_like(x, -1)
        u = torch.full((B, 1), 0.99999)       # p of 61 such logits is below it
        r = M.verify_drafts(target.to(DEV), tokens[:, None].to(I32).to(DEV), u.to(DEV), e.to(DEV))
        if drafted == "looked up":
            weights.scatter_(1, x[:, None], 0.0)
    assert (r["accepted"] == 0).all()
    expect(weights, weights, e, r["tokens"][:, 0].cpu())


def test_no_variate_that_may_win():
    B, V = 8, 40
    target, draft, p, q, x, u, e, g = case(13, B, V, F32)
    call = lambda noise: M.verify_drafts(target.to(DEV), x[:, None].to(I32).to(DEV), u.to(DEV), noise.to(DEV),
                                         draft_logits=draft.to(DEV))
    for bad in (-1.0, math.nan, math.inf):
        r = call(torch.full((B, V), bad))
        assert (r["tokens"] == -1).all() and torch.isnan(r["logprobs"][:, 0]).all() and (r["accepted"] == 0).all()
    # where p - q leaves nothing that may win p is sampled from
    e[p >= q] = -1.0
    r = call(e)
    expect(p, p, e, r["tokens"][:, 0].cpu())


def test_a_whole_row_of_odd_variates():
    """Rows long enough for whole rounds of the race and several CTAs."""
    B, V = 3, 40009
    g = torch.Generator().manual_seed(5)
    target = torch.randn(B, 2, V, generator=g)
    draft = target[:, :1].clone()
    draft[:, 0, 100:200] += 3.0               # q above p here, and a little below it elsewhere
    draft[:, 0, 30000] -= 5.0                 # but for one token that the target wants more
    x = torch.full((B, 1), 150, dtype=I32)
    e = torch.ones(B, V)
    e[:, 100:200] = torch.tensor([-1.0, -0.0, 0.0, math.nan]).repeat(25)
    e[0, 30000], e[1, 30000], e[2, 30000] = -0.0, 0.0, 1e-3
    r = M.verify_drafts(target.to(DEV), x.to(DEV), torch.full((B, 1), 0.9999, device=DEV), e.to(DEV),
                        draft_logits=draft.to(DEV))
    assert r["accepted"].tolist() == [0] * B and r["tokens"][:, 0].tolist() == [30000] * B

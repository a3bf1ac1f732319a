"""Verification of drafted tokens against the definition in 64 bits.

Tolerances. A probability is 2^((x - m) k - log2 s): the difference, the product and
the sum are each off by 2^-24 of a number up to span = max |x - m| k + log2 V, the
exponential by 2 units, the sum of exponentials by at most (64 + 20) 2^-24: together
TOL = 2^-17 + 2^-22 span, relative, is beyond it. A draft whose u q is within 2 TOL of
p may go either way, and of two quotients within each one's error either may win;
everything else has to be as computed. Log probabilities are within 2^-17 + 2^-22 span.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = math.inf


def strided(g, b, r, v, dtype, pad, shift, std=2.0):
    flat = (torch.randn(b * r * (v + pad) + shift, generator=g) * std).to(dtype).to(DEV)
    return flat[shift:].view(b, r, v + pad)[..., :v]


def inputs(seed, B, S, V, dtype, by_model, pad=0, shift=0, ragged=True):
    g = torch.Generator().manual_seed(seed)
    target = strided(g, B, S + 1, V, dtype, pad, shift)
    draft = None
    if by_model:
        draft = strided(g, B, S, V, dtype, pad, shift)
        draft.copy_((target[:, :S].float() + 0.5 * draft.float()).to(dtype))
    q = torch.softmax((target[:, :S] if draft is None else draft).float().cpu() / 0.7, 2).reshape(B * S, V)
    tokens = torch.multinomial(q, 1, generator=g).view(B, S).to(I32) if S else torch.zeros(B, 0, dtype=I32)
    if ragged and S:
        cut = torch.randint(0, 2 * S, (B, 1), generator=g)
        tokens[torch.arange(S)[None] >= cut] = -1
    u = torch.rand(B, S, generator=g)
    e = torch.empty(B, V).exponential_(generator=g).clamp_(min=1e-20)
    return target, draft, tokens.to(DEV), u.to(DEV), e.to(DEV)


def check(target, draft, tokens, u, e, t, r):
    """r is what the definition says, but for what is within rounding of its borders."""
    B, S1, V = target.shape
    S = S1 - 1
    y = target.double().cpu() / t
    logp = torch.log_softmax(y, 2)
    z = None if draft is None else torch.softmax(draft.double().cpu() / t, 2)
    finite = torch.where(torch.isfinite(y), y, 0.0)
    span = (2 * finite.abs().amax(2) * 1.45 + math.log2(V) + 1)
    if draft is not None:
        d = draft.double().cpu()
        span = torch.maximum(span, torch.cat([2 * torch.where(torch.isfinite(d), d, 0.0).abs().amax(2) / t * 1.45,
                                              torch.zeros(B, 1)], 1) + math.log2(V) + 1)
    tol = 2.0 ** -17 + 2.0 ** -22 * span
    got, n, lp = r["tokens"].cpu(), r["accepted"].cpu().tolist(), r["logprobs"].cpu()
    drafts, us, ev = tokens.cpu().tolist(), u.cpu(), e.double().cpu()
    for b in range(B):
        given = next((i for i in range(S) if drafts[b][i] < 0), S)
        assert 0 <= n[b] <= given
        for i in range(min(n[b] + 1, given)):
            x = drafts[b][i]
            p = float(logp[b, i, x].exp())
            q = 1.0 if z is None else float(z[b, i, x])
            uq = float(us[b, i]) * q
            if i < n[b]:
                assert uq < p + 2 * float(tol[b, i]) * (p + uq), (b, i)
                assert int(got[b, i]) == x
            else:
                assert uq >= p - 2 * float(tol[b, i]) * (p + uq), (b, i)
        i = n[b]
        p = logp[b, i].exp()
        rest, err = p.clone(), p.clone()
        if i < given:
            other = z[b, i] if z is not None else torch.zeros(V, dtype=torch.float64).index_fill_(0, torch.tensor([drafts[b][i]]), 1.0)
            rest, err = (p - other).clamp(min=0), p + other
        err = (float(tol[b, i]) * err + 2.0 ** -23 * rest) / ev[b]
        race = rest / ev[b]
        new = int(got[b, i])
        assert 0 <= new < V
        assert race[new] + err[new] >= (race - err).max(), (b, i, new)
        assert (got[b, i + 1:] == -1).all() and (lp[b, i + 1:] == 0).all()
        for j in range(i + 1):
            want = float(logp[b, j, int(got[b, j])])
            assert abs(float(lp[b, j]) - want) <= float(tol[b, j]) * (1 + 0.01 * abs(want)), (b, j)


SHAPES = [(1, 0, 1), (1, 1, 2), (3, 2, 7), (2, 31, 33), (5, 4, 1000), (40, 3, 515), (1, 4, 8192), (2, 5, 40003),
          (300, 1, 130), (1, 0, 131072), (3, 2, 100003)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,S,V", SHAPES)
@pytest.mark.parametrize("by_model", [True, False])
@pytest.mark.parametrize("t,pad,shift", [(1.0, 0, 0), (0.7, 5, 1), (2.0, 8, 8)])
def test_against_the_definition(B, S, V, dtype, by_model, t, pad, shift):
    a = inputs(B + S + V, B, S, V, dtype, by_model, pad, shift)
    target, draft, tokens, u, e = a
    status = torch.zeros(1, dtype=I32, device=DEV)
    r = M.verify_drafts(target, tokens, u, e, draft_logits=draft, temperature=t, status=status)
    assert int(status) == 0
    check(*a, t, r)


def test_types_may_differ_and_noise_may_be_strided():
    target, draft, tokens, u, e = inputs(5, 6, 3, 301, BF, True)
    wide = torch.full((6, 320), -1.0, device=DEV)
    wide[:, :301] = e
    r = M.verify_drafts(target, tokens, u, wide[:, :301], draft_logits=draft.float())
    want = M.verify_drafts(target.float(), tokens, u, e, draft_logits=draft.float())
    check(target, draft, tokens, u, e, 1.0, r)
    assert torch.equal(r["tokens"], want["tokens"])


def test_masked_tokens():
    """A masked draft falls, a masked token is never sampled, one the draft model masks may be."""
    B, S, V = 64, 2, 50
    for low in (-INF, torch.finfo(F32).min):
        target, draft, tokens, u, e = inputs(9, B, S, V, F32, True, ragged=False)
        target[:, :, ::2] = low
        tokens[:, 0] = 4                      # masked by the target
        r = M.verify_drafts(target, tokens, u, e, draft_logits=draft)
        assert (r["accepted"] == 0).all() and (r["tokens"][:, 0] % 2 == 1).all()
        check(target, draft, tokens, u, e, 1.0, r)
        tokens[:, 0] = 5
        draft[:, 0, 5] = low                  # q = 0: stands
        assert (M.verify_drafts(target, tokens, u, e, draft_logits=draft)["accepted"] >= 1).all()
        one = torch.full((B, S + 1, V), low, device=DEV)
        one[..., 7] = 3.0                     # one token left: certain
        tokens[:, 0], tokens[:, 1] = 7, 8
        r = M.verify_drafts(one, tokens, u, e)
        assert (r["accepted"] == 1).all() and (r["tokens"][:, :2] == 7).all() and (r["logprobs"] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t", [0.01, 1.0, 1e4])
def test_logits_near_the_ends_of_their_type(dtype, t):
    """Rows of the type's lowest value alone (all alike then), beside -inf, and of its
    largest; with temperatures that take m / T out of FP32's range."""
    V, low, high = 9000, torch.finfo(dtype).min, torch.finfo(dtype).max
    target = torch.full((5, 1, V), -INF, dtype=dtype, device=DEV)
    target[0] = low
    target[1, 0, 5000:] = low
    target[2, 0, 7] = low
    target[3] = high
    target[4, 0, ::3], target[4, 0, 1::3] = high, low
    ones = [V, 4000, 1, V, 3000]
    e = torch.empty(5, V).exponential_(generator=torch.Generator().manual_seed(1)).to(DEV)
    r = M.verify_drafts(target, torch.zeros(5, 0, dtype=I32, device=DEV), torch.zeros(5, 0, device=DEV), e, temperature=t)
    top = target[:, 0].float() == target[:, 0].float().amax(1, keepdim=True)
    want = torch.where(top, 1 / e, 0.0).argmax(1)
    assert r["tokens"][:, 0].tolist() == want.tolist()
    lp = torch.tensor([-math.log(n) for n in ones])
    assert ((r["logprobs"][:, 0].cpu() - lp).abs() <= 2.0 ** -17 * (1 + lp.abs())).all()


def test_rows_without_probabilities():
    target, draft, tokens, u, e = inputs(3, 6, 2, 40, F32, True, ragged=False)
    u.zero_()                                 # every draft stands that can
    target[0, 0, 3] = math.nan
    target[1, 1] = -INF
    target[2, 2, 5] = INF
    draft[3, 0, 2] = math.nan
    draft[4, 1] = -INF
    r = M.verify_drafts(target, tokens, u, e, draft_logits=draft)
    assert r["accepted"].tolist() == [0, 1, 2, 0, 1, 2]
    for b, n in enumerate([0, 1, 2, 0, 1]):
        assert int(r["tokens"][b, n]) == -1 and math.isnan(float(r["logprobs"][b, n]))
    assert int(r["tokens"][5, 2]) >= 0
    r = M.verify_drafts(target, tokens, u, e)   # without a draft model those rows are not looked at
    assert r["accepted"].tolist() == [0, 1, 2, 2, 2, 2]


def test_draft_tokens_out_of_range():
    target, draft, tokens, u, e = inputs(4, 4, 3, 40, F32, True, ragged=False)
    u.zero_()
    tokens[0, 1], tokens[1, 0], tokens[2, 2] = 40, 2 ** 31 - 1, -7
    tokens[3, 1], tokens[3, 2] = -1, 5        # a token behind the last draft is not one
    for d in (draft, None):
        status = torch.zeros(1, dtype=I32, device=DEV)
        r = M.verify_drafts(target, tokens, u, e, draft_logits=d, status=status)
        assert int(status) == 1 << M.ERR_BAD_TOKEN and r["accepted"].tolist() == [1, 0, 2, 1]
        assert (r["tokens"][torch.arange(4), r["accepted"].long()] >= 0).all()
    status = torch.zeros(1, dtype=I32, device=DEV)
    M.verify_drafts(target[2:], tokens[2:], u[2:], e[2:], draft_logits=draft[2:], status=status)
    assert int(status) == 0
    tokens[2, 2], tokens[3, 2] = -1, 40       # nor is one out of range there
    M.verify_drafts(target[2:], tokens[2:], u[2:], e[2:], draft_logits=draft[2:], status=status)
    assert int(status) == 0
    tokens[3, 1] = 41                         # the one that ends the drafts is
    M.verify_drafts(target[2:], tokens[2:], u[2:], e[2:], draft_logits=draft[2:], status=status)
    assert int(status) == 1 << M.ERR_BAD_TOKEN


def test_the_same_model_accepts_everything():
    target, _, tokens, u, e = inputs(8, 50, 4, 3001, BF, False, ragged=False)
    u.clamp_(max=0.9999)
    r = M.verify_drafts(target, tokens, u, e, draft_logits=target[:, :4].contiguous())
    assert (r["accepted"] == 4).all()


def test_nothing_left_of_p_samples_p():
    """A border that only a uniform of 1 reaches: p = q, and the draft falls all the same."""
    r = M.verify_drafts(torch.zeros(1, 2, 1, device=DEV), torch.zeros(1, 1, dtype=I32, device=DEV),
                        torch.ones(1, 1, device=DEV), torch.ones(1, 1, device=DEV))
    assert r["accepted"].tolist() == [0] and r["tokens"].tolist() == [[0, -1]] and float(r["logprobs"][0, 0]) == 0.0


def test_equal_quotients_go_to_the_lower_id():
    V = 9000
    target, e = torch.zeros(3, 1, V, device=DEV), torch.ones(3, V, device=DEV)
    target[1, 0, :17] = -1.0
    e[2, 8999] = e[2, 4500] = 0.5
    r = M.verify_drafts(target, torch.zeros(3, 0, dtype=I32, device=DEV), torch.zeros(3, 0, device=DEV), e)
    assert r["tokens"][:, 0].tolist() == [0, 17, 4500]


def test_tokens_are_distributed_as_the_target():
    """The first token of many sequences with the same logits, whatever was drafted."""
    B, V = 1 << 16, 8
    g = torch.Generator().manual_seed(1)
    t, d = torch.randn(V, generator=g), torch.randn(V, generator=g)
    p = torch.softmax(t.double() / 0.8, 0)
    target, draft = t.expand(B, 2, V).contiguous().to(DEV), d.expand(B, 1, V).contiguous().to(DEV)
    drawn = torch.multinomial(torch.softmax(d / 0.8, 0).expand(B, V), 1, generator=g).to(I32).to(DEV)
    u, e = torch.rand(B, 1, generator=g).to(DEV), torch.empty(B, V).exponential_(generator=g).to(DEV)
    fixed = torch.full((B, 1), 3, dtype=I32, device=DEV)
    for tokens, q in ((drawn, draft), (fixed, None)):
        r = M.verify_drafts(target, tokens, u, e, draft_logits=q, temperature=0.8)
        share = torch.bincount(r["tokens"][:, 0].long().cpu(), minlength=V).double() / B
        assert ((share - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all()


def test_log_probabilities_are_those_of_token_logprobs():
    target, draft, tokens, u, e = inputs(2, 30, 3, 5000, BF, True)
    r = M.verify_drafts(target, tokens, u, e, draft_logits=draft, temperature=0.9)
    lp = M.token_logprobs(target.reshape(120, 5000), r["tokens"].view(-1).contiguous(), temperature=0.9)["logprob"]
    assert torch.allclose(lp.view(30, 4), r["logprobs"], rtol=1e-5, atol=1e-5)


def test_an_almost_certain_token_keeps_its_log_probability():
    V = 40000
    target = torch.zeros(1, 1, V, device=DEV)
    target[0, 0, 123] = 22.0
    r = M.verify_drafts(target, torch.zeros(1, 0, dtype=I32, device=DEV), torch.zeros(1, 0, device=DEV),
                        torch.ones(1, V, device=DEV))
    want = -math.log1p((V - 1) * math.exp(-22.0))
    assert int(r["tokens"][0, 0]) == 123 and abs(float(r["logprobs"][0, 0]) / want - 1) <= 2.0 ** -18


def test_results_do_not_depend_on_the_other_sequences():
    target, draft, tokens, u, e = inputs(6, 70, 3, 8192, BF, True)
    r = M.verify_drafts(target, tokens, u, e, draft_logits=draft)
    for b in (0, 33, 69):
        s = slice(b, b + 1)
        one = M.verify_drafts(target[s], tokens[s], u[s], e[s], draft_logits=draft[s])
        assert all(torch.equal(one[k][0], r[k][b]) for k in one)


def test_streams_and_graphs():
    a, b = inputs(1, 20, 3, 9000, BF, True), inputs(2, 20, 3, 9000, BF, True)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda x, s=None: M.verify_drafts(x[0], x[2], x[3], x[4], draft_logits=x[1], stream=s)
    for _ in range(5):
        ra, rb = call(a, one), call(b, two)
    torch.cuda.synchronize()
    check(*a, 1.0, ra)
    check(*b, 1.0, rb)
    x = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call(x)
    for src, want in ((b, rb), (a, ra), (b, rb)):
        for t, s in zip(x, src):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r["tokens"], want["tokens"]) and torch.equal(r["accepted"], want["accepted"])


def test_no_sequences():
    r = M.verify_drafts(torch.empty(0, 3, 10, device=DEV), torch.empty(0, 2, dtype=I32, device=DEV),
                        torch.empty(0, 2, device=DEV), torch.empty(0, 10, device=DEV))
    assert r["tokens"].shape == (0, 3)


def test_logits_beyond_two_to_the_31_elements():
    B, V = 17000, 131072
    g = torch.Generator(device=DEV).manual_seed(1)
    target = torch.zeros(B, 1, V, dtype=BF, device=DEV)
    noise = torch.ones(B, V, device=DEV)
    none = torch.zeros(B, 0, dtype=I32, device=DEV), torch.zeros(B, 0, device=DEV)
    want = torch.randint(0, V, (B,), generator=g, device=DEV)
    target[torch.arange(B, device=DEV), 0, want] = 5.0
    r = M.verify_drafts(target, *none, noise)
    assert torch.equal(r["tokens"][:, 0].long(), want)
    lp = 5.0 - math.log(math.exp(5.0) + V - 1)
    assert ((r["logprobs"] - lp).abs() <= 2.0 ** -17 * 8).all()

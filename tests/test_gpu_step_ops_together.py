"""Rows by expert, grouped products, log probabilities, gradient norm, AdamW and the
verification of drafts in one run, as a learner in BF16 and its sampler use them.

Tolerances. The reference takes the same inputs through 64-bit autograd. Forward
intermediates (3 of them) and backward ones (up to 5 in a row) are rounded to BF16,
2^-8 relative each at most and independent, so that whole tensors are within a few
2^-8 of their norm: 2^-5.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M
from nvfp4_w4a4_moe_permute_gb300.learner import PolicyLearner, synthetic_batch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Layer:
    """A mixture of two-layer linear experts whose outputs are weighted at the combine,
    and a head."""

    def __init__(self, H, I, E, V):
        g = torch.Generator().manual_seed(1)
        init = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(DEV)
        self.E = E
        self.master = [init(E, I, H), init(E, H, I), init(1, V, H)]
        self.w = [m.to(BF) for m in self.master]
        self.opt = M.AdamW(self.master, copies=self.w, lr=1e-2, betas=(0.9, 0.95), weight_decay=0.0)
        self.status = torch.zeros(1, dtype=I32, device=DEV)

    def forward(self, x, ids, weights, tokens):
        st = self.status
        self.whole = torch.tensor([0, x.shape[0]], dtype=I32, device=DEV)
        self.r = M.permute_rows(x, ids, self.E, status=st)
        self.a = M.grouped_gemm_bf16(self.r["rows"], self.w[0], self.r["offsets"], status=st)
        self.b = M.grouped_gemm_bf16(self.a, self.w[1], self.r["offsets"], status=st)
        self.y = M.combine_rows(self.b, self.r["dest_row"], weights, status=st)
        self.logits = M.grouped_gemm_bf16(self.y, self.w[2], self.whole, status=st)
        return M.token_logprobs(self.logits, tokens, status=st)

    def backward(self, tokens, out, weights, grad_logprob):
        st, off, dest = self.status, self.r["offsets"], self.r["dest_row"]
        d = M.token_logprobs_backward(self.logits, tokens, out, grad_logprob, status=st)
        head = M.grouped_wgrad_bf16(d, self.y, self.whole, status=st)
        dy = M.grouped_gemm_bf16(d, self.w[2], self.whole, w_as_stored=True, status=st)
        db, dweights = M.combine_rows_backward(dy, self.b, dest, weights, status=st)
        w2 = M.grouped_wgrad_bf16(db, self.a, off, status=st)
        da = M.grouped_gemm_bf16(db, self.w[1], off, w_as_stored=True, status=st)
        w1 = M.grouped_wgrad_bf16(da, self.r["rows"], off, status=st)
        dr = M.grouped_gemm_bf16(da, self.w[0], off, w_as_stored=True, status=st)
        return [w1, w2, head], M.permute_rows_backward(dr, dest, status=st), dweights


def batch(T, H, E, k, V):
    g = torch.Generator().manual_seed(7)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(I32)
    ids[::9, 1] = -1      # dropped slots
    ids[3] = -1           # and a token without any
    w = torch.rand(T, k, generator=g).to(DEV)
    return x, ids.to(DEV), w, torch.randint(0, V, (T,), generator=g).to(I32).to(DEV), torch.rand(T, generator=g).to(DEV)


def reference(L, x, ids, w, tokens, gl):
    leaves = [p.double().clone().requires_grad_() for p in L.w] + [x.double().requires_grad_(), w.double().requires_grad_()]
    w1, w2, head, xd, wd = leaves
    y = torch.zeros_like(xd)
    for e in range(L.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = y.index_add(0, t, (xd[t] @ w1[e].t() @ w2[e].t()) * wd[t, j, None])
    logp = torch.log_softmax(y @ head[0].t(), 1).gather(1, tokens.long()[:, None])[:, 0]
    (logp * gl.double()).sum().backward()
    return logp.detach(), [p.grad for p in leaves]


def near(got, want, tol=2.0 ** -5):
    assert float((got.double() - want).norm() / want.norm()) <= tol


def test_a_step_in_bf16():
    T, H, I, E, k, V = 150, 72, 48, 5, 3, 336
    L = Layer(H, I, E, V)
    x, ids, w, tokens, adv = batch(T, H, E, k, V)
    gl = adv * (-1.0 / T)
    out = L.forward(x, ids, w, tokens)
    grads, dx, dw = L.backward(tokens, out, w, gl)
    assert int(L.status) == 0
    logp, want = reference(L, x, ids, w, tokens, gl)
    assert float((out["logprob"].double() - logp).abs().max()) <= 0.1
    for got, ref in zip(grads + [dx, dw], want):
        near(got, ref)
    assert (dw[ids < 0] == 0).all() and (dx[3] == 0).all()
    norm = math.sqrt(sum(float(g.double().norm()) ** 2 for g in grads))
    r = M.grad_norm(grads, norm / 4)
    assert abs(float(r["norm"]) / norm - 1) <= 2.0 ** -20
    # the factor in the optimizer, and the clipped gradients without one, are the same step
    M2 = Layer(H, I, E, V)
    L.opt.step(grads, grad_scale=r["scale"])
    M.clip_grads(grads, norm / 4)
    M2.opt.step(grads)
    for a, b in zip(L.master, M2.master):
        assert torch.equal(a, b)


def test_a_sampler_next_to_the_learner():
    """Drafts of the old weights verified with the new ones: their log probabilities are
    those that the learner computes."""
    T, H, I, E, k, V = 96, 64, 64, 4, 2, 504
    L = Layer(H, I, E, V)
    x, ids, w, tokens, adv = batch(T, H, E, k, V)
    out = L.forward(x, ids, w, tokens)
    old = L.logits.clone()
    L.opt.step(L.backward(tokens, out, w, adv * (-1.0 / T))[0])
    L.forward(x, ids, w, tokens)
    B, S = 24, 3
    g = torch.Generator(device=DEV).manual_seed(3)
    target, draft = L.logits.view(B, S + 1, V), old.view(B, S + 1, V)[:, :S].contiguous()
    drafted = torch.multinomial(torch.softmax(draft.float().view(B * S, V), 1), 1, generator=g).view(B, S).to(I32)
    u, e = torch.rand(B, S, generator=g, device=DEV), torch.empty(B, V, device=DEV).exponential_(generator=g)
    r = M.verify_drafts(target, drafted, u, e, draft_logits=draft, status=L.status)
    lp = M.token_logprobs(L.logits, r["tokens"].view(-1), status=L.status)["logprob"].view(B, S + 1)
    assert torch.allclose(lp, r["logprobs"], rtol=1e-5, atol=1e-5) and int(L.status) == 0
    assert 0 < int(r["accepted"].sum()) <= B * S


def test_the_policy_learner_clips_its_gradients():
    T, H, I, E, k, V = 64, 128, 64, 4, 2, 512
    a, b = (PolicyLearner(T, H, I, E, k, V, lr=5e-3) for _ in range(2))
    x, ids, w, tokens, adv = synthetic_batch(T, H, E, k, V, seed=4)
    out = a.step(x, ids, w, tokens, adv, max_grad_norm=0.01)
    norm = math.sqrt(sum(float(g.double().norm()) ** 2 for g in a.grads))
    assert abs(float(out["grad_norm"]) / norm - 1) <= 2.0 ** -20 and int(a.status) == 0
    factor = torch.tensor([0.01 / (norm + 1e-6)], device=DEV)
    b.step(x, ids, w, tokens, adv, grad_scale=factor)
    for p, q in zip(a.master, b.master):
        assert torch.allclose(p, q, rtol=0, atol=1e-6)
    with pytest.raises(M.MiniteError):
        a.step(x, ids, w, tokens, adv, grad_scale=factor, max_grad_norm=1.0)

"""The policy-update step that runs the BF16 operators together: its gradients
against 64-bit formulas on the step's own buffers, and a few steps of training.

Tolerances. The reference uses the step's own BF16 intermediates (gate_up, h, y,
logits) and takes every gradient in 64 bits from there; the step rounds each
intermediate gradient to BF16 (2^-9 relative of each element), through at most
four products in a row. Independent roundings of a product's terms average out,
so that a whole tensor is within a few 2^-9 of its norm: 2^-6 for the longest
chain.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M
from nvfp4_w4a4_moe_permute_gb300.learner import PolicyLearner, synthetic_batch

pytestmark = pytest.mark.gpu


def near(got, want, tol, what):
    err = ((got.double() - want).norm() / want.norm()).item()
    assert err <= tol, f"{what}: {err}"


def test_gradients_of_a_step():
    T, H, I, E, k, V = 96, 128, 64, 6, 2, 1000
    L = PolicyLearner(T, H, I, E, k, V, temperature=0.9)
    x, ids, w, tokens, adv = synthetic_batch(T, H, E, k, V, seed=3)
    tokens[::5] = -1
    out = L.forward(x, ids, w, tokens)
    logits, h, gu = L.logits.double(), L.h.double(), L.mlp.gate_up.double()
    y, head = L.y.double(), L.head.double()
    near(L.logits, y @ head.t(), 2.0 ** -8, "logits")
    gl, gh = adv * 0.01, torch.full_like(adv, -0.003)
    for again in (False, True):
        if again:
            L.forward(x, ids, w, tokens)
        dx = L.backward(x, tokens, out, gl, gh, accumulate=again)
        assert int(L.status.item()) == 0
        t = logits.clone().requires_grad_()
        logp = torch.log_softmax(t / 0.9, 1)
        live = (tokens >= 0).double()
        loss = (live * gl.double() * logp.gather(1, tokens.long().clamp(min=0)[:, None])[:, 0]).sum() \
            - (live * gh.double() * (logp.exp() * logp).sum(1)).sum()
        loss.backward()
        d, times = t.grad, 2.0 if again else 1.0
        near(L.grads[2], times * (d.t() @ y), 2.0 ** -7, "head")
        dy = d @ head
        off, src = L.mlp.offsets.tolist(), L.mlp.perm_src.long()
        dd, pw = dy[src], L.mlp.perm_w.double()[:, None]
        g, u = gu[:, :I], gu[:, I:]
        s = torch.sigmoid(g)
        dx_ref = dy.clone()
        for e in range(E):
            r = slice(off[e], off[e + 1])
            near(L.grads[1][e], times * (dd[r].t() @ h[r]), 2.0 ** -6, f"down {e}")
            dh = dd[r] @ L.wd[e].double()
            dg = dh * u[r] * pw[r] * s[r] * (1 + g[r] * (1 - s[r]))
            du = dh * g[r] * s[r] * pw[r]
            dgu = torch.cat([dg, du], 1)
            near(L.grads[0][e], times * (dgu.t() @ x[src][r].double()), 2.0 ** -6, f"gate_up {e}")
            dx_ref.index_add_(0, src[r], dgu @ L.wgu[e].double())
        near(dx, dx_ref, 2.0 ** -6, "x")


@pytest.mark.parametrize("bits", [8, 32])
def test_a_few_steps_raise_the_advantage(bits):
    T, H, I, E, k, V = 64, 128, 64, 4, 2, 512
    L = PolicyLearner(T, H, I, E, k, V, lr=5e-3, state_bits=bits)
    x, ids, w, tokens, adv = synthetic_batch(T, H, E, k, V, seed=4)
    seen = [(adv * L.step(x, ids, w, tokens, adv)["logprob"]).mean().item() for _ in range(8)]
    assert int(L.status.item()) == 0
    assert all(b > a for a, b in zip(seen, seen[1:])), seen
    for master, copy in zip(L.master, (L.wgu, L.wd, L.head)):
        assert torch.equal(master.to(torch.bfloat16), copy)
    ref = M.quantize(L.wgu, per_group=True)
    assert torch.equal(ref["codes"], L.wgu_q["codes"])
